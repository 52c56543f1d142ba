// Token embedding: lookup with scaling, and its gradient from sorted tokens.
//
//   out_i = scale * E[t_i]                    dE_v += scale * sum_{i: t_i = v} dout_i
//
// Forward: a copy of N rows, bound by HBM writes (rows of frequent tokens come from L2): 16384 rows
// of 5376 bf16 from a table of 262144 in 38 us (floor 37). Accesses of 32 or 16 bytes where the rows
// allow it, else two elements, else one (7547 x 4446 bf16 16 us, singly 25).
// Backward: the token positions are sorted by token (stable), so each row of dE is the sum
// of one run of the sorted list. Blocks take fixed pieces of the list; a run inside a piece
// is added to dE at once, a run that crosses pieces leaves one partial row per piece, and the
// block that leaves the last one adds them in piece order. No atomics on data: the same bits
// on every run. Bound by HBM: dout once, the touched rows of dE read and written once. 8192 rows
// of 4096 into an fp32 table of 128256: sort 10 us, sums 34 us (floor of both 27): the sums wait
// for their loads, eight rows a thread in flight at four blocks an SM. (Pairs of elements where 16
// bytes do not fit: 7547 x 4446 bf16 54 us, singly 84.)
#include <math.h>

#include <atomic>

#include "flce_ops.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------------ forward
// Block (x, y): rows x * blockDim.y ..., of each the vectors from y * U * blockDim.x on; each thread
// moves U vectors. Short rows share a block of 128 threads (21049 x 136 bf16: 4.2 us, a block each
// 12.1), but for fewer rows than SMs. Narrow accesses are bound by the instructions around them:
// eight a thread share the row's.
template <int EPV>
constexpr int FWD_U = EPV <= 2 ? 8 : 2;
template <typename T, int EPV>
__global__ void __launch_bounds__(256) k_embed_fwd(const int64_t* __restrict__ tokens, int64_t N, int64_t V, int64_t H,
                                                   int64_t ignore_index, float scale, const T* __restrict__ E,
                                                   int64_t ldE, T* __restrict__ out, int64_t ldout, int* status) {
  constexpr int U = FWD_U<EPV>;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= N) return;
  const int64_t t = tokens[row];
  const bool live = t >= 0 && t < V && t != ignore_index;
  if (!live && t != ignore_index && status != nullptr && threadIdx.x == 0 && blockIdx.y == 0)
    atomicOr(status, ST_TARGET_RANGE);
  const int64_t c0 = ((int64_t)blockIdx.y * U * blockDim.x + threadIdx.x) * EPV;
  const int left = (int)min(H - c0, (int64_t)INT32_MAX), step = (int)blockDim.x * EPV;
  const T* src = E + (live ? t : 0) * ldE + c0;
  T* dst = out + row * ldout + c0;
  Raw<T, EPV> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r[u].zero();
    if (live && u * step < left) r[u].load(src + u * step);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * step >= left) break;
    if (live && scale != 1.0f) {
      float v[EPV];
      r[u].unpack(v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) v[e] *= scale;
      r[u].pack(v);
    }
    r[u].store(dst + u * step);
  }
}

template <typename T, int EPV>
void launch_fwd(const flce_embed_args& a, cudaStream_t s) {
  // as many blocks a row as 256 threads of U vectors need, of as few threads as that takes
  constexpr int U = FWD_U<EPV>;
  const int64_t nvec = cdiv64(a.H, EPV);
  const int64_t by = cdiv64(nvec, 256 * U);
  const int threads = (int)(cdiv64(cdiv64(nvec, by * U), 32) * 32);
  const int64_t rows = threads < 128 && a.N > num_sms() ? 128 / threads : 1;
  k_embed_fwd<T, EPV><<<dim3((unsigned)cdiv64(a.N, rows), (unsigned)by), dim3((unsigned)threads, (unsigned)rows), 0, s>>>(
      a.tokens, a.N, a.V, a.H, a.ignore_index, a.scale, (const T*)a.E, a.ldE, (T*)a.out, a.ldout, a.status);
}

template <typename T>
cudaError_t fwd(const flce_embed_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  auto fits = [&](int bytes) {
    return a.H % (bytes / (int)sizeof(T)) == 0 && rows_by(a.E, a.ldE, sizeof(T), bytes) &&
           rows_by(a.out, a.ldout, sizeof(T), bytes);
  };
  if (fits(32)) launch_fwd<T, 2 * W>(a, s);
  else if (fits(16)) launch_fwd<T, W>(a, s);
  else if (fits(2 * sizeof(T))) launch_fwd<T, 2>(a, s);
  else launch_fwd<T, 1>(a, s);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ sort
// Stable radix sort of (token, position) by one cluster of blocks. Keys are the tokens, V for
// ignored and out-of-range ones (they sort last and are left out). Each warp owns a contiguous
// part of the list; a pass counts the digits per warp, adds the counts up over the warps, the
// blocks (through distributed shared memory) and the digits, and scatters each pair to its
// place. Two passes of up to 10 bits do for a vocabulary below 2^20.
//
// Short lists are bound by latency: k_sort_reg keeps its pairs and their ranks in registers and
// passes the pairs on through the cluster's shared memory (8192 tokens: 10 us; with the pairs in
// L2 and ranked twice a pass: 15 us). One block without cluster barriers takes up to 1024
// tokens. k_sort takes lists of any length, with the pairs in L2.
// Digits have 8, 9 or 10 bits, known to the compiler: the fewest that keep the passes.
constexpr int SORT_CTAS = 8;
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_BITS = 10;

struct SortArgs {
  const int64_t* tokens;
  int64_t ignore_index;
  int64_t V;
  int N;
  int passes;
  uint32_t *k0, *p0;   // sorted keys and positions
  uint32_t *k1, *p1;   // the other list of k_sort, which starts in the one that makes it end in k0
  int* status;
  int* count;          // [pieces][slices] zeroed for k_embed_sum
  int ncount;
  // what the launch's other blocks zero (FLCE_FLAG_DW_OVERWRITE): `zrows` rows of `zlen` bytes, at
  // a pitch of `zpitch`; zrows = 0: nothing, and no other blocks
  uint8_t* zero;
  int64_t zrows, zlen, zpitch;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_remote(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote_addr(p, rank)), "r"(v) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void sort_barrier() {
  if constexpr (CTAS > 1) cluster_barrier();
  else __syncthreads();
}

// The key of position i: its token, V where that takes no part.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int i) {
  const int64_t t = a.tokens[i];
  const bool live = t >= 0 && t < a.V && t != a.ignore_index;
  if (!live && t != a.ignore_index && a.status != nullptr) atomicOr(a.status, ST_TARGET_RANGE);
  return live ? (uint32_t)t : (uint32_t)a.V;
}
// The lanes of `act` whose digit is this lane's: a ballot per bit (the match instruction takes a
// step per different digit: 1500 cycles for a tile of each of 32 warps).
template <int BITS>
__device__ __forceinline__ unsigned same_digit(unsigned act, uint32_t d) {
  unsigned peers = act;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const unsigned m = __ballot_sync(act, d >> b & 1u);
    peers &= d >> b & 1u ? m : ~m;
  }
  return peers;
}

// Turns the warps' digit counts hist[w][bin] into the places of their first elements: sums over
// the warps, the blocks of the cluster, and the digits before. Thread t has digits t * BPT ....
// tot: [CTAS][bins], where every block leaves its counts in every block.
template <int CTAS, int BITS>
__device__ __forceinline__ void sort_places(uint32_t* hist, uint32_t* tot, uint32_t* wsum, int rank) {
  constexpr int BINS = 1 << BITS, BPT = BINS > SORT_THREADS ? BINS / SORT_THREADS : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool mine = tid * BPT < BINS;
  uint32_t c[BPT][SORT_WARPS], before[BPT], all[BPT], sum = 0;
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    const int b = tid * BPT + i;
    before[i] = all[i] = 0;
    if (mine) {
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) c[i][w] = hist[w * BINS + b];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) all[i] += c[i][w];
      if constexpr (CTAS > 1) {
#pragma unroll
        for (int r = 0; r < CTAS; ++r) st_remote(tot + rank * BINS + b, r, all[i]);
      }
    }
  }
  if constexpr (CTAS > 1) {
    cluster_barrier();
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      if (mine) {
        all[i] = 0;
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
          const uint32_t v = tot[r * BINS + tid * BPT + i];
          before[i] += r < rank ? v : 0;
          all[i] += v;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < BPT; ++i) sum += all[i];
  uint32_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  uint32_t base = x - sum;
#pragma unroll
  for (int w = 0; w < SORT_WARPS; ++w) base += w < warp ? wsum[w] : 0;
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    if (mine) {
      uint32_t at = base + before[i];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        hist[w * BINS + tid * BPT + i] = at;
        at += c[i][w];
      }
    }
    base += all[i];
  }
  __syncthreads();
}

template <int CTAS>
__device__ __forceinline__ void sort_prepare(const SortArgs& a, int rank) {
  for (int i = rank * SORT_THREADS + (int)threadIdx.x; i < a.ncount; i += CTAS * SORT_THREADS) a.count[i] = 0;
}

// hist, tot, wsum and the pairs held in shared memory
constexpr size_t sort_smem(int ctas, int bits, int held) {
  return ((size_t)(SORT_WARPS + ctas) << bits) * 4 + SORT_WARPS * 4 + (size_t)held * 8;
}

// The blocks behind those that sort: zeroes, while few SMs are busy with the list. The rows that
// tokens point to are written again by the sums; that costs less than finding out which they are.
// Block z of nz takes every nz-th piece of 64 KB (of a row, where rows lie apart), and one thread
// copies it from zeroed shared memory (32000 x 1003 fp16, 2999 tokens: 22 us for the call, by
// stores of all threads 24). Two blocks an SM: with one, the clusters of eight that did not fit at
// first left SMs idle (28 us; 128256 x 4096 fp32 361 against 546).
constexpr int64_t ZERO_CHUNK = 65536;
__device__ __forceinline__ void zero_rows(const SortArgs& a, int z, int nz, uint4* zeros) {
  constexpr int ZEROS = 16384;
  static_assert(ZEROS <= sort_smem(1, 8, 0), "the smallest launch's shared memory");
  for (int t = threadIdx.x; t < ZEROS / 16; t += SORT_THREADS) zeros[t] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  const uint32_t src = (uint32_t)__cvta_generic_to_shared(zeros);
  const int64_t per = (a.zlen + ZERO_CHUNK - 1) / ZERO_CHUNK, all = a.zrows * per;
  for (int64_t i = z; i < all; i += nz) {
    const int64_t row = i / per, o = (i - row * per) * ZERO_CHUNK;
    uint8_t* p = a.zero + row * a.zpitch + o;
    const int64_t len = min(ZERO_CHUNK, a.zlen - o);
    // two bytes at a time up to a 16-byte boundary, multiples of 16 bytes, two bytes at a time again
    const int64_t head = min((int64_t)((16 - (uintptr_t)p % 16) % 16), len);
    const int64_t tail = head + (len - head) / 16 * 16;
    if (threadIdx.x == 0) {
      for (int64_t t = head; t < tail; t += ZEROS)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p + t), "r"(src),
                     "r"((uint32_t)min((int64_t)ZEROS, tail - t))
                     : "memory");
    }
    for (int64_t t = 2 * threadIdx.x; t < head; t += 2 * SORT_THREADS) *(uint16_t*)(p + t) = 0;
    for (int64_t t = tail + 2 * threadIdx.x; t < len; t += 2 * SORT_THREADS) *(uint16_t*)(p + t) = 0;
  }
  if (threadIdx.x == 0) {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

// TILES tiles of 32 pairs per warp. Pairs past N have the largest key and stay behind the others.
template <int CTAS, int TILES, int BITS>
__global__ void __launch_bounds__(SORT_THREADS, 1) k_sort_reg(const __grid_constant__ SortArgs a) {
  constexpr int PER = SORT_WARPS * TILES * 32;  // pairs per block
  constexpr int BINS = 1 << BITS;
  constexpr uint32_t MASK = BINS - 1;
  extern __shared__ __align__(16) uint2 dyn[];
  uint2* buf = dyn;                             // [PER]
  uint32_t* hist = (uint32_t*)(dyn + PER);      // [SORT_WARPS][BINS]
  uint32_t* tot = hist + SORT_WARPS * BINS;     // [CTAS][BINS]
  uint32_t* wsum = tot + CTAS * BINS;           // [SORT_WARPS]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = CTAS > 1 ? (int)cluster_rank() : 0;
  uint32_t* h = hist + warp * BINS;
  let_next_start();
  if ((int)blockIdx.x >= CTAS) {
    zero_rows(a, (int)blockIdx.x - CTAS, (int)gridDim.x - CTAS, (uint4*)dyn);
    return;
  }
  uint32_t key[TILES], pos[TILES], off[TILES];
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    const int i = rank * PER + (warp * TILES + j) * 32 + lane;
    pos[j] = (uint32_t)i;
    key[j] = i < a.N ? sort_key(a, i) : 0xffffffffu;
  }
  sort_prepare<CTAS>(a, rank);
  if (CTAS > 1) cluster_barrier();  // every block has started: its shared memory may be written
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * BITS;
    const bool last = pass + 1 == a.passes;
#pragma unroll
    for (int b = 0; b < BINS / 32; ++b) h[b * 32 + lane] = 0;
    __syncwarp();
    unsigned peers[TILES];
#pragma unroll
    for (int j = 0; j < TILES; ++j) peers[j] = same_digit<BITS>(0xffffffffu, (key[j] >> shift) & MASK);
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const uint32_t d = (key[j] >> shift) & MASK;
      off[j] = h[d] + __popc(peers[j] & ((1u << lane) - 1));
      __syncwarp();
      if (lane == __ffs(peers[j]) - 1) h[d] = off[j] + __popc(peers[j]);
      __syncwarp();
    }
    __syncthreads();
    sort_places<CTAS, BITS>(hist, tot, wsum, rank);
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const uint32_t at = h[(key[j] >> shift) & MASK] + off[j];
      if (last) {
        if (at < (uint32_t)a.N) {
          a.k0[at] = key[j];
          a.p0[at] = pos[j];
        }
      } else if constexpr (CTAS > 1) {
        // every block has read its pairs of this pass (the barrier in sort_places)
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote_addr(buf + at % PER, at / PER)),
                     "r"(key[j]), "r"(pos[j])
                     : "memory");
      } else {
        buf[at] = make_uint2(key[j], pos[j]);
      }
    }
    if (last) break;      // nothing of another block's is touched after the last barrier
    sort_barrier<CTAS>();  // the pairs are in place, and every block has read the counts
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const uint2 v = buf[(warp * TILES + j) * 32 + lane];
      key[j] = v.x;
      pos[j] = v.y;
    }
  }
}

template <int BITS>
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS, 1)
    k_sort(const __grid_constant__ SortArgs a) {
  constexpr int BINS = 1 << BITS;
  constexpr uint32_t MASK = BINS - 1;
  extern __shared__ __align__(16) uint2 dyn[];
  uint32_t* hist = (uint32_t*)dyn;              // [SORT_WARPS][BINS]
  uint32_t* tot = hist + SORT_WARPS * BINS;     // [SORT_CTAS][BINS]
  uint32_t* wsum = tot + SORT_CTAS * BINS;      // [SORT_WARPS]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_rank();
  uint32_t* h = hist + warp * BINS;
  let_next_start();
  if ((int)blockIdx.x >= SORT_CTAS) {
    zero_rows(a, (int)blockIdx.x - SORT_CTAS, (int)gridDim.x - SORT_CTAS, (uint4*)dyn);
    return;
  }
  sort_prepare<SORT_CTAS>(a, rank);
  cluster_barrier();  // every block has started: its shared memory may be written
  // this warp's part of the list, in whole tiles of 32
  const int64_t tiles = ((int64_t)a.N + 31) / 32;
  const int64_t gw = (int64_t)rank * SORT_WARPS + warp, nw = SORT_CTAS * SORT_WARPS;
  const int64_t i0 = tiles * gw / nw * 32, i1 = min(tiles * (gw + 1) / nw * 32, (int64_t)a.N);
  for (int pass = 0; pass < a.passes; ++pass) {
    const bool to0 = ((a.passes - pass) & 1) != 0;  // the last pass ends in k0, p0
    const uint32_t* ks = to0 ? a.k1 : a.k0;
    const uint32_t* ps = to0 ? a.p1 : a.p0;
    uint32_t* kd = to0 ? a.k0 : a.k1;
    uint32_t* pd = to0 ? a.p0 : a.p1;
    const int shift = pass * BITS;
    for (int b = lane; b < BINS; b += 32) h[b] = 0;
    __syncwarp();
    for (int64_t i = i0 + lane; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const uint32_t key = pass == 0 ? sort_key(a, (int)i) : __ldcg(ks + i);
        const uint32_t d = (key >> shift) & MASK;
        const unsigned peers = same_digit<BITS>(act, d);
        if (lane == __ffs(peers) - 1) h[d] += __popc(peers);
      }
      __syncwarp();
    }
    __syncthreads();
    sort_places<SORT_CTAS, BITS>(hist, tot, wsum, rank);
    for (int64_t i = i0 + lane; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const uint32_t key = pass == 0 ? sort_key(a, (int)i) : __ldcg(ks + i);
        const uint32_t pos = pass == 0 ? (uint32_t)i : __ldcg(ps + i);
        const uint32_t d = (key >> shift) & MASK;
        const unsigned peers = same_digit<BITS>(act, d);
        const uint32_t at = h[d] + __popc(peers & ((1u << lane) - 1));
        kd[at] = key;
        pd[at] = pos;
        __syncwarp(act);
        if (lane == __ffs(peers) - 1) h[d] += __popc(peers);
      }
      __syncwarp();
    }
    cluster_barrier();  // the scattered list is complete; every block has read the counts
  }
}

// One cluster of `ctas` blocks of kern that sorts, and with something to zero a block for each
// other SM (in whole clusters); the shared-memory limit is raised once per kernel and device.
template <typename K>
cudaError_t launch_cluster(K kern, int ctas, size_t smem, const SortArgs& a, cudaStream_t s, std::atomic<bool>* raised) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!raised[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    raised[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  int64_t blocks = ctas + a.zrows * cdiv64(a.zlen, ZERO_CHUNK);
  if (blocks > 2 * num_sms()) blocks = 2 * num_sms();
  cfg.gridDim = dim3((unsigned)(cdiv64(blocks, ctas) * ctas), 1, 1);
  cfg.blockDim = dim3(SORT_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int CTAS, int TILES, int BITS>
cudaError_t launch_sort_reg(const SortArgs& a, cudaStream_t s) {
  static std::atomic<bool> raised[64];
  return launch_cluster(k_sort_reg<CTAS, TILES, BITS>, CTAS, sort_smem(CTAS, BITS, SORT_WARPS * TILES * 32), a, s, raised);
}

template <int BITS>
cudaError_t launch_sort_bits(const SortArgs& a, cudaStream_t s) {
  const int64_t tiles = cdiv64(a.N, 32), warps = SORT_CTAS * SORT_WARPS;
  if (tiles <= SORT_WARPS) return launch_sort_reg<1, 1, BITS>(a, s);
  if (tiles <= 2 * SORT_WARPS) return launch_sort_reg<1, 2, BITS>(a, s);
  if (tiles <= warps) return launch_sort_reg<SORT_CTAS, 1, BITS>(a, s);
  if (tiles <= 2 * warps) return launch_sort_reg<SORT_CTAS, 2, BITS>(a, s);
  if (tiles <= 4 * warps) return launch_sort_reg<SORT_CTAS, 4, BITS>(a, s);
  if (tiles <= 8 * warps) return launch_sort_reg<SORT_CTAS, 8, BITS>(a, s);
  if (tiles <= 16 * warps) return launch_sort_reg<SORT_CTAS, 16, BITS>(a, s);
  static std::atomic<bool> raised[64];
  return launch_cluster(k_sort<BITS>, SORT_CTAS, sort_smem(SORT_CTAS, BITS, 0), a, s, raised);
}

// kb: bits of the largest key
cudaError_t launch_sort(SortArgs a, int kb, cudaStream_t s) {
  a.passes = (kb + MAX_BITS - 1) / MAX_BITS;
  const int bits = (kb + a.passes - 1) / a.passes;
  return bits <= 8 ? launch_sort_bits<8>(a, s) : bits == 9 ? launch_sort_bits<9>(a, s) : launch_sort_bits<10>(a, s);
}

// ------------------------------------------------------------------ sums
constexpr int PIECE = 32;       // sorted positions per block
constexpr int BATCH = 8;        // rows in flight per thread

struct SumArgs {
  const uint32_t *keys, *pos;  // sorted
  int N;
  int64_t V, H;
  const void* dout;
  int64_t lddout;
  void* dE;
  int64_t lddE;
  float scale;
  int ovw;
  int pieces, slices;   // blocks: pieces x slices
  float* part;          // [pieces][2][H]: a piece's run that began before it, and its last run
                        // where that goes on past it
  int* count;           // [pieces][slices]: parts left of the run that begins in the piece
};

// A run whose rows lie in several pieces: each piece leaves a partial row, and the block that
// leaves the last one adds them up in piece order. x: this piece, whose first key is k when the
// run began before it (head). Returns whether this block is the last; x0: the piece where the
// run begins, np: the number of pieces. The piece borders are looked at 32 at a time (not by the
// read-only path: the sort may still write the keys when this kernel starts).
__device__ __forceinline__ bool last_of_run(const SumArgs& a, int x, bool head, uint32_t k, int slice, int& x0, int& np) {
  __shared__ int sh[3];
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = (int)threadIdx.x;
    int b0 = x;
    if (head) {
      for (b0 = x - 1;; b0 -= 32) {  // back over the pieces that it runs into from the one before
        const int p = b0 - lane;
        const bool in = p > 0 && __ldcg(a.keys + (int64_t)p * PIECE - 1) == k;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (m != 0xffffffffu) {
          b0 -= __ffs(~m) - 1;
          break;
        }
      }
    }
    int n = x - b0 + 1;
    for (;;) {  // and on over those that begin with it
      const int p = b0 + n + lane;
      const bool in = p < a.pieces && __ldcg(a.keys + (int64_t)p * PIECE) == k;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      if (m != 0xffffffffu) break;
    }
    if (lane == 0) {
      sh[0] = atomicAdd(a.count + (int64_t)b0 * a.slices + slice, 1) == n - 1;
      sh[1] = n;
      sh[2] = b0;
    }
  }
  __syncthreads();
  np = sh[1];
  x0 = sh[2];
  const bool last = sh[0] != 0;
  if (last) __threadfence();
  return last;
}

template <typename D, int EPV>
struct RowOf {  // EPV elements of dE in accesses of at most 32 bytes
  static constexpr int E = EPV == 1 ? 1 : (EPV * (int)sizeof(D) > 32 ? 32 / (int)sizeof(D) : EPV);
  static constexpr int N = EPV / E;
  Raw<D, E> r[N];
  __device__ __forceinline__ void load(const D* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].load(p + i * E);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].zero();
  }
  // p = s * scale (+ the loaded elements)
  __device__ __forceinline__ void add_store(D* p, const float (&s)[EPV], float scale) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = s[i * E + e] * scale + r[i].get(e);
      Vec<D, E>::store(p + i * E, o);
    }
  }
};

// Blocks 0 .. pieces * slices - 1: piece x = block / slices, columns (block % slices) * threads *
// EPV .... BATCH rows of dout are loaded together, and with them the rows of dE that their runs
// end at.
template <typename T, typename D, int EPV>
__global__ void __launch_bounds__(128) k_embed_sum(const __grid_constant__ SumArgs a) {
  after_previous();
  __shared__ uint32_t key[PIECE + 2], pos[PIECE];
  const int x = blockIdx.x / a.slices, slice = blockIdx.x - x * a.slices;
  const int i0 = x * PIECE;
  const int n = min(PIECE, a.N - i0);
  const uint32_t none = (uint32_t)a.V;
  for (int i = threadIdx.x; i < PIECE + 2; i += blockDim.x) {
    const int g = i0 + i - 1;
    key[i] = g >= 0 && g < a.N ? a.keys[g] : none;
    if (i >= 1 && i <= PIECE) pos[i - 1] = i <= n ? a.pos[g] : 0u;
  }
  __syncthreads();
  if (key[1] == none) return;  // nothing but ignored positions from here on
  const int64_t c = ((int64_t)slice * blockDim.x + threadIdx.x) * EPV;
  const bool in = c < a.H;
  const T* dout = (const T*)a.dout + c;
  float s[EPV];
#pragma unroll
  for (int e = 0; e < EPV; ++e) s[e] = 0.0f;
  const bool head = key[0] == key[1];   // the first run began in an earlier piece
  bool first = true, left_head = false, left_tail = false;
  for (int b = 0; b < n; b += BATCH) {
    Raw<T, EPV> r[BATCH];
    RowOf<D, EPV> old[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = b + j;
      const uint32_t k = key[min(i, PIECE - 1) + 1];
      r[j].zero();
      old[j].zero();
      if (in && i < n && k != none) {
        r[j].load(dout + (int64_t)pos[i] * a.lddout);
        if (!a.ovw && key[i + 2] != k) old[j].load((const D*)a.dE + (int64_t)k * a.lddE + c);
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = b + j;
      if (i < n && key[i + 1] != none) {
        const uint32_t k = key[i + 1];
#pragma unroll
        for (int e = 0; e < EPV; ++e) s[e] += r[j].get(e);
        if (i + 1 == n || key[i + 2] != k) {  // the run's end in this piece
          const bool began = first && head, goes_on = i + 1 == n && key[i + 2] == k;
          if (began || goes_on) {
            float* p = a.part + ((int64_t)x * 2 + (began ? 0 : 1)) * a.H + c;
            if (in) {
#pragma unroll
              for (int e = 0; e < EPV; ++e) __stcg(p + e, s[e]);
            }
            left_head |= began;
            left_tail |= !began;
          } else if (in) {
            old[j].add_store((D*)a.dE + (int64_t)k * a.lddE + c, s, a.scale);
          }
          first = false;
#pragma unroll
          for (int e = 0; e < EPV; ++e) s[e] = 0.0f;
        }
      }
    }
  }
  // the partial rows left: of the run that began before the piece, and of the one that goes on
  for (int tail = 0; tail < 2; ++tail) {
    if (!(tail ? left_tail : left_head)) continue;
    const uint32_t k = tail ? key[n] : key[1];
    int x0, np;
    if (!last_of_run(a, x, tail == 0, k, slice, x0, np) || !in) continue;
    const float* q = a.part + ((int64_t)x0 * 2 + 1) * a.H + c;
    float t[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) t[e] = __ldcg(q + e);
    q += a.H;  // slot 0 of the next piece
#pragma unroll 4
    for (int m = 1; m < np; ++m, q += 2 * a.H) {
#pragma unroll
      for (int e = 0; e < EPV; ++e) t[e] += __ldcg(q + e);
    }
    D* d = (D*)a.dE + (int64_t)k * a.lddE + c;
    RowOf<D, EPV> o;
    o.zero();
    if (!a.ovw) o.load(d);
    o.add_store(d, t, a.scale);
  }
}

struct Layout {
  size_t k0, p0, k1, p1, count, part, total;
};
// Column slices of the sums: the narrowest (single elements) decide the counters' size.
int64_t max_slices(int64_t H) { return cdiv64(H, 32); }
Layout layout(int64_t N, int64_t H) {
  Layout l;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = round_up(off + bytes, 256);
    return o;
  };
  const int64_t pieces = cdiv64(N, PIECE);
  l.k0 = take(4 * (size_t)N);
  l.p0 = take(4 * (size_t)N);
  l.k1 = take(4 * (size_t)N);
  l.p1 = take(4 * (size_t)N);
  l.count = take(4 * (size_t)pieces * max_slices(H));
  l.part = take((size_t)pieces * 2 * (size_t)H * 4);
  l.total = off ? off : 256;
  return l;
}

// Threads and column slices of a row in vectors of EPV elements.
void sum_shape(int64_t H, int epv, int& threads, int& slices) {
  const int64_t nvec = cdiv64(H, epv);
  slices = (int)cdiv64(nvec, 128);
  threads = (int)(cdiv64(cdiv64(nvec, slices), 32) * 32);
}

template <typename T, typename D>
cudaError_t sums(SumArgs a, int epv, int threads, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const unsigned blocks = (unsigned)(a.pieces * a.slices);
  if (epv == W) return launch_after(k_embed_sum<T, D, W>, blocks, threads, 0, s, a);
  if (epv == 2) return launch_after(k_embed_sum<T, D, 2>, blocks, threads, 0, s, a);
  return launch_after(k_embed_sum<T, D, 1>, blocks, threads, 0, s, a);
}

bool sizes_ok(int64_t N, int64_t H, int64_t V) {
  return N >= 0 && H >= 1 && V >= 1 && N <= 0x7fffff00LL && H <= 65535LL * 512 && V <= 0x7fffffffLL;
}

int32_t check(const flce_embed_args* x) {
  if (x == nullptr || !sizes_ok(x->N, x->H, x->V) || !valid_dtype(x->dtype)) return FLCE_ERR_INVALID_ARG;
  if (!isfinite(x->scale)) return FLCE_ERR_INVALID_ARG;
  if (x->N > 0 && (!x->tokens || !aligned_to(x->tokens, 8))) return FLCE_ERR_INVALID_ARG;
  if (x->status && !aligned_to(x->status, 4)) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int32_t flce_embed_fwd(const flce_embed_args* x, void* stream) {
  const int32_t c = check(x);
  if (c != FLCE_OK) return c;
  if (x->flags != 0) return FLCE_ERR_INVALID_ARG;
  const int esz = dtype_size(x->dtype);
  if (x->N > 0 && (!x->E || !x->out || !aligned_to(x->E, esz) || !aligned_to(x->out, esz) || x->ldE < x->H ||
                   x->ldout < x->H))
    return FLCE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (x->status) {
    const cudaError_t e = cudaMemsetAsync(x->status, 0, sizeof(int), s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (x->N == 0) return FLCE_OK;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(fwd<float>(*x, s));
    case FLCE_BF16: return cuda_status(fwd<__nv_bfloat16>(*x, s));
    default: return cuda_status(fwd<__half>(*x, s));
  }
}

extern "C" size_t flce_embed_workspace_size(int64_t N, int64_t H, int64_t V) {
  return sizes_ok(N, H, V) ? layout(N, H).total : 0;
}

extern "C" int32_t flce_embed_bwd(const flce_embed_args* x, void* stream) {
  const int32_t c = check(x);
  if (c != FLCE_OK) return c;
  if ((x->flags & ~FLCE_FLAG_DW_OVERWRITE) != 0) return FLCE_ERR_INVALID_ARG;
  if (x->dE_dtype != FLCE_F32 && x->dE_dtype != x->dtype) return FLCE_ERR_UNSUPPORTED;
  const int esz = dtype_size(x->dtype), dsz = dtype_size(x->dE_dtype);
  if (!x->dE || !aligned_to(x->dE, dsz) || x->lddE < x->H) return FLCE_ERR_INVALID_ARG;
  if (x->N > 0) {
    if (!x->dout || !aligned_to(x->dout, esz) || x->lddout < x->H) return FLCE_ERR_INVALID_ARG;
    if (!x->workspace || !aligned_to(x->workspace, 256)) return FLCE_ERR_INVALID_ARG;
    if (x->workspace_bytes < layout(x->N, x->H).total) return FLCE_ERR_WORKSPACE;
  }
  const bool ovw = (x->flags & FLCE_FLAG_DW_OVERWRITE) != 0;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (x->status) e = cudaMemsetAsync(x->status, 0, sizeof(int), s);
  if (e == cudaSuccess && x->N == 0 && ovw)
    e = cudaMemset2DAsync(x->dE, (size_t)x->lddE * dsz, 0, (size_t)x->H * dsz, (size_t)x->V, s);
  if (e != cudaSuccess || x->N == 0) return cuda_status(e);

  const Layout l = layout(x->N, x->H);
  char* ws = (char*)x->workspace;
  SumArgs a = {};
  a.N = (int)x->N;
  a.V = x->V;
  a.H = x->H;
  a.dout = x->dout;
  a.lddout = x->lddout;
  a.dE = x->dE;
  a.lddE = x->lddE;
  a.scale = x->scale;
  a.ovw = ovw;
  a.pieces = (int)cdiv64(x->N, PIECE);
  a.part = (float*)(ws + l.part);
  a.count = (int*)(ws + l.count);
  const int wide = 16 / esz;
  auto fits = [&](int v) {
    return x->H % v == 0 && rows_by(x->dout, x->lddout, esz, (size_t)(v * esz)) &&
           rows_by(x->dE, x->lddE, dsz, (size_t)(v * dsz > 32 ? 32 : v * dsz));
  };
  const int epv = fits(wide) ? wide : fits(2) ? 2 : 1;
  int threads;
  sum_shape(x->H, epv, threads, a.slices);

  SortArgs so = {};
  so.tokens = x->tokens;
  so.ignore_index = x->ignore_index;
  so.V = x->V;
  so.N = (int)x->N;
  int kb = 1;
  while ((x->V >> kb) != 0) ++kb;  // bits of the largest key, V
  so.k0 = (uint32_t*)(ws + l.k0);
  so.p0 = (uint32_t*)(ws + l.p0);
  so.k1 = (uint32_t*)(ws + l.k1);
  so.p1 = (uint32_t*)(ws + l.p1);
  so.status = x->status;
  so.count = a.count;
  so.ncount = a.pieces * a.slices;
  if (ovw) {
    const bool dense = x->lddE == x->H;
    so.zero = (uint8_t*)x->dE;
    so.zrows = dense ? 1 : x->V;
    so.zlen = (dense ? x->V : 1) * x->H * dsz;
    so.zpitch = x->lddE * dsz;
  }
  a.keys = so.k0;
  a.pos = so.p0;
  e = launch_sort(so, kb, s);
  if (e != cudaSuccess) return cuda_status(e);

  const bool same = x->dE_dtype == x->dtype;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(sums<float, float>(a, epv, threads, s));
    case FLCE_BF16:
      return cuda_status(same ? sums<__nv_bfloat16, __nv_bfloat16>(a, epv, threads, s)
                              : sums<__nv_bfloat16, float>(a, epv, threads, s));
    default:
      return cuda_status(same ? sums<__half, __half>(a, epv, threads, s) : sums<__half, float>(a, epv, threads, s));
  }
}
