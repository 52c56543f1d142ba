// Token embedding: lookup with scaling, and its gradient from sorted tokens.
//
//   out_i = scale * E[t_i]                    dE_v += scale * sum_{i: t_i = v} dout_i
//
// Forward: a copy of N rows, bound by HBM writes (rows of frequent tokens come from L2).
// Backward: the token positions are sorted by token (stable), so each row of dE is the sum
// of one run of the sorted list. Blocks take fixed pieces of the list; a run inside a piece
// is added to dE at once, a run that crosses pieces leaves one partial row per piece, and the
// block that leaves the last one adds them in piece order. No atomics on data: the same bits
// on every run. Bound by HBM: dout once, the touched rows of dE read and written once.
#include <math.h>

#include "flce_ops.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------------ forward
// Block (x, y): row x, vectors y * U * threads ... of it; each thread moves U vectors.
constexpr int FWD_U = 2;
template <typename T, int EPV>
__global__ void __launch_bounds__(256) k_embed_fwd(const int64_t* __restrict__ tokens, int64_t V, int64_t H,
                                                   int64_t ignore_index, float scale, const T* __restrict__ E,
                                                   int64_t ldE, T* __restrict__ out, int64_t ldout, int* status) {
  const int64_t row = blockIdx.x;
  const int64_t t = tokens[row];
  const bool live = t >= 0 && t < V && t != ignore_index;
  if (!live && t != ignore_index && status != nullptr && threadIdx.x == 0 && blockIdx.y == 0)
    atomicOr(status, ST_TARGET_RANGE);
  const int64_t v0 = (int64_t)blockIdx.y * FWD_U * blockDim.x + threadIdx.x;
  Raw<T, EPV> r[FWD_U];
#pragma unroll
  for (int u = 0; u < FWD_U; ++u) {
    const int64_t c = (v0 + u * blockDim.x) * EPV;
    r[u].zero();
    if (live && c < H) r[u].load(E + t * ldE + c);
  }
#pragma unroll
  for (int u = 0; u < FWD_U; ++u) {
    const int64_t c = (v0 + u * blockDim.x) * EPV;
    if (c >= H) continue;
    if (live && scale != 1.0f) {
      float v[EPV];
      r[u].unpack(v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) v[e] *= scale;
      r[u].pack(v);
    }
    r[u].store(out + row * ldout + c);
  }
}

template <typename T, int EPV>
void launch_fwd(const flce_embed_args& a, cudaStream_t s) {
  // as many blocks a row as 256 threads of FWD_U vectors need, of as few threads as that takes
  const int64_t nvec = cdiv64(a.H, EPV);
  const int64_t by = cdiv64(nvec, 256 * FWD_U);
  const int threads = (int)(cdiv64(cdiv64(nvec, by * FWD_U), 32) * 32);
  k_embed_fwd<T, EPV><<<dim3((unsigned)a.N, (unsigned)by), threads, 0, s>>>(
      a.tokens, a.V, a.H, a.ignore_index, a.scale, (const T*)a.E, a.ldE, (T*)a.out, a.ldout, a.status);
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
  else launch_fwd<T, 1>(a, s);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ sort
// Stable radix sort of (token, position) by one cluster of CTAS blocks (one block for short
// lists: no cluster barriers, no distributed shared memory). Keys are the tokens, V for ignored
// and out-of-range ones (they sort last and are left out). Each block owns a contiguous share
// of the list, each of its warps a contiguous part of that; a pass counts the digits per warp,
// adds the counts up over the warps, the blocks (through distributed shared memory) and the
// digits, and scatters each pair to its place. Sixteen warps a block: more would lengthen the
// sums over the warps, which is what a pass over a short list consists of.
constexpr int SORT_CTAS = 8;
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ONE = 1024;  // longest list for a single block: two tiles of 32 per warp
constexpr int MAX_BINS = 512;
static_assert(MAX_BINS <= SORT_THREADS, "a thread per digit");

struct SortArgs {
  const int64_t* tokens;
  int64_t ignore_index;
  int64_t V;
  int N;
  int passes, bits;    // passes of `bits` bits each
  uint32_t *k0, *p0;   // ping
  uint32_t *k1, *p1;   // pong
  int* status;
  int* count;          // [pieces][slices] zeroed for k_embed_sum
  int ncount;
  uint32_t* used;      // bit v: token v occurs; null when not wanted
  int nused;           // its words
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t ld_remote(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <int CTAS>
__device__ __forceinline__ void sort_barrier() {
  if constexpr (CTAS > 1) cluster_barrier();
  else __syncthreads();
}

template <int CTAS>
__global__ void __launch_bounds__(SORT_THREADS, 1) k_sort(const __grid_constant__ SortArgs a) {
  __shared__ uint32_t hist[SORT_WARPS][MAX_BINS];
  __shared__ uint32_t tot[MAX_BINS];   // this block's digit counts
  __shared__ uint32_t wsum[MAX_BINS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CTAS > 1 ? (int)cluster_rank() : 0;
  const int bins = 1 << a.bits;
  const uint32_t mask = (uint32_t)bins - 1;
  for (int i = rank * SORT_THREADS + tid; i < a.ncount; i += CTAS * SORT_THREADS) a.count[i] = 0;
  if (a.used != nullptr) {
    for (int i = rank * SORT_THREADS + tid; i < a.nused; i += CTAS * SORT_THREADS) a.used[i] = 0u;
    sort_barrier<CTAS>();
  }
  // this warp's part of the list, in whole tiles of 32
  const int64_t tiles = (a.N + 31) / 32;
  const int64_t gw = (int64_t)rank * SORT_WARPS + warp, nw = CTAS * SORT_WARPS;
  const int i0 = (int)(tiles * gw / nw) * 32, i1 = min((int)(tiles * (gw + 1) / nw) * 32, a.N);
  uint32_t* h = hist[warp];
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint32_t* ks = pass & 1 ? a.k1 : a.k0;
    const uint32_t* ps = pass & 1 ? a.p1 : a.p0;
    uint32_t* kd = pass & 1 ? a.k0 : a.k1;
    uint32_t* pd = pass & 1 ? a.p0 : a.p1;
    const int shift = pass * a.bits;
    auto load = [&](int i, uint32_t& key, uint32_t& pos) {
      if (pass == 0) {
        const int64_t t = a.tokens[i];
        const bool live = t >= 0 && t < a.V && t != a.ignore_index;
        if (!live && t != a.ignore_index && a.status != nullptr) atomicOr(a.status, ST_TARGET_RANGE);
        key = live ? (uint32_t)t : (uint32_t)a.V;
        pos = (uint32_t)i;
      } else {
        key = __ldcg(ks + i);
        pos = __ldcg(ps + i);
      }
    };
    for (int b = lane; b < bins; b += 32) h[b] = 0;
    __syncwarp();
    for (int i = i0 + lane; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        uint32_t key, pos;
        load(i, key, pos);
        const uint32_t d = (key >> shift) & mask;
        const unsigned peers = __match_any_sync(act, d);
        if (lane == __ffs(peers) - 1) h[d] += __popc(peers);
        if (pass == 0 && a.used != nullptr && key < (uint32_t)a.V) atomicOr(a.used + (key >> 5), 1u << (key & 31));
      }
      __syncwarp();
    }
    __syncthreads();
    // counts over the block's warps: each digit's column becomes an exclusive sum
    uint32_t before = 0, all = 0;
    if (tid < bins) {
      uint32_t c[SORT_WARPS], s = 0;
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) c[w] = hist[w][tid];
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) {
        hist[w][tid] = s;
        s += c[w];
      }
      all = s;
      if (CTAS > 1) tot[tid] = s;
    }
    if constexpr (CTAS > 1) {
      cluster_barrier();
      if (tid < bins) {
        all = 0;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) {
          const uint32_t v = ld_remote(tot + tid, c);
          before += c < rank ? v : 0;
          all += v;
        }
      }
    }
    // exclusive sum of `all` over the digits (zero past bins)
    uint32_t x = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (tid < MAX_BINS && lane == 31) wsum[warp] = x;
    __syncthreads();
    uint32_t base = x - all + before;
    if (tid < MAX_BINS)
      for (int w = 0; w < warp; ++w) base += wsum[w];
    if (tid < bins) {
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) hist[w][tid] += base;
    }
    __syncthreads();
    for (int i = i0 + lane; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        uint32_t key, pos;
        load(i, key, pos);
        const uint32_t d = (key >> shift) & mask;
        const unsigned peers = __match_any_sync(act, d);
        const uint32_t at = h[d] + __popc(peers & ((1u << lane) - 1));
        kd[at] = key;
        pd[at] = pos;
        __syncwarp(act);
        if (lane == __ffs(peers) - 1) h[d] += __popc(peers);
      }
      __syncwarp();
    }
    sort_barrier<CTAS>();  // the scattered list is complete; every block has read the counts
  }
}

// ------------------------------------------------------------------ sums
constexpr int PIECE = 32;       // sorted positions per block
constexpr int BATCH = 4;        // rows in flight per thread
constexpr int ZERO_ROWS = 64;   // rows of dE per block that zeroes unused ones

__device__ __forceinline__ int64_t cdiv_dev(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
  int pieces, slices;   // blocks: pieces x slices that sum, then those that zero
  float* part;          // [pieces][2][H]: a piece's run that began before it, and its last run
                        // where that goes on past it
  int* count;           // [pieces][slices]: parts left of the run that begins in the piece
  const uint32_t* used;
};

// A run whose rows lie in several pieces: each piece leaves a partial row, and the block that
// leaves the last one adds them up in piece order. x0: the piece where the run begins, k: its
// key. Returns whether this block is the last; np: the number of pieces.
__device__ __forceinline__ bool last_of_run(const SumArgs& a, int x0, uint32_t k, int slice, int& np) {
  __shared__ int sh[2];
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 32) {
    // pieces x0 + 1 ... that begin with the key
    int n = 1;
    for (;;) {
      const int p = x0 + n + (int)threadIdx.x;
      const bool in = p < a.pieces && __ldg(a.keys + (int64_t)p * PIECE) == k;
      const unsigned b = __ballot_sync(0xffffffffu, in);
      n += b == 0xffffffffu ? 32 : __ffs(~b) - 1;
      if (b != 0xffffffffu) break;
    }
    if (threadIdx.x == 0) {
      sh[0] = atomicAdd(a.count + (int64_t)x0 * a.slices + slice, 1) == n - 1;
      sh[1] = n;
    }
  }
  __syncthreads();
  np = sh[1];
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
// end at. The blocks after those zero the rows of dE that no token points to
// (FLCE_FLAG_DW_OVERWRITE).
template <typename T, typename D, int EPV>
__global__ void __launch_bounds__(128) k_embed_sum(const __grid_constant__ SumArgs a) {
  const int sums = a.pieces * a.slices;
  if ((int)blockIdx.x >= sums) {
    const int64_t v0 = (int64_t)(blockIdx.x - sums) * ZERO_ROWS;
    float z[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) z[e] = 0.0f;
    RowOf<D, EPV> row;
    row.zero();
    const int64_t nvec = cdiv_dev(a.H, EPV);
    for (int r = 0; r < ZERO_ROWS && v0 + r < a.V; ++r) {
      const int64_t v = v0 + r;
      if (a.used[v >> 5] >> (v & 31) & 1u) continue;
      for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x)
        row.add_store((D*)a.dE + v * a.lddE + i * EPV, z, 0.0f);
    }
    return;
  }
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
  bool first = true;
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
            int x0 = x;
            if (began) {  // where did it begin? the first piece whose last key is k
              int lo = 0, hi = x - 1;
              while (lo < hi) {
                const int m = (lo + hi) / 2;
                if (__ldg(a.keys + (int64_t)(m + 1) * PIECE - 1) < k) lo = m + 1;
                else hi = m;
              }
              x0 = lo;
            }
            int np;
            if (last_of_run(a, x0, k, slice, np) && in) {
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
}

struct Layout {
  size_t k0, p0, k1, p1, count, used, part, total;
  int ncount, nused;
};
// Column slices of the sums: the narrowest (single elements) decide the counters' size.
int64_t max_slices(int64_t H) { return cdiv64(H, 32); }
Layout layout(int64_t N, int64_t H, int64_t V) {
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
  l.nused = (int)cdiv64(V, 32);
  l.used = take(N > 0 ? 4 * (size_t)l.nused : 0);
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
  const unsigned blocks = (unsigned)(a.pieces * a.slices + (a.ovw ? cdiv64(a.V, ZERO_ROWS) : 0));
  if (epv == W) k_embed_sum<T, D, W><<<blocks, threads, 0, s>>>(a);
  else k_embed_sum<T, D, 1><<<blocks, threads, 0, s>>>(a);
  return cudaGetLastError();
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
  return sizes_ok(N, H, V) ? layout(N, H, V).total : 0;
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
    if (x->workspace_bytes < layout(x->N, x->H, x->V).total) return FLCE_ERR_WORKSPACE;
  }
  const bool ovw = (x->flags & FLCE_FLAG_DW_OVERWRITE) != 0;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (x->status) e = cudaMemsetAsync(x->status, 0, sizeof(int), s);
  if (e == cudaSuccess && x->N == 0 && ovw)
    e = cudaMemset2DAsync(x->dE, (size_t)x->lddE * dsz, 0, (size_t)x->H * dsz, (size_t)x->V, s);
  if (e != cudaSuccess || x->N == 0) return cuda_status(e);

  const Layout l = layout(x->N, x->H, x->V);
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
  a.used = (const uint32_t*)(ws + l.used);
  const int wide = 16 / esz;
  const bool fits = x->H % wide == 0 && rows16(x->dout, x->lddout, esz) &&
                    rows_by(x->dE, x->lddE, dsz, (size_t)(wide * dsz > 32 ? 32 : wide * dsz));
  const int epv = fits ? wide : 1;
  int threads;
  sum_shape(x->H, epv, threads, a.slices);

  SortArgs so = {};
  so.tokens = x->tokens;
  so.ignore_index = x->ignore_index;
  so.V = x->V;
  so.N = (int)x->N;
  int kb = 1;
  while ((x->V >> kb) != 0) ++kb;  // bits of the largest key, V
  so.passes = (kb + 8) / 9;
  so.bits = (kb + so.passes - 1) / so.passes;
  so.k0 = (uint32_t*)(ws + l.k0);
  so.p0 = (uint32_t*)(ws + l.p0);
  so.k1 = (uint32_t*)(ws + l.k1);
  so.p1 = (uint32_t*)(ws + l.p1);
  so.status = x->status;
  so.count = a.count;
  so.ncount = a.pieces * a.slices;
  so.used = ovw ? (uint32_t*)(ws + l.used) : nullptr;
  so.nused = l.nused;
  a.keys = so.passes & 1 ? so.k1 : so.k0;
  a.pos = so.passes & 1 ? so.p1 : so.p0;
  if (x->N <= SORT_ONE) {
    k_sort<1><<<1, SORT_THREADS, 0, s>>>(so);
    e = cudaGetLastError();
  } else {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SORT_CTAS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(SORT_CTAS, 1, 1);
    cfg.blockDim = dim3(SORT_THREADS, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_sort<SORT_CTAS>, so);
  }
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
