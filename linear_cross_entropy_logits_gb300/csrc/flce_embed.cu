// Token embedding: lookup with scaling, and its gradient from sorted tokens.
//
//   out_i = scale * E[t_i]                    dE_v += scale * sum_{i: t_i = v} dout_i
//
// Forward: a copy of N rows, bound by HBM writes (rows of frequent tokens come from L2).
// Backward: the token positions are sorted by token (stable), so each row of dE is the sum
// of one run of the sorted list. Blocks take fixed pieces of the list; a run inside a piece
// is added to dE at once, a run that crosses pieces leaves one partial row per piece, which
// a second kernel adds in piece order. No atomics on data: the same bits on every run.
#include <math.h>

#include "flce_ops.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------------ forward
// Block (x, y): row x, vectors y * 4 * threads ... of it; each thread moves four vectors.
template <typename T, int EPV>
__global__ void __launch_bounds__(256) k_embed_fwd(const int64_t* __restrict__ tokens, int64_t V, int64_t H,
                                                   int64_t ignore_index, float scale, const T* __restrict__ E,
                                                   int64_t ldE, T* __restrict__ out, int64_t ldout, int* status) {
  constexpr int U = 4;
  const int64_t row = blockIdx.x;
  const int64_t t = tokens[row];
  const bool live = t >= 0 && t < V && t != ignore_index;
  if (!live && t != ignore_index && status != nullptr && threadIdx.x == 0 && blockIdx.y == 0)
    atomicOr(status, ST_TARGET_RANGE);
  const int64_t v0 = (int64_t)blockIdx.y * U * blockDim.x + threadIdx.x;
  float r[U][EPV];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = (v0 + u * blockDim.x) * EPV;
#pragma unroll
    for (int e = 0; e < EPV; ++e) r[u][e] = 0.0f;
    if (live && c < H) Vec<T, EPV>::load(E + t * ldE + c, r[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = (v0 + u * blockDim.x) * EPV;
    if (c < H) {
      if (live) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) r[u][e] *= scale;
      }
      Vec<T, EPV>::store(out + row * ldout + c, r[u]);
    }
  }
}

template <typename T, int EPV>
void launch_fwd(const flce_embed_args& a, cudaStream_t s) {
  const int64_t nvec = cdiv64(a.H, EPV);
  int threads = 32;
  while (threads < 256 && threads * 4 < nvec) threads *= 2;
  const dim3 grid((unsigned)a.N, (unsigned)cdiv64(nvec, 4 * threads));
  k_embed_fwd<T, EPV><<<grid, threads, 0, s>>>(a.tokens, a.V, a.H, a.ignore_index, a.scale, (const T*)a.E, a.ldE,
                                              (T*)a.out, a.ldout, a.status);
}

template <typename T>
cudaError_t fwd(const flce_embed_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  if (a.H % W == 0 && rows16(a.E, a.ldE, sizeof(T)) && rows16(a.out, a.ldout, sizeof(T))) launch_fwd<T, W>(a, s);
  else launch_fwd<T, 1>(a, s);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ sort
// Stable radix sort of (token, position) by one cluster of 8 blocks. Keys are the tokens,
// V for ignored and out-of-range ones (they sort last and are left out). Each block owns a
// contiguous share of the list, each of its warps a contiguous part of that; a pass counts
// the digits per warp, adds the counts up over the warps, the blocks (through distributed
// shared memory) and the digits, and scatters each pair to its place.
constexpr int SORT_CTAS = 8;
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_BINS = 512;

struct SortArgs {
  const int64_t* tokens;
  int64_t ignore_index;
  int64_t V;
  int N;
  int passes, bits;    // passes of `bits` bits each
  uint32_t *k0, *p0;   // ping
  uint32_t *k1, *p1;   // pong
  int* status;
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

__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS, 1)
    k_sort(const __grid_constant__ SortArgs a) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                               // [SORT_WARPS][MAX_BINS]
  uint32_t* tot = sm + SORT_WARPS * MAX_BINS;        // [MAX_BINS] this block's digit counts
  uint32_t* wsum = tot + MAX_BINS;                   // [MAX_BINS / 32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int bins = 1 << a.bits;
  const uint32_t mask = (uint32_t)bins - 1;
  // this warp's part of the list, in whole tiles of 32
  const int64_t tiles = (a.N + 31) / 32;
  const int64_t gw = (int64_t)rank * SORT_WARPS + warp, nw = SORT_CTAS * SORT_WARPS;
  const int i0 = (int)(tiles * gw / nw) * 32, i1 = min((int)(tiles * (gw + 1) / nw) * 32, a.N);
  uint32_t* h = hist + warp * MAX_BINS;
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
      }
      __syncwarp();
    }
    __syncthreads();
    // counts over the block's warps: each digit's column becomes an exclusive sum
    if (tid < bins) {
      uint32_t s = 0;
      for (int w = 0; w < SORT_WARPS; ++w) {
        const uint32_t c = hist[w * MAX_BINS + tid];
        hist[w * MAX_BINS + tid] = s;
        s += c;
      }
      tot[tid] = s;
    }
    cluster_barrier();
    uint32_t before = 0, all = 0;
    if (tid < bins) {
#pragma unroll
      for (int c = 0; c < SORT_CTAS; ++c) {
        const uint32_t v = ld_remote(tot + tid, c);
        before += c < rank ? v : 0;
        all += v;
      }
    }
    // exclusive sum of `all` over the digits (tid < MAX_BINS; zero past bins)
    uint32_t x = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (tid < MAX_BINS && lane == 31) wsum[warp] = x;
    __syncthreads();
    uint32_t base = x - all;
    if (tid < MAX_BINS)
      for (int w = 0; w < warp; ++w) base += wsum[w];
    base += before;
    if (tid < bins)
      for (int w = 0; w < SORT_WARPS; ++w) hist[w * MAX_BINS + tid] += base;
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
    cluster_barrier();  // the scattered list is complete; every block has read the counts
  }
}

// ------------------------------------------------------------------ sums
constexpr int PIECE = 32;  // sorted positions per block

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
  float* part;  // [pieces][2][H]: a piece's run that began before it, and its last run where
                // that goes on past it
};

template <typename D, int EPV>
__device__ __forceinline__ void add_row(D* p, const float (&s)[EPV], float scale, int ovw) {
  float o[EPV];
#pragma unroll
  for (int e = 0; e < EPV; ++e) o[e] = s[e] * scale;
  if (!ovw) {
#pragma unroll
    for (int e = 0; e < EPV; ++e) o[e] += to_f<D>(p[e]);
  }
#pragma unroll
  for (int e = 0; e < EPV; ++e) p[e] = from_f<D>(o[e]);
}

// Block (x, y): piece x, columns y * threads * EPV ....
template <typename T, typename D, int EPV>
__global__ void __launch_bounds__(256) k_embed_sum(const __grid_constant__ SumArgs a) {
  __shared__ uint32_t key[PIECE + 2], pos[PIECE];
  const int i0 = blockIdx.x * PIECE;
  const int n = min(PIECE, a.N - i0);
  const uint32_t none = (uint32_t)a.V;
  for (int i = threadIdx.x; i < PIECE + 2; i += blockDim.x) {
    const int g = i0 + i - 1;
    key[i] = g >= 0 && g < a.N ? a.keys[g] : none;
    if (i >= 1 && i <= n) pos[i - 1] = a.pos[g];
  }
  __syncthreads();
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * EPV;
  if (c >= a.H) return;
  const T* dout = (const T*)a.dout + c;
  float s[EPV];
#pragma unroll
  for (int e = 0; e < EPV; ++e) s[e] = 0.0f;
  bool first = true;  // still in the piece's first run
  for (int i = 0; i < n; ++i) {
    const uint32_t k = key[i + 1];
    if (k == none) break;
    float r[EPV];
    Vec<T, EPV>::load(dout + (int64_t)pos[i] * a.lddout, r);
#pragma unroll
    for (int e = 0; e < EPV; ++e) s[e] += r[e];
    if (i + 1 < n && key[i + 2] == k) continue;
    const bool began = first && key[0] == k;              // the run began in an earlier piece
    const bool goes_on = i + 1 == n && key[i + 2] == k;   // it goes on in the next one
    if (began || goes_on) {
      float* p = a.part + ((int64_t)blockIdx.x * 2 + (began ? 0 : 1)) * a.H + c;
#pragma unroll
      for (int e = 0; e < EPV; ++e) p[e] = s[e];
    } else {
      add_row<D, EPV>((D*)a.dE + (int64_t)k * a.lddE + c, s, a.scale, a.ovw);
    }
    first = false;
#pragma unroll
    for (int e = 0; e < EPV; ++e) s[e] = 0.0f;
  }
}

// Block (x, y): the run that begins in piece x and goes on past it, if there is one: its
// partial rows in piece order.
template <typename D>
__global__ void __launch_bounds__(128) k_embed_join(const __grid_constant__ SumArgs a) {
  const int x = blockIdx.x;
  const int end = (x + 1) * PIECE;  // first position of the next piece
  const uint32_t k = a.keys[end - 1];
  if (k == (uint32_t)a.V || a.keys[end] != k) return;
  if (x > 0 && a.keys[x * PIECE] == k && a.keys[x * PIECE - 1] == k) return;  // began earlier
  const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= a.H) return;
  float s[1] = {a.part[((int64_t)x * 2 + 1) * a.H + c]};
  for (int p = x + 1; p * PIECE < a.N && a.keys[p * PIECE] == k; ++p) s[0] += a.part[(int64_t)p * 2 * a.H + c];
  add_row<D, 1>((D*)a.dE + (int64_t)k * a.lddE + c, s, a.scale, a.ovw);
}

// FLCE_FLAG_DW_OVERWRITE: zero the rows of dE that no token points to. Block x: rows
// x * 64 ...; each is looked up in the sorted keys.
template <typename D>
__global__ void __launch_bounds__(256) k_embed_zero(const __grid_constant__ SumArgs a) {
  __shared__ uint8_t used[64];
  const int64_t v0 = (int64_t)blockIdx.x * 64;
  if (threadIdx.x < 64) {
    const uint32_t v = (uint32_t)(v0 + threadIdx.x);
    int lo = 0, hi = a.N;
    while (lo < hi) {
      const int m = (lo + hi) / 2;
      if (a.keys[m] < v) lo = m + 1;
      else hi = m;
    }
    used[threadIdx.x] = lo < a.N && a.keys[lo] == v;
  }
  __syncthreads();
  for (int r = 0; r < 64 && v0 + r < a.V; ++r) {
    if (used[r]) continue;
    D* p = (D*)a.dE + (v0 + r) * a.lddE;
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) p[c] = from_f<D>(0.0f);
  }
}

struct Layout {
  size_t k0, p0, k1, p1, part, total;
};
Layout layout(int64_t N, int64_t H) {
  Layout l;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = round_up(off + bytes, 256);
    return o;
  };
  l.k0 = take(4 * (size_t)N);
  l.p0 = take(4 * (size_t)N);
  l.k1 = take(4 * (size_t)N);
  l.p1 = take(4 * (size_t)N);
  l.part = take((size_t)cdiv64(N, PIECE) * 2 * (size_t)H * 4);
  l.total = off ? off : 256;
  return l;
}

template <typename T, typename D, int EPV>
void launch_sum(const SumArgs& a, cudaStream_t s) {
  const int64_t nvec = cdiv64(a.H, EPV);
  int threads = 32;
  while (threads < 128 && threads < nvec) threads *= 2;
  const dim3 grid((unsigned)cdiv64(a.N, PIECE), (unsigned)cdiv64(nvec, threads));
  k_embed_sum<T, D, EPV><<<grid, threads, 0, s>>>(a);
}

template <typename T, typename D>
cudaError_t sums(const SumArgs& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  if (a.H % W == 0 && rows16(a.dout, a.lddout, sizeof(T)) && rows16(a.dE, a.lddE, sizeof(D)))
    launch_sum<T, D, W>(a, s);
  else
    launch_sum<T, D, 1>(a, s);
  const int64_t pieces = cdiv64(a.N, PIECE);
  if (pieces > 1)
    k_embed_join<D><<<dim3((unsigned)(pieces - 1), (unsigned)cdiv64(a.H, 128)), 128, 0, s>>>(a);
  if (a.ovw) k_embed_zero<D><<<(unsigned)cdiv64(a.V, 64), 256, 0, s>>>(a);
  return cudaGetLastError();
}

bool sizes_ok(int64_t N, int64_t H, int64_t V) {
  return N >= 0 && H >= 1 && V >= 1 && N <= 0x7fffff00LL && H <= 0x7fffffffLL && V <= 0x7fffffffLL;
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
  constexpr int smem = (SORT_WARPS * MAX_BINS + MAX_BINS + MAX_BINS / 32) * 4;
  e = cudaFuncSetAttribute(k_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_status(e);
  k_sort<<<SORT_CTAS, SORT_THREADS, smem, s>>>(so);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_status(e);

  SumArgs a = {};
  a.keys = so.passes & 1 ? so.k1 : so.k0;
  a.pos = so.passes & 1 ? so.p1 : so.p0;
  a.N = (int)x->N;
  a.V = x->V;
  a.H = x->H;
  a.dout = x->dout;
  a.lddout = x->lddout;
  a.dE = x->dE;
  a.lddE = x->lddE;
  a.scale = x->scale;
  a.ovw = ovw;
  a.part = (float*)(ws + l.part);
  const bool same = x->dE_dtype == x->dtype;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(sums<float, float>(a, s));
    case FLCE_BF16:
      return cuda_status(same ? sums<__nv_bfloat16, __nv_bfloat16>(a, s) : sums<__nv_bfloat16, float>(a, s));
    default: return cuda_status(same ? sums<__half, __half>(a, s) : sums<__half, float>(a, s));
  }
}
