// Residual-adding RMS norm, forward and backward, with 8-bit outputs.
//
//   h = x + r,  rstd = (mean_c h_c^2 + eps)^-1/2,  y_c = h_c rstd (w_c + off)
//   xhat = h rstd,  g = dy (w + off),
//   dx = rstd (g - xhat mean_c(g_c xhat_c)) + dh,   dw_c += sum_rows dy_c xhat_c
//
// Both directions read every operand once and write every output once; they are bound by
// HBM. A row is held in the registers of a group of warps between the reduction over its
// columns and the outputs, so nothing is read twice. Rows too long for the registers
// (k_rms_fwd_long / k_rms_bwd_long) are read twice, the second time mostly from L2.
#include <math.h>

#include "flce_ops.cuh"

namespace flce {
namespace {

struct FwdArgs {
  int64_t N, H;
  float eps, off, inv_h;
  const void *x, *res, *w;
  int64_t ldx, ldres;
  void *h, *y;
  int64_t ldh, ldy;
  float* rstd;
  uint8_t *y8, *h8;
  int64_t ldy8, ldh8;
  float *y8s, *h8s;
  int64_t nblk;  // scales per row
};

struct BwdArgs {
  int64_t N, H;
  float off, inv_h;
  const void *dy, *h, *w, *dh;
  int64_t lddy, ldh, lddh;
  const uint8_t* h8;
  int64_t ldh8;
  const float *h8s, *rstd;
  int64_t nblk;
  void* dx;
  int64_t lddx;
  float* part;  // [row groups, H] partial dweight sums, or null
};

constexpr int MAX_WARPS = 32;

// Sum over the `wpr` warps of a row group; every thread of the block calls it. `red` holds
// one float per warp of the block; two buffers are used in turn, so one barrier per sum is
// enough.
__device__ __forceinline__ float group_sum(float v, float* red, int wpr, int warp_in_block, int group) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp_in_block] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < wpr; ++i) t += red[group * wpr + i];
  return t;
}

template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(512) k_rms_fwd(const __grid_constant__ FwdArgs a, int wpr) {
  __shared__ float red[MAX_WARPS];
  const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5;
  const int group = wb / wpr, w = wb % wpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32 / wpr) + group;
  const bool live = row < a.N;
  float v[NV][EPV];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[j][e] = 0.0f;
    if (live && c < a.H) Vec<T, EPV>::load((const T*)a.x + row * a.ldx + c, v[j]);
  }
  if (a.res != nullptr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
      if (live && c < a.H) {
        float r[EPV];
        Vec<T, EPV>::load((const T*)a.res + row * a.ldres + c, r);
#pragma unroll
        for (int e = 0; e < EPV; ++e) v[j][e] += r[e];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < EPV; ++e) ss = fmaf(v[j][e], v[j][e], ss);
  const float var = group_sum(ss, red, wpr, wb, group) * a.inv_h;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (!live) return;
  if (a.rstd != nullptr && w == 0 && lane == 0) a.rstd[row] = rstd;
  if (a.h != nullptr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
      if (c < a.H) Vec<T, EPV>::store((T*)a.h + row * a.ldh + c, v[j]);
    }
  }
  if (a.h8 != nullptr) q_row_piece<EPV, NV>(v, w, lane, a.H, a.h8 + row * a.ldh8, a.h8s + row * a.nblk, 1.0f);
  if (a.y == nullptr && a.y8 == nullptr) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
    if (c < a.H) {
      float wt[EPV], o[EPV];
      Vec<T, EPV>::load((const T*)a.w + c, wt);
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        v[j][e] *= wt[e] + a.off;
        o[e] = v[j][e] * rstd;
      }
      if (a.y != nullptr) Vec<T, EPV>::store((T*)a.y + row * a.ldy + c, o);
    }
  }
  if (a.y8 != nullptr) q_row_piece<EPV, NV>(v, w, lane, a.H, a.y8 + row * a.ldy8, a.y8s + row * a.nblk, rstd);
}

// Rows of any length: a block per row, two passes over it in pieces of 4 x 128 columns per
// warp; the second pass writes (h may be x or the residual: a thread rewrites only what it
// has just read).
template <typename T>
__global__ void __launch_bounds__(512) k_rms_fwd_long(const __grid_constant__ FwdArgs a) {
  __shared__ float red[MAX_WARPS];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* r = a.res ? (const T*)a.res + row * a.ldres : nullptr;
  float ss = 0.0f;
  for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
    const float h = r ? to_f<T>(x[c]) + to_f<T>(r[c]) : to_f<T>(x[c]);
    ss = fmaf(h, h, ss);
  }
  const float rstd = 1.0f / sqrtf(group_sum(ss, red, nw, w, 0) * a.inv_h + a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
  for (int64_t p = w; p * Q_BLOCK < a.H; p += nw) {  // one 128-column block per warp and turn
    float v[4][1];
    const int64_t c0 = p * Q_BLOCK;
    const int64_t left = a.H - c0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + j * 32 + lane;
      v[j][0] = 0.0f;
      if (c < a.H) {
        v[j][0] = r ? to_f<T>(x[c]) + to_f<T>(r[c]) : to_f<T>(x[c]);
        if (a.h != nullptr) ((T*)a.h)[row * a.ldh + c] = from_f<T>(v[j][0]);
      }
    }
    if (a.h8 != nullptr)
      q_row_piece<1, 4>(v, 0, lane, left, a.h8 + row * a.ldh8 + c0, a.h8s + row * a.nblk + p, 1.0f);
    if (a.y == nullptr && a.y8 == nullptr) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + j * 32 + lane;
      if (c < a.H) {
        v[j][0] *= to_f<T>(((const T*)a.w)[c]) + a.off;
        if (a.y != nullptr) ((T*)a.y)[row * a.ldy + c] = from_f<T>(v[j][0] * rstd);
      }
    }
    if (a.y8 != nullptr)
      q_row_piece<1, 4>(v, 0, lane, left, a.y8 + row * a.ldy8 + c0, a.y8s + row * a.nblk + p, rstd);
  }
}

// Backward: a row group walks the rows group, group + groups, ...; its threads keep their
// columns' dweight sums in registers and write them once, as one row of a.part.
template <typename T, int EPV, int NV, bool Q8>
__global__ void __launch_bounds__(512) k_rms_bwd(const __grid_constant__ BwdArgs a, int wpr) {
  __shared__ float red[2][MAX_WARPS];
  const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5;
  const int rpb = blockDim.x / 32 / wpr;
  const int group = wb / wpr, w = wb % wpr;
  const int64_t g0 = (int64_t)blockIdx.x * rpb + group, step = (int64_t)gridDim.x * rpb;
  float wt[NV][EPV], dw[NV][EPV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
#pragma unroll
    for (int e = 0; e < EPV; ++e) wt[j][e] = dw[j][e] = 0.0f;
    if (c < a.H) {
      Vec<T, EPV>::load((const T*)a.w + c, wt[j]);
#pragma unroll
      for (int e = 0; e < EPV; ++e) wt[j][e] += a.off;
    }
  }
  int buf = 0;
  // every group of the block takes the same number of turns (the sums hold barriers)
  const int64_t turns = (a.N - (int64_t)blockIdx.x * rpb + step - 1) / step;
  for (int64_t t = 0; t < turns; ++t, buf ^= 1) {
    const int64_t row = g0 + t * step;
    const bool live = row < a.N;
    const float rstd = live ? a.rstd[row] : 0.0f;
    float dy[NV][EPV], xh[NV][EPV];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
#pragma unroll
      for (int e = 0; e < EPV; ++e) dy[j][e] = xh[j][e] = 0.0f;
      if (live && c < a.H) {
        Vec<T, EPV>::load((const T*)a.dy + row * a.lddy + c, dy[j]);
        float f = rstd;
        if constexpr (Q8) {
          q_load<EPV>(a.h8 + row * a.ldh8 + c, xh[j]);
          f *= a.h8s[row * a.nblk + c / Q_BLOCK];
        } else {
          Vec<T, EPV>::load((const T*)a.h + row * a.ldh + c, xh[j]);
        }
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          xh[j][e] *= f;
          dot = fmaf(dy[j][e] * wt[j][e], xh[j][e], dot);
          dw[j][e] = fmaf(dy[j][e], xh[j][e], dw[j][e]);
        }
      }
    }
    const float m = group_sum(dot, red[buf], wpr, wb, group) * a.inv_h;
    if (!live || a.dx == nullptr) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
      if (c < a.H) {
        float o[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) o[e] = rstd * (dy[j][e] * wt[j][e] - xh[j][e] * m);
        if (a.dh != nullptr) {
          float d[EPV];
          Vec<T, EPV>::load((const T*)a.dh + row * a.lddh + c, d);
#pragma unroll
          for (int e = 0; e < EPV; ++e) o[e] += d[e];
        }
        Vec<T, EPV>::store((T*)a.dx + row * a.lddx + c, o);
      }
    }
  }
  if (a.part != nullptr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
      if (c < a.H) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) a.part[g0 * a.H + c + e] = dw[j][e];
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ float long_xhat(const BwdArgs& a, int64_t row, int64_t c, float rstd) {
  if (a.h8 != nullptr)
    return q_unpack2(a.h8[row * a.ldh8 + c]).x * (rstd * a.h8s[row * a.nblk + c / Q_BLOCK]);
  return to_f<T>(((const T*)a.h)[row * a.ldh + c]) * rstd;
}

// Rows of any length, dx alone: a block per row, two passes.
template <typename T>
__global__ void __launch_bounds__(512) k_rms_bwd_long(const __grid_constant__ BwdArgs a) {
  __shared__ float red[MAX_WARPS];
  const int64_t row = blockIdx.x;
  const float rstd = a.rstd[row];
  const T* dy = (const T*)a.dy + row * a.lddy;
  const T* w = (const T*)a.w;
  float dot = 0.0f;
  for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x)
    dot = fmaf(to_f<T>(dy[c]) * (to_f<T>(w[c]) + a.off), long_xhat<T>(a, row, c, rstd), dot);
  const float m = group_sum(dot, red, blockDim.x >> 5, threadIdx.x >> 5, 0) * a.inv_h;
  for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
    float o = rstd * (to_f<T>(dy[c]) * (to_f<T>(w[c]) + a.off) - long_xhat<T>(a, row, c, rstd) * m);
    if (a.dh != nullptr) o += to_f<T>(((const T*)a.dh)[row * a.lddh + c]);
    ((T*)a.dx)[row * a.lddx + c] = from_f<T>(o);
  }
}

// Rows of any length, dweight partials alone: block (x, y) sums rows y, y + gridDim.y, ...
// of 256 columns.
template <typename T>
__global__ void __launch_bounds__(256) k_rms_dw_long(const __grid_constant__ BwdArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.N; row += gridDim.y)
    s = fmaf(to_f<T>(((const T*)a.dy)[row * a.lddy + c]), long_xhat<T>(a, row, c, a.rstd[row]), s);
  a.part[(int64_t)blockIdx.y * a.H + c] = s;
}

// dweight (+)= sum of the partial rows, in a fixed order: a block takes 32 columns, its
// eight warps every eighth row, then the eight sums are added in warp order.
template <typename D>
__global__ void __launch_bounds__(256) k_rms_dw_sum(const float* part, int64_t rows, int64_t H, D* dw, bool ovw) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < H)
    for (int64_t r = w; r < rows; r += 8) t += part[r * H + c];
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < H) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) u += s[i][lane];
    dw[c] = from_f<D>(ovw ? u : to_f<D>(dw[c]) + u);
  }
}

constexpr int BWD_BLOCKS_PER_SM = 2;
constexpr int LONG_DW_ROWS = 64;  // row groups of k_rms_dw_long

// Warps per row and vectors per thread of a row of H elements in vectors of EPV: the fewest
// warps that hold it; 0 when none does.
struct Shape {
  int wpr, nv;
};
Shape row_shape(int64_t H, int epv) {
  const int64_t nvec = cdiv64(H, epv);
  const int small = epv == 1 ? 8 : 2, large = epv == 1 ? 16 : 4;
  for (int wpr = 1; wpr <= 16; wpr *= 2)
    if ((int64_t)wpr * 32 * small >= nvec) return {wpr, small};
  if ((int64_t)16 * 32 * large >= nvec) return {16, large};
  return {0, 0};
}

// Rows in the dweight partials of a backward over N rows: at most one per row group of the
// largest grid.
int64_t partial_rows(int64_t N) {
  const int64_t most = (int64_t)num_sms() * BWD_BLOCKS_PER_SM * 16;
  const int64_t rows = N < most ? N + 16 : most;
  return rows > LONG_DW_ROWS ? rows : LONG_DW_ROWS;
}

template <typename T, int EPV, int NV>
void launch_fwd(const FwdArgs& a, int wpr, cudaStream_t s) {
  const int threads = wpr * 32 < 128 ? 128 : wpr * 32;
  const int64_t rpb = threads / 32 / wpr;
  k_rms_fwd<T, EPV, NV><<<(unsigned)cdiv64(a.N, rpb), threads, 0, s>>>(a, wpr);
}

template <typename T>
cudaError_t fwd(const FwdArgs& a, bool wide, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const Shape p = row_shape(a.H, wide ? W : 1);
  if (p.wpr == 0) {
    k_rms_fwd_long<T><<<(unsigned)a.N, 512, 0, s>>>(a);
  } else if (wide) {
    if (p.nv == 2) launch_fwd<T, W, 2>(a, p.wpr, s);
    else launch_fwd<T, W, 4>(a, p.wpr, s);
  } else {
    if (p.nv == 8) launch_fwd<T, 1, 8>(a, p.wpr, s);
    else launch_fwd<T, 1, 16>(a, p.wpr, s);
  }
  return cudaGetLastError();
}

// Grid of the backward and the number of partial rows it writes.
template <typename T, int EPV, int NV>
int64_t launch_bwd(const BwdArgs& a, int wpr, cudaStream_t s) {
  const int threads = 512;
  const int64_t rpb = threads / 32 / wpr;
  int64_t blocks = (int64_t)num_sms() * BWD_BLOCKS_PER_SM;
  if (blocks > cdiv64(a.N, rpb)) blocks = cdiv64(a.N, rpb);
  if (a.h8 != nullptr) k_rms_bwd<T, EPV, NV, true><<<(unsigned)blocks, threads, 0, s>>>(a, wpr);
  else k_rms_bwd<T, EPV, NV, false><<<(unsigned)blocks, threads, 0, s>>>(a, wpr);
  return blocks * rpb;
}

template <typename T>
cudaError_t bwd(const BwdArgs& a, bool wide, int64_t& part_rows, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const Shape p = row_shape(a.H, wide ? W : 1);
  if (p.wpr == 0) {
    if (a.dx != nullptr) k_rms_bwd_long<T><<<(unsigned)a.N, 512, 0, s>>>(a);
    if (a.part != nullptr) {
      part_rows = LONG_DW_ROWS;
      k_rms_dw_long<T><<<dim3((unsigned)cdiv64(a.H, 256), LONG_DW_ROWS), 256, 0, s>>>(a);
    }
  } else if (wide) {
    part_rows = p.nv == 2 ? launch_bwd<T, W, 2>(a, p.wpr, s) : launch_bwd<T, W, 4>(a, p.wpr, s);
  } else {
    part_rows = p.nv == 8 ? launch_bwd<T, 1, 8>(a, p.wpr, s) : launch_bwd<T, 1, 16>(a, p.wpr, s);
  }
  return cudaGetLastError();
}

bool sizes_ok(int64_t N, int64_t H) { return N >= 0 && H >= 1 && N <= 0x7fffffffLL && H <= 0x7fffffffLL; }
// A matrix operand: element-aligned, pitch at least a row.
bool mat_ok(const void* p, int64_t ld, int64_t H, int esz) { return p != nullptr && aligned_to(p, esz) && ld >= H; }

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int32_t flce_rmsnorm_fwd(const flce_rmsnorm_args* x, void* stream) {
  if (x == nullptr || !sizes_ok(x->N, x->H) || !valid_dtype(x->dtype) || x->flags != 0) return FLCE_ERR_INVALID_ARG;
  if (!(x->eps > 0.0f) || !isfinite(x->eps) || !isfinite(x->weight_offset)) return FLCE_ERR_INVALID_ARG;
  if (x->N == 0) return FLCE_OK;
  const int esz = dtype_size(x->dtype);
  const int64_t H = x->H;
  if (!mat_ok(x->x, x->ldx, H, esz) || !x->weight || !aligned_to(x->weight, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->residual && !mat_ok(x->residual, x->ldres, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->h && !mat_ok(x->h, x->ldh, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->y && !mat_ok(x->y, x->ldy, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->rstd && !aligned_to(x->rstd, 4)) return FLCE_ERR_INVALID_ARG;
  if (x->y8 && (x->ldy8 < H || !x->y8_scale || !aligned_to(x->y8_scale, 4))) return FLCE_ERR_INVALID_ARG;
  if (x->h8 && (x->ldh8 < H || !x->h8_scale || !aligned_to(x->h8_scale, 4))) return FLCE_ERR_INVALID_ARG;

  FwdArgs a = {};
  a.N = x->N;
  a.H = H;
  a.eps = x->eps;
  a.off = x->weight_offset;
  a.inv_h = (float)(1.0 / (double)H);
  a.x = x->x;
  a.ldx = x->ldx;
  a.res = x->residual;
  a.ldres = x->ldres;
  a.w = x->weight;
  a.h = x->h;
  a.ldh = x->ldh;
  a.y = x->y;
  a.ldy = x->ldy;
  a.rstd = x->rstd;
  a.y8 = (uint8_t*)x->y8;
  a.ldy8 = x->ldy8;
  a.y8s = x->y8_scale;
  a.h8 = (uint8_t*)x->h8;
  a.ldh8 = x->ldh8;
  a.h8s = x->h8_scale;
  a.nblk = cdiv64(H, Q_BLOCK);
  const int epv = 16 / esz;
  const bool wide = H % epv == 0 && rows16(a.x, a.ldx, esz) && (!a.res || rows16(a.res, a.ldres, esz)) &&
                    aligned_to(a.w, 16) && (!a.h || rows16(a.h, a.ldh, esz)) && (!a.y || rows16(a.y, a.ldy, esz)) &&
                    (!a.y8 || (aligned_to(a.y8, epv) && a.ldy8 % epv == 0)) &&
                    (!a.h8 || (aligned_to(a.h8, epv) && a.ldh8 % epv == 0));
  cudaStream_t s = (cudaStream_t)stream;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(fwd<float>(a, wide, s));
    case FLCE_BF16: return cuda_status(fwd<__nv_bfloat16>(a, wide, s));
    default: return cuda_status(fwd<__half>(a, wide, s));
  }
}

extern "C" size_t flce_rmsnorm_workspace_size(int64_t N, int64_t H) {
  if (!sizes_ok(N, H)) return 0;
  return round_up((size_t)partial_rows(N) * (size_t)H * 4, 256);
}

extern "C" int32_t flce_rmsnorm_bwd(const flce_rmsnorm_bwd_args* x, void* stream) {
  if (x == nullptr || !sizes_ok(x->N, x->H) || !valid_dtype(x->dtype)) return FLCE_ERR_INVALID_ARG;
  if ((x->flags & ~FLCE_FLAG_DW_OVERWRITE) != 0 || !isfinite(x->weight_offset)) return FLCE_ERR_INVALID_ARG;
  if (x->dweight && x->dweight_dtype != FLCE_F32 && x->dweight_dtype != x->dtype) return FLCE_ERR_UNSUPPORTED;
  const int esz = dtype_size(x->dtype);
  const int64_t N = x->N, H = x->H;
  const int wsz = x->dweight ? dtype_size(x->dweight_dtype) : 4;
  if (x->dweight && !aligned_to(x->dweight, wsz)) return FLCE_ERR_INVALID_ARG;
  const bool ovw = (x->flags & FLCE_FLAG_DW_OVERWRITE) != 0;
  cudaStream_t s = (cudaStream_t)stream;
  if (N == 0)
    return x->dweight && ovw ? cuda_status(cudaMemsetAsync(x->dweight, 0, (size_t)H * wsz, s)) : FLCE_OK;
  if (!mat_ok(x->dy, x->lddy, H, esz) || !x->weight || !aligned_to(x->weight, esz)) return FLCE_ERR_INVALID_ARG;
  if ((x->h != nullptr) == (x->h8 != nullptr) || !x->rstd || !aligned_to(x->rstd, 4)) return FLCE_ERR_INVALID_ARG;
  if (x->h && !mat_ok(x->h, x->ldh, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->h8 && (x->ldh8 < H || !x->h8_scale || !aligned_to(x->h8_scale, 4))) return FLCE_ERR_INVALID_ARG;
  if (x->dh && !mat_ok(x->dh, x->lddh, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (x->dx && !mat_ok(x->dx, x->lddx, H, esz)) return FLCE_ERR_INVALID_ARG;
  if (!x->dx && !x->dweight) return FLCE_OK;
  if (x->dweight) {
    if (!x->workspace || !aligned_to(x->workspace, 256)) return FLCE_ERR_INVALID_ARG;
    if (x->workspace_bytes < flce_rmsnorm_workspace_size(N, H)) return FLCE_ERR_WORKSPACE;
  }
  BwdArgs a = {};
  a.N = N;
  a.H = H;
  a.off = x->weight_offset;
  a.inv_h = (float)(1.0 / (double)H);
  a.dy = x->dy;
  a.lddy = x->lddy;
  a.h = x->h;
  a.ldh = x->ldh;
  a.w = x->weight;
  a.dh = x->dh;
  a.lddh = x->lddh;
  a.h8 = (const uint8_t*)x->h8;
  a.ldh8 = x->ldh8;
  a.h8s = x->h8_scale;
  a.rstd = x->rstd;
  a.nblk = cdiv64(H, Q_BLOCK);
  a.dx = x->dx;
  a.lddx = x->lddx;
  a.part = x->dweight ? (float*)x->workspace : nullptr;
  const int epv = 16 / esz;
  const bool wide = H % epv == 0 && rows16(a.dy, a.lddy, esz) && (!a.h || rows16(a.h, a.ldh, esz)) &&
                    (!a.h8 || (aligned_to(a.h8, epv) && a.ldh8 % epv == 0)) && aligned_to(a.w, 16) &&
                    (!a.dh || rows16(a.dh, a.lddh, esz)) && (!a.dx || rows16(a.dx, a.lddx, esz));
  int64_t rows = 0;
  cudaError_t e;
  switch (x->dtype) {
    case FLCE_F32: e = bwd<float>(a, wide, rows, s); break;
    case FLCE_BF16: e = bwd<__nv_bfloat16>(a, wide, rows, s); break;
    default: e = bwd<__half>(a, wide, rows, s); break;
  }
  if (e != cudaSuccess || !x->dweight) return cuda_status(e);
  const unsigned blocks = (unsigned)cdiv64(H, 32);
  if (x->dweight_dtype == FLCE_F32)
    k_rms_dw_sum<float><<<blocks, 256, 0, s>>>(a.part, rows, H, (float*)x->dweight, ovw);
  else if (x->dweight_dtype == FLCE_BF16)
    k_rms_dw_sum<__nv_bfloat16><<<blocks, 256, 0, s>>>(a.part, rows, H, (__nv_bfloat16*)x->dweight, ovw);
  else
    k_rms_dw_sum<__half><<<blocks, 256, 0, s>>>(a.part, rows, H, (__half*)x->dweight, ovw);
  return cuda_status(cudaGetLastError());
}
