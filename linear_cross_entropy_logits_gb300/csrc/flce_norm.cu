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
//
// Accesses are 32 bytes a thread where every operand's rows allow it, else 16, else two elements,
// else one: 8192 x 4096 bf16 with residual, 16-bit and 8-bit output and 8-bit checkpoint in
// 55 us (5.0 TB/s in DRAM under ncu; floor 50) against 68 with 16 bytes and a test for
// infinities per element. Backward of the same shape from the checkpoint, with the residual's
// gradient: 46 + 6 us (floor 35).
#include <math.h>

#include <atomic>

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
__global__ void __launch_bounds__(EPV <= 2 ? 1024 : 512) k_rms_fwd(const __grid_constant__ FwdArgs a, int wpr) {
  __shared__ float red[MAX_WARPS];
  const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5;
  const int group = wb / wpr, w = wb - group * wpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32 / wpr) + group;
  const bool live = row < a.N;
  const int c0 = (w * NV * 32 + lane) * EPV, H = (int)a.H;
  const T* xp = (const T*)a.x + row * a.ldx;
  const T* resp = (const T*)a.res + row * a.ldres;
  float v[NV][EPV];
  Raw<T, EPV> x[NV], r[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * 32 * EPV;
    x[j].zero();
    r[j].zero();
    if (live && c < H) {
      x[j].load(xp + c);
      if (a.res != nullptr) r[j].load(resp + c);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      v[j][e] = x[j].get(e);
      if (a.res != nullptr) v[j][e] += r[j].get(e);
      ss = fmaf(v[j][e], v[j][e], ss);
    }
  }
  const float var = group_sum(ss, red, wpr, wb, group) * a.inv_h;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (!live) return;
  if (a.rstd != nullptr && w == 0 && lane == 0) a.rstd[row] = rstd;
  if (a.h != nullptr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * 32 * EPV;
      if (c < H) Vec<T, EPV>::store((T*)a.h + row * a.ldh + c, v[j]);
    }
  }
  if (a.h8 != nullptr) q_row_piece<EPV, NV>(v, w, lane, H, a.h8 + row * a.ldh8, a.h8s + row * a.nblk, 1.0f);
  if (a.y == nullptr && a.y8 == nullptr) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * 32 * EPV;
    if (c < H) {
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
  if (a.y8 != nullptr) q_row_piece<EPV, NV>(v, w, lane, H, a.y8 + row * a.ldy8, a.y8s + row * a.nblk, rstd);
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
    const int left = (int)(a.H - c0 < Q_BLOCK ? a.H - c0 : Q_BLOCK);
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

// Sum over a row group by a barrier of its own (wpr > 1), for groups that walk their rows
// independently. `red`: the group's floats, wpr of them and zeros up to a multiple of four; two
// buffers are used in turn.
__device__ __forceinline__ float group_sum_own(float v, float* red, int wpr, int w, int group) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) red[w] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(wpr * 32) : "memory");
  float t = 0.0f;
  for (int i = 0; i < wpr; i += 4) {
    const float4 u = *(const float4*)(red + i);
    t += (u.x + u.y) + (u.z + u.w);
  }
  return t;
}

// The dweight sums of a block's groups, added in group order, as row blockIdx.x of a.part.
template <int EPV, int NV>
__device__ __forceinline__ void put_partials(const BwdArgs& a, const float (&dw)[NV][EPV], float* sums, int rpb,
                                             int group, int w, int lane) {
  float* out = a.part + (int64_t)blockIdx.x * a.H;
  for (int g = 0; g < rpb; ++g) {
    if (group == g) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t c = ((int64_t)(w * NV + j) * 32 + lane) * EPV;
        if (c < a.H) {
#pragma unroll
          for (int e = 0; e < EPV; ++e) {
            const float u = g == 0 ? dw[j][e] : sums[c + e] + dw[j][e];
            if (g == rpb - 1) out[c + e] = u;
            else sums[c + e] = u;
          }
        }
      }
    }
    if (g < rpb - 1) __syncthreads();
  }
}

// Copies to shared memory without registers.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// Backward of rows whose operands allow 16-byte copies: a row group walks the rows group,
// group + groups, .... Each thread copies its own pieces of the next RING - 1 rows to shared
// memory (cp.async) and reads back only those: no registers and no barriers for what is in
// flight. g and xhat stay in registers over the row's sum, and the arithmetic is done two
// elements at a time (packed fp32). The columns' dweight sums stay in registers throughout.
// RING is 4; fp32 rows over 4096 columns, of which four do not fit shared memory, take 2 (4096 x
// 8192 from the checkpoint 69 us, 107 with the row in registers as in k_rms_bwd). One block of 512
// threads an SM: with 768 threads (80 registers) it took 15 us longer, with the next
// row in registers instead of shared memory 2 to 10 us. What bounds it now is the row's chain of
// loads, sum and barrier at four warps a scheduler.
template <typename T, int RING>
constexpr int RING_WARPS = 32 * RING * sizeof(T) > 256 ? 8 : 16;  // a block's, for its ring to fit
template <typename T, int NV, bool Q8, int RING>
__global__ void __launch_bounds__(512, 1) k_rms_bwd_ring(const __grid_constant__ BwdArgs a, int wpr) {
  constexpr int EPV = 16 / sizeof(T);
  constexpr int NP = EPV / 2;        // pairs per vector
  constexpr int HB = Q8 ? EPV : 16;  // bytes of a vector of h
  constexpr int VSTEP = 32 * EPV;    // elements from one of a thread's vectors to the next
  extern __shared__ uint4 ring[];    // [RING][dy, dh, h of the threads' vectors], then the groups' sums
  __shared__ __align__(16) float red[2][4 * MAX_WARPS];
  let_next_start();
  const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5;
  const int rpb = blockDim.x / 32 / wpr;
  const int group = wb / wpr, w = wb - group * wpr;
  const int64_t g0 = (int64_t)blockIdx.x * rpb + group, step = (int64_t)gridDim.x * rpb;
  const int64_t c0 = ((int64_t)w * NV * 32 + lane) * EPV;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = c0 + j * VSTEP < a.H;
  for (int i = threadIdx.x; i < 8 * MAX_WARPS; i += blockDim.x) (&red[0][0])[i] = 0.0f;
  __syncthreads();
  float* gred = &red[0][0] + group * ((wpr + 3) & ~3);

  const uint32_t stage = blockDim.x * NV * (32 + HB);  // bytes
  const uint32_t vstep = blockDim.x * 16, hstep = blockDim.x * HB;
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
  const uint32_t hat = (uint32_t)__cvta_generic_to_shared(ring) + blockDim.x * NV * 32 + threadIdx.x * HB;
  // where the next row to be copied lies
  int64_t left = a.N - g0;  // rows from it on
  const T* s_dy = (const T*)a.dy + g0 * a.lddy + c0;
  const T* s_dh = (const T*)a.dh + g0 * a.lddh + c0;
  const uint8_t* s_h = Q8 ? a.h8 + g0 * a.ldh8 + c0 : (const uint8_t*)((const T*)a.h + g0 * a.ldh + c0);
  const int64_t hpitch = Q8 ? step * a.ldh8 : step * a.ldh * (int64_t)sizeof(T);
  constexpr int HSTEP = VSTEP * (Q8 ? 1 : (int)sizeof(T));
  const bool has_dh = a.dh != nullptr;
  auto fetch = [&](uint32_t off) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j]) {
          copy_async<16>(at + off + j * vstep, s_dy + j * VSTEP);
          if (has_dh) copy_async<16>(at + off + (NV + j) * vstep, s_dh + j * VSTEP);
          copy_async<HB>(hat + off + j * hstep, s_h + j * HSTEP);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    left -= step;
    s_dy += step * a.lddy;
    s_dh += step * a.lddh;
    s_h += hpitch;
  };
#pragma unroll
  for (int r = 0; r < RING - 1; ++r) fetch(r * stage);

  f2 wt[NV][NP], dw[NV][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = 0.0f;
    if (in[j]) Vec<T, EPV>::load((const T*)a.w + c0 + j * VSTEP, v);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      wt[j][e] = f2_make(v[2 * e] + a.off, v[2 * e + 1] + a.off);
      dw[j][e] = f2_make(0.0f, 0.0f);
    }
  }
  // a row's 1/rms and block scales, read one turn ahead
  const float* s_r = a.rstd + g0;
  const float* s_f = Q8 ? a.h8s + g0 * a.nblk + c0 / Q_BLOCK : nullptr;
  float rs_next = 0.0f, f_next[NV];
  auto factors = [&](bool live) {
    if (live) {
      rs_next = *s_r;
      s_r += step;
#pragma unroll
      for (int j = 0; j < NV; ++j) f_next[j] = Q8 && in[j] ? s_f[j * VSTEP / Q_BLOCK] : 1.0f;
      s_f += step * a.nblk;
    }
  };
  factors(g0 < a.N);
  T* dx = (T*)a.dx + g0 * a.lddx + c0;
  uint32_t off = 0, free_off = (RING - 1) * stage;  // the slot of this row, and the one read last turn
  int buf = 0;
  for (int64_t row = g0; row < a.N; row += step, buf ^= 4 * MAX_WARPS) {
    const float rstd = rs_next;
    float f[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) f[j] = f_next[j] * rstd;
    factors(row + step < a.N);
    fetch(free_off);
    asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
    auto vec = [&](uint32_t p, f2 (&x)[NP]) {
      Raw<T, EPV> r;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(p));
#pragma unroll
      for (int e = 0; e < NP; ++e) x[e] = f2_make(r.get(2 * e), r.get(2 * e + 1));
    };
    f2 g[NV][NP], xh[NV][NP], dot = f2_make(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < NP; ++e) g[j][e] = xh[j][e] = f2_make(0.0f, 0.0f);
      if (in[j]) {
        f2 d[NP], x[NP];
        vec(at + off + j * vstep, d);
        if constexpr (Q8) {
          RawQ<EPV> q;
          if constexpr (EPV == 8)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.w[0]), "=r"(q.w[1]) : "r"(hat + off + j * hstep));
          else
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(q.w[0]) : "r"(hat + off + j * hstep));
          float v[EPV];
          q.unpack(v);
#pragma unroll
          for (int e = 0; e < NP; ++e) x[e] = f2_make(v[2 * e], v[2 * e + 1]);
        } else {
          vec(hat + off + j * hstep, x);
        }
        const f2 ff = f2_make(f[j], f[j]);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          xh[j][e] = f2_mul(x[e], ff);
          g[j][e] = f2_mul(d[e], wt[j][e]);
          dot = f2_fma(g[j][e], xh[j][e], dot);
          dw[j][e] = f2_fma(d[e], xh[j][e], dw[j][e]);
        }
      }
    }
    float dlo, dhi;
    f2_get(dot, dlo, dhi);
    const float m = group_sum_own(dlo + dhi, gred + buf, wpr, w, group) * a.inv_h;
    if (a.dx != nullptr) {
      const f2 r2 = f2_make(rstd, rstd), m2 = f2_make(-rstd * m, -rstd * m);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j]) {
          f2 d[NP];
#pragma unroll
          for (int e = 0; e < NP; ++e) d[e] = f2_make(0.0f, 0.0f);
          if (has_dh) vec(at + off + (NV + j) * vstep, d);
          float o[EPV];
#pragma unroll
          for (int e = 0; e < NP; ++e)
            f2_get(f2_fma(r2, g[j][e], f2_fma(m2, xh[j][e], d[e])), o[2 * e], o[2 * e + 1]);
          Vec<T, EPV>::store(dx + j * VSTEP, o);
        }
      }
      dx += step * a.lddx;
    }
    free_off = off;
    off = off == (RING - 1) * stage ? 0 : off + stage;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (a.part == nullptr) return;
  __syncthreads();  // the ring's memory is free: it takes the groups' sums
  float dws[NV][EPV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < NP; ++e) f2_get(dw[j][e], dws[j][2 * e], dws[j][2 * e + 1]);
  put_partials<EPV, NV>(a, dws, (float*)ring, rpb, group, w, lane);
}

// Backward of other rows (longer, or without 16-byte accesses): a row group walks the rows group,
// group + groups, ...; its threads keep their columns' dweight sums in registers. All of a row is
// loaded before its sum is taken. At the end the block's groups add their sums in group order and
// write one row of a.part. Accesses of one or two elements are bound by the instructions they take:
// eight elements a thread, 64 registers and all 32 warps' worth an SM (4097 x 5122 bf16 in pairs
// 60 us, singly 67, singly with sixteen a thread 127).
template <typename T, int EPV, int NV, bool Q8>
__global__ void __launch_bounds__(EPV <= 2 ? 1024 : 512, 1) k_rms_bwd(const __grid_constant__ BwdArgs a, int wpr) {
  constexpr int JB = Q_VECTORS<EPV>;  // a thread's vectors that share an 8-bit row's scale
  __shared__ float red[2][MAX_WARPS];
  extern __shared__ float sums[];  // [H] where the block has several groups
  let_next_start();
  const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5;
  const int rpb = blockDim.x / 32 / wpr;
  const int group = wb / wpr, w = wb - group * wpr;
  const int64_t g0 = (int64_t)blockIdx.x * rpb + group, step = (int64_t)gridDim.x * rpb;
  const int c0 = (w * NV * 32 + lane) * EPV, H = (int)a.H;
  Raw<T, EPV> wt[NV];
  float dw[NV][EPV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * 32 * EPV;
    wt[j].zero();
    if (c < H) wt[j].load((const T*)a.w + c);
#pragma unroll
    for (int e = 0; e < EPV; ++e) dw[j][e] = 0.0f;
  }
  int buf = 0;
  // every group of the block takes the same number of turns (the sums hold barriers)
  const int64_t turns = (a.N - (int64_t)blockIdx.x * rpb + step - 1) / step;
  for (int64_t t = 0; t < turns; ++t, buf ^= 1) {
    const int64_t row = g0 + t * step;
    const bool live = row < a.N;
    Raw<T, EPV> dy[NV], dh[NV];
    typename std::conditional<Q8, RawQ<EPV>, Raw<T, EPV>>::type h[NV];
    float f[NV / JB];  // what h is multiplied by to give xhat
    const float rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * 32 * EPV;
      if (j % JB == 0) f[j / JB] = rstd;
      dy[j].zero();
      dh[j].zero();
#pragma unroll
      for (int i = 0; i < h[j].W; ++i) h[j].w[i] = 0u;
      if (live && c < H) {
        dy[j].load((const T*)a.dy + row * a.lddy + c);
        if constexpr (Q8) {
          h[j].load(a.h8 + row * a.ldh8 + c);
          if (j % JB == 0) f[j / JB] = a.h8s[row * a.nblk + c / Q_BLOCK];
        } else {
          h[j].load((const T*)a.h + row * a.ldh + c);
        }
        if (a.dh != nullptr) dh[j].load((const T*)a.dh + row * a.lddh + c);
      }
    }
    float dot = 0.0f, keep[NV];  // single elements: xhat
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (Q8 && j % JB == 0) f[j / JB] *= rstd;
      float xh[EPV];
      h[j].unpack(xh);
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        const float d = dy[j].get(e), x = xh[e] * f[j / JB];
        dot = fmaf(d * (wt[j].get(e) + a.off), x, dot);
        dw[j][e] = fmaf(d, x, dw[j][e]);
        keep[j] = x;
      }
    }
    const float m = group_sum(dot, red[buf], wpr, wb, group) * a.inv_h;
    if (!live || a.dx == nullptr) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * 32 * EPV;
      if (c < H) {
        float xh[EPV], o[EPV];
        if constexpr (EPV > 1) h[j].unpack(xh);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const float x = EPV > 1 ? xh[e] * f[j / JB] : keep[j];
          o[e] = rstd * (dy[j].get(e) * (wt[j].get(e) + a.off) - x * m);
          if (a.dh != nullptr) o[e] += dh[j].get(e);
        }
        Vec<T, EPV>::store((T*)a.dx + row * a.lddx + c, o);
      }
    }
  }
  if (a.part == nullptr) return;
  put_partials<EPV, NV>(a, dw, sums, rpb, group, w, lane);
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

// dweight (+)= sum of the partial rows, in a fixed order: a block takes 32 columns, its 32
// warps every 32nd row, then the 32 sums are added in warp order.
template <typename D>
__global__ void __launch_bounds__(1024) k_rms_dw_sum(const float* part, int64_t rows, int64_t H, D* dw, bool ovw) {
  __shared__ float s[32][33];
  after_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < H) {
#pragma unroll 4
    for (int64_t r = w; r < rows; r += 32) t += part[r * H + c];
  }
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < H) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) u += s[i][lane];
    dw[c] = from_f<D>(ovw ? u : to_f<D>(dw[c]) + u);
  }
}

constexpr int BWD_BLOCKS_PER_SM = 2;
constexpr int LONG_DW_ROWS = 64;  // row groups of k_rms_dw_long

// Rows that take accesses of 32 bytes, 16 bytes, two elements or one.
enum Width { W32, W16, W2, W1 };

// Warps per row and vectors per thread of a row of H elements in vectors of EPV: the fewest
// warps with 16 elements a thread, else 16 warps with 32 (one or two elements an access: up to
// 32 warps with 8); 0 when none holds it.
struct Shape {
  int wpr, nv;
};
Shape row_shape(int64_t H, int epv) {
  const int64_t nvec = cdiv64(H, epv);
  if (epv <= 2) return {H <= 32 * 32 * 8 ? (int)cdiv64(H, 32 * 8) : 0, 8 / epv};
  const int small = 16 / epv, large = 2 * small;
  if (cdiv64(nvec, 32 * small) <= 16) return {(int)cdiv64(nvec, 32 * small), small};
  if (cdiv64(nvec, 32 * large) <= 16) return {16, large};
  return {0, 0};
}

// Rows of the dweight partials: at most one per block of the largest grid.
int64_t partial_rows() {
  const int64_t most = (int64_t)num_sms() * BWD_BLOCKS_PER_SM;
  return most > LONG_DW_ROWS ? most : LONG_DW_ROWS;
}

template <typename T, int EPV>
cudaError_t fwd_w(const FwdArgs& a, cudaStream_t s) {
  constexpr int NV = (EPV <= 2 ? 8 : 16) / EPV;
  const Shape p = row_shape(a.H, EPV);
  if (p.wpr == 0) {
    k_rms_fwd_long<T><<<(unsigned)a.N, 512, 0, s>>>(a);
  } else {
    const int64_t rpb = p.wpr >= 4 ? 1 : 4 / p.wpr;
    const unsigned blocks = (unsigned)cdiv64(a.N, rpb);
    const int threads = (int)rpb * p.wpr * 32;
    if (p.nv == NV) k_rms_fwd<T, EPV, NV><<<blocks, threads, 0, s>>>(a, p.wpr);
    else if constexpr (EPV > 2) k_rms_fwd<T, EPV, 2 * NV><<<blocks, threads, 0, s>>>(a, p.wpr);
  }
  return cudaGetLastError();
}
template <typename T>
cudaError_t fwd(const FwdArgs& a, Width w, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  switch (w) {
    case W32: return fwd_w<T, 2 * E>(a, s);
    case W16: return fwd_w<T, E>(a, s);
    case W2: return fwd_w<T, 2>(a, s);
    default: return fwd_w<T, 1>(a, s);
  }
}

template <typename T, int EPV, int NV>
int64_t launch_bwd(const BwdArgs& a, int wpr, cudaStream_t s) {
  const int64_t rpb = wpr > 16 ? 1 : 16 / wpr;
  const int threads = (int)rpb * wpr * 32;
  const size_t smem = rpb > 1 ? (size_t)a.H * 4 : 0;
  int64_t blocks = (int64_t)num_sms() * (EPV <= 2 && wpr <= 16 ? BWD_BLOCKS_PER_SM : 1);
  if (blocks > cdiv64(a.N, rpb)) blocks = cdiv64(a.N, rpb);
  if (a.h8 != nullptr) k_rms_bwd<T, EPV, NV, true><<<(unsigned)blocks, threads, smem, s>>>(a, wpr);
  else k_rms_bwd<T, EPV, NV, false><<<(unsigned)blocks, threads, smem, s>>>(a, wpr);
  return blocks;
}
template <typename T, int EPV>
cudaError_t bwd_w(const BwdArgs& a, int64_t& part_rows, cudaStream_t s) {
  constexpr int NV = (EPV <= 2 ? 8 : 16) / EPV;
  const Shape p = row_shape(a.H, EPV);
  if (p.wpr == 0) {
    // the sums first: dx may be dy itself
    if (a.part != nullptr) {
      part_rows = LONG_DW_ROWS;
      k_rms_dw_long<T><<<dim3((unsigned)cdiv64(a.H, 256), LONG_DW_ROWS), 256, 0, s>>>(a);
    }
    if (a.dx != nullptr) k_rms_bwd_long<T><<<(unsigned)a.N, 512, 0, s>>>(a);
  } else {
    // (rows in wider accesses come here with 32 elements a thread only)
    part_rows = launch_bwd<T, EPV, EPV <= 2 ? NV : 2 * NV>(a, p.wpr, s);
  }
  return cudaGetLastError();
}
template <typename T, int NV, bool Q8, int RING>
cudaError_t launch_ring(const BwdArgs& a, int wpr, int64_t& part_rows, cudaStream_t s) {
  constexpr int EPV = 16 / sizeof(T);
  const int64_t sms = num_sms();
  // as many groups a block as there are rows for
  int64_t rpb = cdiv64(a.N, sms);
  if (rpb > RING_WARPS<T, RING> / wpr) rpb = RING_WARPS<T, RING> / wpr;
  const int threads = (int)rpb * wpr * 32;
  constexpr int most = RING * 32 * RING_WARPS<T, RING> * NV * (32 + (Q8 ? EPV : 16));
  static_assert(most <= 232448 - 1024, "shared memory per block");
  const size_t smem = (size_t)RING * threads * NV * (32 + (Q8 ? EPV : 16));
  static std::atomic<bool> raised[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!raised[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_rms_bwd_ring<T, NV, Q8, RING>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    raised[dev].store(true, std::memory_order_relaxed);
  }
  part_rows = cdiv64(a.N, rpb) < sms ? cdiv64(a.N, rpb) : sms;
  k_rms_bwd_ring<T, NV, Q8, RING><<<(unsigned)part_rows, threads, smem, s>>>(a, wpr);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const BwdArgs& a, Width w, int64_t& part_rows, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  if (w == W1) return bwd_w<T, 1>(a, part_rows, s);
  if (w == W2) return bwd_w<T, 2>(a, part_rows, s);
  const int64_t wpr = cdiv64(a.H, 512);  // 16 elements a thread
  if (wpr <= RING_WARPS<T, 4>)
    return a.h8 ? launch_ring<T, 16 / E, true, 4>(a, (int)wpr, part_rows, s)
                : launch_ring<T, 16 / E, false, 4>(a, (int)wpr, part_rows, s);
  if constexpr (RING_WARPS<T, 4> < RING_WARPS<T, 2>) {
    if (wpr <= RING_WARPS<T, 2>)
      return a.h8 ? launch_ring<T, 16 / E, true, 2>(a, (int)wpr, part_rows, s)
                  : launch_ring<T, 16 / E, false, 2>(a, (int)wpr, part_rows, s);
  }
  return bwd_w<T, E>(a, part_rows, s);
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
  // the widest accesses that every operand's rows allow
  auto fits = [&](int bytes) {
    const int e = bytes / esz;  // elements, and bytes of the 8-bit rows
    return H % e == 0 && rows_by(a.x, a.ldx, esz, bytes) && (!a.res || rows_by(a.res, a.ldres, esz, bytes)) &&
           aligned_to(a.w, bytes) && (!a.h || rows_by(a.h, a.ldh, esz, bytes)) &&
           (!a.y || rows_by(a.y, a.ldy, esz, bytes)) && (!a.y8 || rows_by(a.y8, a.ldy8, 1, e)) &&
           (!a.h8 || rows_by(a.h8, a.ldh8, 1, e));
  };
  const Width w = fits(32) ? W32 : fits(16) ? W16 : fits(2 * esz) ? W2 : W1;
  cudaStream_t s = (cudaStream_t)stream;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(fwd<float>(a, w, s));
    case FLCE_BF16: return cuda_status(fwd<__nv_bfloat16>(a, w, s));
    default: return cuda_status(fwd<__half>(a, w, s));
  }
}

extern "C" size_t flce_rmsnorm_workspace_size(int64_t N, int64_t H) {
  if (!sizes_ok(N, H)) return 0;
  return round_up((size_t)partial_rows() * (size_t)H * 4, 256);
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
  auto fits = [&](int bytes) {
    const int e = bytes / esz;
    return H % e == 0 && rows_by(a.dy, a.lddy, esz, bytes) && (!a.h || rows_by(a.h, a.ldh, esz, bytes)) &&
           (!a.h8 || rows_by(a.h8, a.ldh8, 1, e)) && aligned_to(a.w, bytes) &&
           (!a.dh || rows_by(a.dh, a.lddh, esz, bytes)) && (!a.dx || rows_by(a.dx, a.lddx, esz, bytes));
  };
  const Width w = fits(16) ? W16 : fits(2 * esz) ? W2 : W1;
  int64_t rows = 0;
  cudaError_t e;
  switch (x->dtype) {
    case FLCE_F32: e = bwd<float>(a, w, rows, s); break;
    case FLCE_BF16: e = bwd<__nv_bfloat16>(a, w, rows, s); break;
    default: e = bwd<__half>(a, w, rows, s); break;
  }
  if (e != cudaSuccess || !x->dweight) return cuda_status(e);
  const unsigned blocks = (unsigned)cdiv64(H, 32);
  if (x->dweight_dtype == FLCE_F32)
    e = launch_after(k_rms_dw_sum<float>, blocks, 1024, 0, s, a.part, rows, H, (float*)x->dweight, ovw);
  else if (x->dweight_dtype == FLCE_BF16)
    e = launch_after(k_rms_dw_sum<__nv_bfloat16>, blocks, 1024, 0, s, a.part, rows, H, (__nv_bfloat16*)x->dweight, ovw);
  else
    e = launch_after(k_rms_dw_sum<__half>, blocks, 1024, 0, s, a.part, rows, H, (__half*)x->dweight, ovw);
  return cuda_status(e);
}
