// 8-bit activation checkpoints: packing, and the entry of the weight gradient that reads
// them (tensor-core kernel in flce_ckpt8_tc.cu).
//
//   q = e4m3(x / s), s = the smallest power of two with max |x| <= 448 s per row and 128 columns
//   dW[n, k] += sum_m dy[m, n] q[m, k] s[m, k / 128]
//
// Packing is bound by HBM: 2 bytes read and 1.03 written per 16-bit element. 16384 x 4096 bf16 in
// 32 us (5.3 TB/s in DRAM under ncu; floor 30). Rows of even length that allow no 16-byte accesses go
// in pairs of elements (4097 x 5122 bf16 20 us, singly 28).
#include <math.h>

#include "flce_ckpt8.cuh"

namespace flce {
namespace {

// Warp per 32 * EPV * NV columns of a row.
template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(256) k_pack(const T* __restrict__ x, int64_t ldx, int64_t N, int64_t H,
                                              uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale,
                                              int64_t nblk, int64_t wpr) {
  const int lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int64_t row = g / wpr, w = g - row * wpr;
  if (row >= N) return;
  constexpr int SPAN = NV * 32 * EPV;  // the warp's columns: whole blocks
  static_assert(SPAN % Q_BLOCK == 0, "a block belongs to one warp");
  const int64_t c0 = w * SPAN;
  const int left = (int)(H - c0 < SPAN ? H - c0 : SPAN);
  x += row * ldx + c0;
  float v[NV][EPV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * 32 + lane) * EPV;
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[j][e] = 0.0f;
    if (c < left) Vec<T, EPV>::load(x + c, v[j]);
  }
  q_row_piece<EPV, NV>(v, 0, lane, left, q + row * ldq + c0, scale + row * nblk + c0 / Q_BLOCK, 1.0f);
}

template <typename T, int EPV, int NV>
void launch_pack(const flce_ckpt8_args& a, cudaStream_t s) {
  const int64_t wpr = cdiv64(a.H, 32 * EPV * NV);
  k_pack<T, EPV, NV><<<(unsigned)cdiv64(a.N * wpr, 8), 256, 0, s>>>((const T*)a.x, a.ldx, a.N, a.H, (uint8_t*)a.q,
                                                                    a.ldq, a.scale, cdiv64(a.H, Q_BLOCK), wpr);
}

template <typename T>
cudaError_t pack(const flce_ckpt8_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  auto fits = [&](int bytes) {
    const int e = bytes / (int)sizeof(T);
    return a.H % e == 0 && rows_by(a.x, a.ldx, sizeof(T), bytes) && rows_by(a.q, a.ldq, 1, e);
  };
  if (fits(32)) launch_pack<T, 2 * W, 2>(a, s);
  else if (fits(16)) launch_pack<T, W, 2>(a, s);
  else if (fits(2 * sizeof(T))) launch_pack<T, 2, 4>(a, s);
  else launch_pack<T, 1, 4>(a, s);
  return cudaGetLastError();
}

// The product in fp32 FMAs (FLCE_FLAG_FORCE_SIMT): a block makes a 64 x 64 tile of dW, 256 threads with 4 x 4 sums each,
// 16 rows of dy and of the expanded checkpoint at a time in shared memory.
template <typename T, typename D>
__global__ void __launch_bounds__(256) k_dw_simt(const __grid_constant__ DwArgs a) {
  __shared__ __align__(16) float as[16][64], bs[16][64];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * 64, k0 = (int64_t)blockIdx.x * 64;
  float acc[4][4] = {};
  for (int64_t m0 = 0; m0 < a.M; m0 += 16) {
    for (int i = threadIdx.x; i < 16 * 64; i += 256) {
      const int64_t m = m0 + i / 64, n = n0 + i % 64, k = k0 + i % 64;
      as[i / 64][i % 64] = m < a.M && n < a.N ? to_f<T>(((const T*)a.dy)[m * a.lddy + n]) : 0.0f;
      bs[i / 64][i % 64] =
          m < a.M && k < a.K ? q_unpack2(a.q[m * a.ldq + k]).x * a.scale[m * a.nblk + k / Q_BLOCK] : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float4 av = *(const float4*)&as[m][ty * 4], bv = *(const float4*)&bs[m][tx * 4];
      const float x[4] = {av.x, av.y, av.z, av.w}, y[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (n >= a.N || k >= a.K) continue;
      D* p = (D*)a.dW + n * a.lddW + k;
      *p = from_f<D>(a.ovw ? acc[i][j] : to_f<D>(*p) + acc[i][j]);
    }
  }
}

template <typename T>
cudaError_t dw_simt(const DwArgs& a, bool f32, cudaStream_t s) {
  const dim3 grid((unsigned)cdiv64(a.K, 64), (unsigned)cdiv64(a.N, 64));
  if (f32) k_dw_simt<T, float><<<grid, 256, 0, s>>>(a);
  else k_dw_simt<T, T><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 1 && K >= 1 && M <= (1LL << 29) && N <= 65535LL * 64 && K <= 65535LL * 64;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" int32_t flce_ckpt8_pack(const flce_ckpt8_args* x, void* stream) {
  if (x == nullptr || x->N < 0 || x->H < 1 || x->N > 0x7fffffffLL || x->H > 0x7fffffffLL || !valid_dtype(x->dtype) ||
      x->flags != 0)
    return FLCE_ERR_INVALID_ARG;
  if (x->N == 0) return FLCE_OK;
  if (!x->x || !x->q || !x->scale || !aligned_to(x->x, dtype_size(x->dtype)) || !aligned_to(x->scale, 4) ||
      x->ldx < x->H || x->ldq < x->H)
    return FLCE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(pack<float>(*x, s));
    case FLCE_BF16: return cuda_status(pack<__nv_bfloat16>(*x, s));
    default: return cuda_status(pack<__half>(*x, s));
  }
}

namespace {
DwArgs dw_args(const flce_ckpt8_dw_args& x) {
  return {x.M, x.N, x.K, cdiv64(x.K, Q_BLOCK), x.dy, x.lddy, (const uint8_t*)x.q, x.ldq,
          x.scale, x.dW, x.lddW, (x.flags & FLCE_FLAG_DW_OVERWRITE) != 0};
}
}  // namespace

extern "C" size_t flce_ckpt8_dw_workspace_size(const flce_ckpt8_dw_args* x) {
  if (x == nullptr || !sizes_ok(x->M, x->N, x->K) || !valid_dtype(x->dtype)) return 0;
  if (x->M == 0 || (x->flags & FLCE_FLAG_FORCE_SIMT)) return sizeof(Ctrl);
  return dw_tc_workspace(dw_args(*x), x->dtype);
}

extern "C" int32_t flce_ckpt8_dw(const flce_ckpt8_dw_args* x, void* stream) {
  if (x == nullptr || !sizes_ok(x->M, x->N, x->K) || !valid_dtype(x->dtype)) return FLCE_ERR_INVALID_ARG;
  if ((x->flags & ~(FLCE_FLAG_DW_OVERWRITE | FLCE_FLAG_FORCE_SIMT | FLCE_FLAG_DEBUG_STALL)) != 0) return FLCE_ERR_INVALID_ARG;
  if (x->dW_dtype != FLCE_F32 && x->dW_dtype != x->dtype) return FLCE_ERR_UNSUPPORTED;
  const int esz = dtype_size(x->dtype), wsz = dtype_size(x->dW_dtype);
  if (!x->dW || !aligned_to(x->dW, wsz) || x->lddW < x->K) return FLCE_ERR_INVALID_ARG;
  if (x->status && !aligned_to(x->status, 4)) return FLCE_ERR_INVALID_ARG;
  if (x->M > 0) {
    if (!x->dy || !x->q || !x->scale || !aligned_to(x->dy, esz) || !aligned_to(x->scale, 4) || x->lddy < x->N ||
        x->ldq < x->K)
      return FLCE_ERR_INVALID_ARG;
    if (!x->workspace || !aligned_to(x->workspace, 256)) return FLCE_ERR_INVALID_ARG;
    if (x->workspace_bytes < flce_ckpt8_dw_workspace_size(x)) return FLCE_ERR_WORKSPACE;
  }
  const bool ovw = (x->flags & FLCE_FLAG_DW_OVERWRITE) != 0;
  const bool simt = (x->flags & FLCE_FLAG_FORCE_SIMT) != 0;
  if (x->M > 0 && !simt && !dw_tc_supported()) return FLCE_ERR_UNSUPPORTED;  // no tensor-map encoder in the driver
  cudaStream_t s = (cudaStream_t)stream;
  // without a status word of the caller's: the one flce_get_status reads in a workspace
  int* status = x->status ? (int*)x->status : x->M > 0 ? &((Ctrl*)x->workspace)->status : nullptr;
  cudaError_t e = cudaSuccess;
  // (the tensor-core path zeroes it itself)
  if (status && (x->M == 0 || simt)) e = cudaMemsetAsync(status, 0, sizeof(int), s);
  if (e == cudaSuccess && x->M == 0 && ovw)
    e = cudaMemset2DAsync(x->dW, (size_t)x->lddW * wsz, 0, (size_t)x->K * wsz, (size_t)x->N, s);
  if (e != cudaSuccess || x->M == 0) return cuda_status(e);
  const DwArgs a = dw_args(*x);
  if (!simt) {
    const uint32_t ms = x->wait_timeout_ms ? x->wait_timeout_ms : DEFAULT_TIMEOUT_MS;
    return cuda_status(
        launch_dw_tc8(a, x->dtype, x->dW_dtype, x->workspace, status, (uint64_t)ms * 1000000ull,
                                     (x->flags & FLCE_FLAG_DEBUG_STALL) != 0, s));
  }
  const bool f32 = x->dW_dtype == FLCE_F32;
  switch (x->dtype) {
    case FLCE_F32: return cuda_status(dw_simt<float>(a, f32, s));
    case FLCE_BF16: return cuda_status(dw_simt<__nv_bfloat16>(a, f32, s));
    default: return cuda_status(dw_simt<__half>(a, f32, s));
  }
}
