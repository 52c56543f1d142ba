// Shared by the operators around the head (embedding, RMS norm, 8-bit checkpoints): wide
// loads and stores of row pieces, warp sums, and the 8-bit row format.
#pragma once

#include <cuda_fp8.h>

#include "flce_internal.cuh"

namespace flce {

// Records the error behind FLCE_ERR_CUDA for flce_last_cuda_error (flce_api.cu keeps the
// variable) and turns it into a status.
int32_t cuda_status(cudaError_t e);

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up(size_t a, size_t b) { return (a + b - 1) / b * b; }
inline bool valid_dtype(int32_t dt) { return dt == FLCE_F32 || dt == FLCE_BF16 || dt == FLCE_F16; }
inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }
// Base and pitch of a row-major matrix allow 16-byte accesses to every row.
inline bool rows16(const void* p, int64_t ld, int esz) {
  return aligned_to(p, 16) && (size_t)ld * esz % 16 == 0;
}

// EPV consecutive elements as fp32: one 16-byte access (EPV * sizeof(T) == 16), one 8-byte
// access, or single elements (EPV == 1).
template <typename T, int EPV>
struct Vec {
  static_assert(EPV == 1 || EPV * sizeof(T) == 16, "vector width");
  static __device__ __forceinline__ void load(const T* p, float (&v)[EPV]) {
    if constexpr (EPV == 1) {
      v[0] = to_f<T>(*p);
    } else {
      const uint4 u = *(const uint4*)p;
      unpack(u, v);
    }
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[EPV]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const T* h = (const T*)&w[i];
        v[2 * i] = to_f<T>(h[0]);
        v[2 * i + 1] = to_f<T>(h[1]);
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[EPV]) {
    if constexpr (EPV == 1) {
      *p = from_f<T>(v[0]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = __float_as_uint(v[i]);
        } else {
          T* h = (T*)&w[i];
          h[0] = from_f<T>(v[2 * i]);
          h[1] = from_f<T>(v[2 * i + 1]);
        }
      }
      *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- 8-bit rows: e4m3 with one scale per 128 columns ----
constexpr int Q_BLOCK = 128;
constexpr int Q_MIN_EXP = -117;  // 2^-117 times e4m3's smallest value 2^-9 is still normal in fp32 and bf16

// The value to be stored for x: infinities become NaN (e4m3 has none).
__device__ __forceinline__ float q_input(float x) { return fabsf(x) < INFINITY ? x : NAN; }
// Its share in the block's maximum: non-finite values take no part.
__device__ __forceinline__ float q_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}
// Exponent e of the smallest power of two 2^e >= 2^Q_MIN_EXP with amax <= 448 * 2^e; 448 =
// 1.75 * 2^8, so e = exponent(amax) - 8, one more where amax's significand is over 1.75.
__device__ __forceinline__ int q_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax > 0.0f ? (e < Q_MIN_EXP ? Q_MIN_EXP : e) : 0;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two and four e4m3 values (round to nearest even; the inputs are within +-448 or NaN).
__device__ __forceinline__ uint32_t q_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint8_t q_pack1(float a) {
  return (uint8_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
}
// Two e4m3 values (low 16 bits of u) as fp32; exact.
__device__ __forceinline__ float2 q_unpack2(uint32_t u) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffffu), __NV_E4M3);
  return __half22float2(*(const __half2*)&h);
}

template <int EPV>
__device__ __forceinline__ void q_store(uint8_t* p, const float (&v)[EPV]) {
  if constexpr (EPV == 8) {
    *(uint2*)p = make_uint2(q_pack4(v[0], v[1], v[2], v[3]), q_pack4(v[4], v[5], v[6], v[7]));
  } else if constexpr (EPV == 4) {
    *(uint32_t*)p = q_pack4(v[0], v[1], v[2], v[3]);
  } else {
    *p = q_pack1(v[0]);
  }
}
template <int EPV>
__device__ __forceinline__ void q_load(const uint8_t* p, float (&v)[EPV]) {
  if constexpr (EPV == 8) {
    const uint2 u = *(const uint2*)p;
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = q_unpack2(w[i]), b = q_unpack2(w[i] >> 16);
      v[4 * i] = a.x;
      v[4 * i + 1] = a.y;
      v[4 * i + 2] = b.x;
      v[4 * i + 3] = b.y;
    }
  } else if constexpr (EPV == 4) {
    const uint32_t w = *(const uint32_t*)p;
    const float2 a = q_unpack2(w), b = q_unpack2(w >> 16);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  } else {
    v[0] = q_unpack2(*p).x;
  }
}

// A row held by a group of warps: warp w of the group holds vectors (w * NV + j) * 32 + lane,
// j < NV, of EPV elements each, so that every access of a warp is contiguous and a 128-column
// block lies in 16 lanes (EPV 8), one vector of a warp (EPV 4) or four vectors (EPV 1).
// Quantises such a row piece: block maxima of |v| by shuffles, then e4m3 values to q and one
// scale per block (the power of two times `factor`) to s. cols[j]: first column of vector j.
template <int EPV, int NV>
__device__ __forceinline__ void q_row_piece(const float (&v)[NV][EPV], int warp, int lane, int64_t H, uint8_t* q,
                                            float* s, float factor) {
  static_assert(EPV != 1 || NV % 4 == 0, "a block of single elements spans four vectors");
  constexpr int JB = EPV == 1 ? 4 : 1;      // vectors per block
  constexpr int LB = EPV == 8 ? 16 : 32;    // lanes per block
#pragma unroll
  for (int j0 = 0; j0 < NV; j0 += JB) {
    float m = 0.0f;
#pragma unroll
    for (int j = j0; j < j0 + JB; ++j)
#pragma unroll
      for (int e = 0; e < EPV; ++e) m = fmaxf(m, q_abs(v[j][e]));
#pragma unroll
    for (int o = LB / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e2 = q_exponent(m);
    const float inv = exp2_int(-e2);
    const int64_t c0 = ((int64_t)(warp * NV + j0) * 32 + lane) * EPV;
#pragma unroll
    for (int j = j0; j < j0 + JB; ++j) {
      const int64_t c = c0 + (int64_t)(j - j0) * 32 * EPV;
      if (c < H) {
        float o[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) o[e] = q_input(v[j][e]) * inv;
        q_store<EPV>(q + c, o);
      }
    }
    if ((lane & (LB - 1)) == 0 && c0 < H) s[c0 / Q_BLOCK] = exp2_int(e2) * factor;
  }
}

}  // namespace flce
