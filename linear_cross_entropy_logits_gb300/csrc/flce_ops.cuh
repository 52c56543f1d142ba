// Shared by the operators around the head (embedding, RMS norm, 8-bit checkpoints): wide
// loads and stores of row pieces, warp sums, and the 8-bit row format.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "flce_internal.cuh"

namespace flce {

// Records the error behind FLCE_ERR_CUDA for flce_last_cuda_error (flce_api.cu keeps the
// variable) and turns it into a status.
int32_t cuda_status(cudaError_t e);

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up(size_t a, size_t b) { return (a + b - 1) / b * b; }
inline bool valid_dtype(int32_t dt) { return dt == FLCE_F32 || dt == FLCE_BF16 || dt == FLCE_F16; }
inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }
// Base and pitch of a row-major matrix allow accesses of `bytes` bytes in every row.
inline bool rows_by(const void* p, int64_t ld, int esz, size_t bytes) {
  return aligned_to(p, bytes) && (size_t)ld * esz % bytes == 0;
}
inline bool rows16(const void* p, int64_t ld, int esz) { return rows_by(p, ld, esz, 16); }

// Launch of a kernel that follows another one of the same call on the stream: it may start
// while the first still runs, and waits in after_previous() for its results.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (P)args...);
}
// In the first kernel: the next one may be launched (every block has started).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// In the second: the first has finished and its writes are visible.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// EPV consecutive elements of a row as they lie in memory: 32, 16, 8 or 4 bytes in one access,
// or a single element (EPV == 1).
template <typename T, int EPV>
struct Raw {
  static constexpr int BYTES = EPV * (int)sizeof(T);
  static_assert(EPV == 1 || BYTES == 32 || BYTES == 16 || BYTES == 8 || BYTES == 4,
                "vector width");
  static constexpr int W = EPV == 1 ? 1 : BYTES / 4;
  uint32_t w[W];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (EPV == 1) {
      if constexpr (sizeof(T) == 4) w[0] = *(const uint32_t*)p;
      else w[0] = *(const uint16_t*)p;
    } else if constexpr (BYTES == 32) {
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p)
                   : "memory");
    } else if constexpr (BYTES == 4) {
      w[0] = *(const uint32_t*)p;
    } else if constexpr (BYTES == 8) {
      const uint2 u = *(const uint2*)p;
      w[0] = u.x;
      w[1] = u.y;
    } else {
      const uint4 u = *(const uint4*)p;
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (EPV == 1) {
      if constexpr (sizeof(T) == 4) *(uint32_t*)p = w[0];
      else *(uint16_t*)p = (uint16_t)w[0];
    } else if constexpr (BYTES == 32) {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else if constexpr (BYTES == 4) {
      *(uint32_t*)p = w[0];
    } else if constexpr (BYTES == 8) {
      *(uint2*)p = make_uint2(w[0], w[1]);
    } else {
      *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ float get(int e) const {  // e is a compile-time constant where it is called
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[e]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    } else {
      const __half2 h = *(const __half2*)&w[e >> 1];
      return e & 1 ? __high2float(h) : __low2float(h);
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[EPV]) const {
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = get(e);
  }
  __device__ __forceinline__ void pack(const float (&v)[EPV]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (EPV == 1) {
      const T t = from_f<T>(v[0]);
      w[0] = *(const uint16_t*)&t;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        T* h = (T*)&w[i];
        h[0] = from_f<T>(v[2 * i]);
        h[1] = from_f<T>(v[2 * i + 1]);
      }
    }
  }
};

// The same as fp32 values.
template <typename T, int EPV>
struct Vec {
  static __device__ __forceinline__ void load(const T* p, float (&v)[EPV]) {
    Raw<T, EPV> r;
    r.load(p);
    r.unpack(v);
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[EPV]) {
    Raw<T, EPV> r;
    r.pack(v);
    r.store(p);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- pairs of fp32 values, two products or sums in one instruction
typedef uint64_t f2;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_get(f2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ---- 8-bit rows: e4m3 with one scale per 128 columns ----
constexpr int Q_BLOCK = 128;
constexpr int Q_MIN_EXP = -117;  // 2^-117 times e4m3's smallest value 2^-9 is still normal in fp32 and bf16

// Exponent e of the smallest power of two 2^e >= 2^Q_MIN_EXP with amax <= 448 * 2^e; 448 =
// 1.75 * 2^8, so e = exponent(amax) - 8, one more where amax's significand is over 1.75.
__device__ __forceinline__ int q_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax > 0.0f ? (e < Q_MIN_EXP ? Q_MIN_EXP : e) : 0;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two and four e4m3 values (round to nearest even; the inputs are within +-448 or NaN).
__device__ __forceinline__ uint16_t q_pack2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t q_pack4(float a, float b, float c, float d) {
  return q_pack2(a, b) | ((uint32_t)q_pack2(c, d) << 16);
}
__device__ __forceinline__ uint8_t q_pack1(float a) {
  return (uint8_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
}
// Two e4m3 values (low 16 bits of u) as fp32; exact.
__device__ __forceinline__ float2 q_unpack2(uint32_t u) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffffu), __NV_E4M3);
  return __half22float2(*(const __half2*)&h);
}

// EPV e4m3 values as they lie in memory.
template <int EPV>
struct RawQ {
  static_assert(EPV == 8 || EPV == 4 || EPV == 2 || EPV == 1, "vector width");
  static constexpr int W = EPV < 4 ? 1 : EPV / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (EPV == 8) {
      const uint2 u = *(const uint2*)p;
      w[0] = u.x;
      w[1] = u.y;
    } else if constexpr (EPV == 4) {
      w[0] = *(const uint32_t*)p;
    } else if constexpr (EPV == 2) {
      w[0] = *(const uint16_t*)p;
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[EPV]) const {
    if constexpr (EPV == 1) {
      v[0] = q_unpack2(w[0]).x;
    } else if constexpr (EPV == 2) {
      const float2 a = q_unpack2(w[0]);
      v[0] = a.x;
      v[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 a = q_unpack2(w[i]), b = q_unpack2(w[i] >> 16);
        v[4 * i] = a.x;
        v[4 * i + 1] = a.y;
        v[4 * i + 2] = b.x;
        v[4 * i + 3] = b.y;
      }
    }
  }
};
template <int EPV>
__device__ __forceinline__ void q_store(uint8_t* p, const float (&v)[EPV]) {
  if constexpr (EPV == 16) {
    *(uint4*)p = make_uint4(q_pack4(v[0], v[1], v[2], v[3]), q_pack4(v[4], v[5], v[6], v[7]),
                            q_pack4(v[8], v[9], v[10], v[11]), q_pack4(v[12], v[13], v[14], v[15]));
  } else if constexpr (EPV == 8) {
    *(uint2*)p = make_uint2(q_pack4(v[0], v[1], v[2], v[3]), q_pack4(v[4], v[5], v[6], v[7]));
  } else if constexpr (EPV == 4) {
    *(uint32_t*)p = q_pack4(v[0], v[1], v[2], v[3]);
  } else if constexpr (EPV == 2) {
    *(uint16_t*)p = q_pack2(v[0], v[1]);
  } else {
    *p = q_pack1(v[0]);
  }
}

// A thread's vectors in one block, where a row's vectors lie as below.
template <int EPV>
constexpr int Q_VECTORS = EPV >= 4 ? 1 : Q_BLOCK / (32 * EPV);

// A row held by a group of warps: warp w of the group holds vectors (w * NV + j) * 32 + lane,
// j < NV, of EPV elements each, so that every access of a warp is contiguous and a 128-column
// block lies in 128 / EPV neighbouring lanes (EPV 16, 8, 4) or two or four vectors of a warp
// (EPV 2, 1).
// Quantises such a row piece: block maxima of |v| by shuffles, then e4m3 values to q and one
// scale per block (the power of two times `factor`) to s. A NaN takes no part in a maximum
// (fmaxf) and is stored as NaN; a warp that meets an infinity makes the maxima again without
// it and stores NaN for it (e4m3 has no infinity).
template <int EPV, int NV>
__device__ __forceinline__ void q_row_piece(const float (&v)[NV][EPV], int warp, int lane, int H, uint8_t* q,
                                            float* s, float factor) {
  constexpr int JB = Q_VECTORS<EPV>;            // vectors per block
  constexpr int LB = Q_BLOCK / (EPV * JB);      // lanes per block
  static_assert(NV % JB == 0, "a block belongs to one warp");
#pragma unroll
  for (int j0 = 0; j0 < NV; j0 += JB) {
    float m = 0.0f;
#pragma unroll
    for (int j = j0; j < j0 + JB; ++j)
#pragma unroll
      for (int e = 0; e < EPV; ++e) m = fmaxf(m, fabsf(v[j][e]));
#pragma unroll
    for (int o = LB / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bool inf = false;
    if (__any_sync(0xffffffffu, m == INFINITY)) {
      inf = true;
      m = 0.0f;
#pragma unroll
      for (int j = j0; j < j0 + JB; ++j)
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const float a = fabsf(v[j][e]);
          m = fmaxf(m, a < INFINITY ? a : 0.0f);
        }
#pragma unroll
      for (int o = LB / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const int e2 = q_exponent(m);
    const float inv = exp2_int(-e2);
    const int c0 = ((warp * NV + j0) * 32 + lane) * EPV;
#pragma unroll
    for (int j = j0; j < j0 + JB; ++j) {
      const int c = c0 + (j - j0) * 32 * EPV;
      if (c < H) {
        float o[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) o[e] = v[j][e] * inv;
        if (inf) {
#pragma unroll
          for (int e = 0; e < EPV; ++e) o[e] = fabsf(o[e]) < INFINITY ? o[e] : NAN;
        }
        q_store<EPV>(q + c, o);
      }
    }
    if ((lane & (LB - 1)) == 0 && c0 < H) s[c0 / Q_BLOCK] = exp2_int(e2) * factor;
  }
}

}  // namespace flce
