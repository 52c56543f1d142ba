// Tensor-core weight gradient from 8-bit checkpoints for sm_103a:
//
//   dW[n, k] (+)= sum_m dy[m, n] * (q[m, k] * scale[m, k / 128])
//
// The scale varies along m, the axis that is summed over, so it cannot be applied to the
// product afterwards, and dy keeps its 16 bits, so the 8-bit tensor-core formats do not apply:
// the checkpoint is expanded to dy's type on the way to the tensor cores, in shared memory,
// and never in HBM. (bf16: exact where the scales are powers of two. fp16 has fewer exponents than
// a checkpoint: a kernel in front finds the largest scale, a power of two brings that to 2^7, and
// the sums are multiplied back. Exact, then, down to 2^-22 of the largest scale.)
//
// Shape: persistent pairs of CTAs (tcgen05 cta_group::2), a pair tile of 256 (n) x 256 (k), 64
// rows m per step. Each CTA stages its 128 columns of dy (TMA, 16 KB) and its 128 columns of
// q (TMA, 8 KB: one scale block), expands q into 16 KB of bf16 / fp16 in the swizzled MN-major
// layout that the tensor cores read, and holds a 128 x 256 fp32 accumulator in its TMEM (two,
// used in turn). The copies run up to six steps ahead, the expansion up to four.
// 768 threads:
//   warp 0   TMA producer               warps 4..15   expand q
//   warp 1   MMA issuer (leader CTA)    warps 16..23  sums and output
//   warp 2   the steps' scales (cp.async)
// A step's MMAs take 512 cycles at the nominal rate and 640 at the library product's. Expanding its
// 8192 values takes about 230 instructions of each scheduler, and reading and writing them in
// shared memory 24 KB beside the 56 KB of the copies and the MMAs' operands: together as much as
// its 128 bytes a cycle carry in 640. Three groups of four warps take the steps in turn.
// 4096 x 4096 over 8192 rows, bf16 into fp32: 201 us (1370 TFLOP/s; two groups 208, without the
// expansion's reads, arithmetic and writes 173, a library bf16 product of the expanded operand
// 156). What bounds it is the expansion sharing shared memory and issue slots with the rest.
// The tensor cores truncate when they add to an accumulator; over M rows that adds up to an
// error of about M * 1.1e-9 relative (9e-6 at 8192 rows). So the accumulator is read out after
// 2048 rows and added, rounded to nearest, to fp32 sums in the registers of the output warps
// (128 x 256 sums over 256 threads); the other accumulator is filled meanwhile. 8192 x 4096 x 4096:
// bf16 6.8e-7 (every 1024 rows 3.1e-7, 208 us; every 512 1.6e-7, 220 us; a plain fp32 product
// 3.7e-7). fp16 products have three bits more to lose, 1.8e-6 with 2048 rows: it takes 1024, 8.4e-7
// (211 us, 206 with 2048; 512 rows 3.9e-7, 226 us; plain 7.9e-7), as do the terms of fp32 dy.
//
// Work split: whole tiles go round-robin over the pairs; the tiles of the last, partly filled
// wave are split along m into S parts so that they fill the pairs. Parts are left as fp32 in
// the workspace and added in part order by a second kernel (the warp that finished a tile's
// last part took 90 us to add 16 parts).
//
// fp32 dy is split into three bf16 terms d0 + d1 + d2 beforehand (8 + 8 + 8 bits: exact), which
// run as three passes over the same checkpoint rows. Where a scale is no power of two, q * scale
// has up to 24 bits too: it is split in the same way (x0 + x1 + x2, rounded to nearest) as it is
// expanded, and the products down to 2^-16 of the largest make six passes (those left out: 2^-22).
// The smallest go first, so that what their additions lose is small too. A kernel in front looks at
// the scales; the host does not wait. 8192 x 4096 x 4096: 615 us, with six passes 1250.
#include <atomic>
#include <type_traits>

#include "flce_ckpt8.cuh"
#include "flce_ptx.cuh"

namespace flce {
namespace {

using namespace ptx;

constexpr int BK = 64;                    // rows m per step
constexpr int TILE = 256;                 // pair tile, both ways
constexpr int A_BYTES = 128 * BK * 2;     // dy: 128 columns
constexpr int B_BYTES = 128 * BK * 2;     // expanded q
constexpr int Q_BYTES = 128 * BK;
constexpr int S_BYTES = BK * 4;           // the rows' scales
constexpr int STAGES = 6;                 // of dy, q and scales
constexpr int STAGE_BYTES = A_BYTES + Q_BYTES;
constexpr int SLOTS = 4;                  // of expanded q
constexpr int OFF_B = STAGES * STAGE_BYTES;
constexpr int OFF_S = OFF_B + SLOTS * B_BYTES;
constexpr int OUT_ROW = 64;               // bytes of a row that an output warp writes at a time
constexpr int OUT_BYTES = 32 * OUT_ROW;
constexpr int OFF_OUT = OFF_S + STAGES * S_BYTES;
constexpr int OFF_BARS = OFF_OUT + 8 * OUT_BYTES;
constexpr int BOX = 64 * 64 * 2;          // one 64 x 64 MN-major box
constexpr int CONV_GROUPS = 3;
constexpr int CONV_WARPS = 4 * CONV_GROUPS;
constexpr int THREADS = 128 + 32 * CONV_WARPS + 256;
constexpr int SMEM = OFF_BARS + 512 + 1024;
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(STAGES > SLOTS, "the expanding warps watch a stage's barrier for their slot");
constexpr int SEG_BF16 = 32;              // steps per accumulator for bf16 dy (2048 rows)
constexpr int SEG = 16;                   // for the others (1024 rows of a term)
constexpr int MAX_SPLIT = 16;
constexpr int SCAN_BLOCKS = 128;          // of k_scan_scales
constexpr int SCAN_LOADS = 8;             // its threads' loads in flight

// The passes of fp32 dy: d0 x2, d1 x1, d0 x1, d2 x0, d1 x0, d0 x0; where scales are powers of two the
// last three. The term of dy in pass p, four bits each:
__device__ __forceinline__ int dy_term(int p) { return 0x012010 >> (4 * p) & 3; }

struct Params {
  DwArgs d;
  int tn, tk;          // pair tiles along n and k
  int steps, mstep;    // steps in all, steps per pass over the rows (fp32 dy: three passes, or six)
  int whole;           // tiles done whole
  int S;               // parts of each other tile
  int seg;             // steps per accumulator
  float* part;         // [split tiles][S][TILE][TILE]
  const uint32_t* scan;  // what k_scan_scales found, a word per block
  int nscan;
  int* status;
  uint64_t timeout_ns;
  int access;          // bytes of an access that dW's rows allow: 16, 4 or (16-bit values) 2
  int stall;           // testing: the first step of the launch is never filled
};

// Work item i: whole tile i, or part (i - whole) % S of tile whole + (i - whole) / S.
struct Item {
  int tile, part, s0, s1;
};
__device__ __forceinline__ bool get_item(const Params& p, int steps, int i, Item& it) {
  if (i < p.whole) {
    it = {i, -1, 0, steps};
    return true;
  }
  const int j = i - p.whole, t = p.whole + j / p.S;
  if (t >= p.tn * p.tk) return false;
  const int s = j % p.S;
  it.tile = t;
  it.part = p.S > 1 ? s : -1;
  // (32 bits: 64-bit divisions took 0.5 us before the first copy; steps * S < 2^30)
  it.s0 = (int)((uint32_t)steps * (uint32_t)s / (uint32_t)p.S);
  it.s1 = (int)((uint32_t)steps * (uint32_t)(s + 1) / (uint32_t)p.S);
  return true;
}

// Whether block blk of q's row m holds a value other than zero.
__device__ __forceinline__ bool any_value(const DwArgs& d, int64_t m, int64_t blk, bool wide) {
  const uint8_t* q = d.q + m * d.ldq + blk * Q_BLOCK;
  const int n = (int)min((int64_t)Q_BLOCK, d.K - blk * Q_BLOCK);
  if (wide && n == Q_BLOCK) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < Q_BLOCK; i += 16) {
      const uint4 u = *(const uint4*)(q + i);
      any |= u.x | u.y | u.z | u.w;
    }
    return (any & 0x7f7f7f7fu) != 0;
  } else {
    for (int i = 0; i < n; ++i)
      if ((q[i] & 0x7f) != 0) return true;
  }
  return false;
}

// Looks at the scales: each block leaves, for fp16 (LARGEST), the exponent 2^(e - 127) that its largest
// finite magnitude does not pass (0 for none), else 256 where one is no power of two. The scale of a
// block of zeros says nothing about the others and is left out: a warp asks for values where its
// largest scales are, then, if there are none, where the next ones are (1 us of 1531 x 520 x 2008's
// 21.9). Zeroes the status word.
template <bool LARGEST>
__global__ void __launch_bounds__(256) k_scan_scales(const __grid_constant__ DwArgs d, bool wide, uint32_t* out, int* status) {
  __shared__ uint32_t red[8];
  let_next_start();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  constexpr int U = SCAN_LOADS;
  const int lane = threadIdx.x & 31;
  const int64_t n = d.M * d.nblk, step = (int64_t)gridDim.x * 256;
  uint32_t e = 0, odd = 0;  // e: the same in all lanes
  for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x - lane; i0 < n; i0 += U * step) {
    uint32_t b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + lane + u * step;
      b[u] = i < n ? __float_as_uint(d.scale[i]) & 0x7fffffffu : 0u;
      if (b[u] >= 0x7f800000u) b[u] = 0u;
    }
    if constexpr (LARGEST) {
#pragma unroll
      for (int u = 0; u < U; ++u) b[u] = (b[u] + 0x7fffffu) >> 23;
      for (;;) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) m = max(m, b[u]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (m <= e) break;
        int64_t i = -1;  // each lane looks at one such block at a time
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i < 0 && b[u] == m) {
            b[u] = 0u;
            i = i0 + lane + u * step;
          }
        }
        if (__any_sync(0xffffffffu, i >= 0 && any_value(d, i / d.nblk, i % d.nblk, wide))) e = m;
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) odd |= b[u] & 0x7fffffu;
    }
  }
  odd = __reduce_or_sync(0xffffffffu, odd);
  if (lane == 0) red[threadIdx.x >> 5] = e | (odd ? 256u : 0u);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      e = max(e, red[w] & 255u);
      odd |= red[w] & 256u;
    }
    out[blockIdx.x] = e | (odd ? 256u : 0u);
  }
}
// The same of all scales, for a warp.
__device__ __forceinline__ uint32_t scan_result(const Params& p, int lane) {
  uint32_t e = 0, odd = 0;
  for (int i = lane; i < p.nscan; i += 32) {
    const uint32_t v = __ldcg(p.scan + i);
    e = max(e, v & 255u);
    odd |= v & 256u;
  }
  return __reduce_max_sync(0xffffffffu, e) | __reduce_or_sync(0xffffffffu, odd);
}
// c of the power of two 2^c that fp16 values are expanded without: the largest scale becomes at
// most 2^7, its largest value 448 * 2^7 = 57344. e: what the scan found (2^-110 at least).
__device__ __forceinline__ int fp16_shift(uint32_t e) { return max((int)(e & 255u) - 127, -110) - 7; }

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four e4m3 values times a scale, as two pairs of 16-bit values (packed fp32 products). TERM: which
// of the product's bf16 terms, each the rounding of what the ones before leave.
template <typename T, int TERM = 0>
__device__ __forceinline__ uint2 expand4(uint32_t u, f2 sc2) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = q_unpack2(i ? u >> 16 : u);
    f2 v = f2_mul(f2_make(x.x, x.y), sc2);
    float lo, hi;
#pragma unroll
    for (int t = 0; t < TERM; ++t) {
      f2_get(v, lo, hi);
      const uint32_t h = pack16<__nv_bfloat16>(lo, hi);
      v = f2_fma(f2_make(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), f2_make(-1.0f, -1.0f), v);
    }
    f2_get(v, lo, hi);
    o[i] = pack16<T>(lo, hi);
  }
  return make_uint2(o[0], o[1]);
}

// A warp's 32 rows x 128 columns of sums (lane = row) and where they go in a matrix. fp32 is added
// by L2 (one add an element: nothing to wait for, and the same bits on every run). 16-bit values are
// rounded once: the sums start from them (start), so that their reads overlap the first MMAs (512 x
// 4096 x 4096 bf16 36 us; each lane its row's 43; read beside the writes 52). The sums pass
// through shared memory, 64 bytes of each row at a time, so that a store covers 64 bytes of each of
// 8 rows: stored a row per lane, 16 bytes of 32 rows at a time, the rows' pitch puts most of a
// warp's accesses on few L2 slices (28 tiles of 256 x 256 at a pitch of 16 KB took 77 us). With 128
// bytes at a time 16-bit values are 8 percent faster, fp32 the same, but the shared memory for it
// costs a stage of the copies: 10 us of the 201 over 8192 rows.
template <typename D>
struct Out {
  D* dst;        // the warp's element (0, 0)
  int64_t ld;
  int rows, cols;  // that exist, of 32 x 128
  uint32_t stage;  // the warp's shared memory: 32 rows of OUT_ROW bytes, 16-byte chunks permuted
  static constexpr int PER = 16 / sizeof(D);  // elements a chunk
  static constexpr int CH = OUT_ROW / 16;     // chunks of a row
  static constexpr int LR = 32 / CH;          // rows a warp covers at a time
  static constexpr int BLOCK = CH * PER;      // columns at a time

  // chunk c of row r: free of bank conflicts with a lane per row and with lanes along a row
  __device__ __forceinline__ uint32_t chunk(int r, int c) const {
    return stage + (uint32_t)(r * OUT_ROW + ((c ^ ((r >> 1) & 3)) << 4));
  }
  // acc = the 16-bit values that the sums are added to, zero outside: 8 rows an access, two blocks of
  // columns in flight, through shared memory.
  __device__ __forceinline__ void start(float (&acc)[128], int lane) const {
    constexpr int P = 2;  // (1 and 4: 2 to 8 percent slower)
#pragma unroll
    for (int j0 = 0; j0 < 128 / BLOCK; j0 += P) {
      uint4 u[P][CH];
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int c = (j0 + j) * BLOCK + lane % CH * PER;
        const D* p = dst + lane / CH * ld + c;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int there = lane / CH + LR * i < rows && c + PER <= cols;
          asm volatile("{.reg .pred q; setp.ne.s32 q, %5, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0; "
                       "@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                       : "=r"(u[j][i].x), "=r"(u[j][i].y), "=r"(u[j][i].z), "=r"(u[j][i].w)
                       : "l"(p), "r"(there)
                       : "memory");
          if (lane / CH + LR * i < rows && c < cols && c + PER > cols) {
            uint32_t* w = (uint32_t*)&u[j][i];
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (c + e < cols) w[e / 2] |= (uint32_t)((const uint16_t*)p)[e] << (16 * (e & 1));
          }
          p += LR * ld;
        }
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        __syncwarp();  // the block before has been read
#pragma unroll
        for (int i = 0; i < CH; ++i)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(lane / CH + LR * i, lane % CH)), "r"(u[j][i].x),
                       "r"(u[j][i].y), "r"(u[j][i].z), "r"(u[j][i].w)
                       : "memory");
        __syncwarp();
        take(acc, j0 + j, lane);
      }
    }
    __syncwarp();
  }
  // This lane's row of a block in shared memory.
  __device__ __forceinline__ void take(float (&acc)[128], int j, int lane) const {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      uint32_t u[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                   : "r"(chunk(lane, k)));
      const D* h = (const D*)u;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[j * BLOCK + k * PER + e] = to_f<D>(h[e]);
    }
  }
  // The same by accesses of A = 4 or 2 bytes, through shared memory: a pair of rows or a row at a time
  // (500 x 4096 x 4098 and x 4097 bf16 41 and 46 us, 80 with the values read beside the writes).
  template <int A>
  __device__ __forceinline__ void start_narrow(float (&acc)[128], int lane) const {
    constexpr int LPR = OUT_ROW / A, RPI = 32 / LPR;  // lanes per row, rows per access
    constexpr int B = LPR / 2;                        // accesses in flight
    const int byte = lane % LPR * A;
#pragma unroll
    for (int j = 0; j < 128 / BLOCK; ++j) {
      const int c = j * BLOCK + byte / (int)sizeof(D);
      const int left = c < cols ? rows - lane / LPR : 0;  // rows from this lane's first on
      const D* p = dst + lane / LPR * ld + c;
      __syncwarp();  // the block before has been read
#pragma unroll 1
      for (int i0 = 0; i0 < 32; i0 += B * RPI) {
        uint32_t v[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
          // (volatile: all of a batch before the first is used)
          const int there = i0 + i * RPI < left;
          if constexpr (A == 2)
            asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; mov.b32 %0, 0; @q ld.global.u16 %0, [%1];}"
                         : "=r"(v[i])
                         : "l"(p), "r"(there)
                         : "memory");
          else
            asm volatile("{.reg .pred q; setp.ne.s32 q, %2, 0; mov.b32 %0, 0; @q ld.global.u32 %0, [%1];}"
                         : "=r"(v[i])
                         : "l"(p), "r"(there)
                         : "memory");
          p += RPI * ld;
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const uint32_t at = chunk(i0 + i * RPI + lane / LPR, byte >> 4) + (byte & 15);
          if constexpr (A == 2) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)v[i]) : "memory");
          else asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v[i]) : "memory");
        }
      }
      __syncwarp();
      take(acc, j, lane);
    }
    __syncwarp();
  }
  // The matrix = acc by accesses of A bytes; with !ovw and fp32, += acc.
  template <bool ovw, int A>
  __device__ __forceinline__ void put(const float (&acc)[128], int lane) const {
#pragma unroll
    for (int j = 0; j < 128 / BLOCK; ++j) {
      if (j * BLOCK >= cols) break;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint4 u;
        const float* v = &acc[j * BLOCK + c * PER];
        if constexpr (sizeof(D) == 4) {
          u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            D* h = (D*)&o[e];
            h[0] = from_f<D>(v[2 * e]);
            h[1] = from_f<D>(v[2 * e + 1]);
          }
          u = make_uint4(o[0], o[1], o[2], o[3]);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(lane, c)), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
                     : "memory");
      }
      __syncwarp();
      if constexpr (A < 16) {
        constexpr int LPR = OUT_ROW / A, RPI = 32 / LPR;
        const int byte = lane % LPR * A, c = j * BLOCK + byte / (int)sizeof(D);
        const int left = c < cols ? rows - lane / LPR : 0;  // rows from this lane's first on
        D* p = dst + lane / LPR * ld + c;
        constexpr int B = 8;
#pragma unroll 1
        for (int i0 = 0; i0 < LPR; i0 += B) {
          uint32_t v[B];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const uint32_t at = chunk((i0 + i) * RPI + lane / LPR, byte >> 4) + (byte & 15);
            if constexpr (A == 2) {
              uint16_t u;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at));
              v[i] = u;
            } else {
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i]) : "r"(at));
            }
          }
#pragma unroll
          for (int i = 0; i < B; ++i) {
            if ((i0 + i) * RPI < left) {
              if constexpr (A == 2) *(uint16_t*)p = (uint16_t)v[i];
              else if constexpr (ovw) *(uint32_t*)p = v[i];
              else atomicAdd((float*)p, __uint_as_float(v[i]));
            }
            p += RPI * ld;
          }
        }
        continue;
      }
      const int c = j * BLOCK + (lane % CH) * PER;
      D* p = dst + lane / CH * ld + c;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int r = lane / CH + LR * i;
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(chunk(r, lane % CH)));
        if (r < rows && c < cols) {
          if (c + PER <= cols) {
            if constexpr (ovw)
              *(uint4*)p = u;
            else
              asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p),
                           "f"(__uint_as_float(u.x)), "f"(__uint_as_float(u.y)), "f"(__uint_as_float(u.z)),
                           "f"(__uint_as_float(u.w))
                           : "memory");
          } else {
            const D* h = (const D*)&u;
#pragma unroll
            for (int e = 0; e < PER - 1; ++e)
              if (c + e < cols) {
                if constexpr (ovw) p[e] = h[e];
                else atomicAdd(p + e, h[e]);
              }
          }
        }
        p += LR * ld;
      }
    }
    __syncwarp();
  }
};

// F32: dy is staged in three terms, and the scales decide the passes.
template <typename T, typename D, bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    k_dw_tc8(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_q,
             const __grid_constant__ Params p) {
  constexpr bool F16 = std::is_same<T, __half>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(smem + OFF_BARS);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };                    // this CTA's dy and q
  auto full_s = [&](int s) { return bar0 + 8u * (STAGES + s); };       // and its scales
  auto empty = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };    // MMAs done with the stage (and its slot)
  auto conv = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };     // dy there and q expanded, both CTAs (leader)
  auto tfull = [&](int s) { return bar0 + 8u * (3 * STAGES + SLOTS + s); };       // accumulator filled
  auto tempty = [&](int s) { return bar0 + 8u * (3 * STAGES + SLOTS + 2 + s); };  // and read out (leader)
  const uint32_t drain = bar0 + 8u * (3 * STAGES + SLOTS + 4);
  constexpr int NBARS = 3 * STAGES + SLOTS + 5;
  static_assert(NBARS * 8 + 8 + STAGES * 4 <= 512, "barrier block");
  uint32_t* tmem_slot = (uint32_t*)(bars + NBARS);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  int* copies = (int*)(tmem_slot + 2);  // per stage: phases this CTA's producer filled

  const uint32_t rank = cta_rank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Abort ab{abort_flag, mapa(smem_u32((const void*)abort_flag), rank ^ 1u), p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      bar_init(full(s), 1);
      bar_init(full_s(s), 32);
      bar_init(empty(s), 1);
      copies[s] = 0;
    }
    for (int s = 0; s < SLOTS; ++s) bar_init(conv(s), 8);  // four warps of each CTA
    for (int s = 0; s < 2; ++s) {
      bar_init(tfull(s), 1);
      bar_init(tempty(s), 16);  // eight warps of each CTA
    }
    bar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&tm_dy);
    prefetch_map(&tm_q);
  }
  let_next_start();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_before();
  cluster_sync();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  after_previous();  // staged operands are there, and the scales have been looked at
  int steps = p.steps, pass0 = 3;
  if constexpr (F32) {
    if (scan_result(p, lane) & 256u) steps *= 2, pass0 = 0;
  }

  // Registers: 80 a thread at launch (6 warpgroups: 480 in all) = 32 + 3 * 48 + 2 * 152.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer, both CTAs
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      Item it;
      for (int i = pair; ok && get_item(p, steps, i, it); i += npairs) {
        const int n0 = it.tile / p.tk * TILE + (int)rank * 128, k0 = it.tile % p.tk * TILE + (int)rank * 128;
        int row = it.s0 % p.mstep;  // step within a pass
        int pass = pass0 + it.s0 / p.mstep;
        for (int st = it.s0; st < it.s1; ++st) {
          if (!bar_wait(empty(s), ph ^ 1u, ab, true)) {
            ok = false;
            break;
          }
          bar_expect(full(s), A_BYTES + Q_BYTES);
          const uint32_t a = smem_u32(smem + s * STAGE_BYTES);
          if (!(p.stall && leader && i == 0 && st == it.s0)) {
            tma_load(a + A_BYTES, &tm_q, full(s), k0, row * BK);
            const int m = (F32 ? dy_term(pass) * p.mstep + row : st) * BK;
            tma_load(a, &tm_dy, full(s), n0, m);
            tma_load(a + BOX, &tm_dy, full(s), n0 + 64, m);
          }
          if (++row == p.mstep) {
            row = 0;
            ++pass;
          }
          copies[s] += 1;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && leader) {
      // ---------------- MMA issuer
      constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      // kind::f16, fp32 accumulator, both operands MN-major, N = 256, M = 256
      constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | (1u << 16) |
                                 ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
      const uint64_t desc0 = desc_mn(smem_u32(smem), BOX);  // the address counts 16 bytes from bit 0
      int s = 0, b = 0, g = 0;
      uint32_t bph = 0;
      bool ok = true, ready = false;
      Item it;
      for (int i = pair; ok && get_item(p, steps, i, it); i += npairs) {
        for (int st = it.s0; ok && st < it.s1; ++g) {
          const int as = g & 1;
          if (!bar_wait(tempty(as), ((uint32_t)(g >> 1) & 1u) ^ 1u, ab, true)) {
            ok = false;
            break;
          }
          tc_after();
          const int end = min(st + p.seg, it.s1);
          for (bool first = true; st < end; ++st, first = false) {
            if (!ready && !bar_wait(conv(b), bph, ab, true)) {
              ok = false;
              break;
            }
            tc_after();
            // look at the next step's barrier while this step's MMAs are issued: the pipe holds
            // few of them, and a wait between two steps leaves it idle
            const int nb = b + 1 == SLOTS ? 0 : b + 1;
            ready = bar_test(conv(nb), b + 1 == SLOTS ? bph ^ 1u : bph);
            const uint64_t da = desc0 + (uint32_t)(s * (STAGE_BYTES >> 4));
            const uint64_t db = desc0 + (uint32_t)((OFF_B + b * B_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              mma_pair(tmem + (uint32_t)(as * TILE), da + (uint64_t)(k * (2048 >> 4)), db + (uint64_t)(k * (2048 >> 4)),
                       idesc, !first || k != 0);
            mma_commit_pair(empty(s));
            if (++s == STAGES) s = 0;
            if (++b == SLOTS) {
              b = 0;
              bph ^= 1u;
            }
          }
          if (ok) mma_commit_pair(tfull(as));
        }
      }
      // every MMA issued completes before TMEM is freed or shared memory released
      mma_commit_local(drain);
      bar_wait(drain, 0u, ab, false);
    } else if (warp == 2) {
      // ---------------- scales of a step's 64 rows, that of row 16 j + r at 4 r + j
      const uint32_t dst = smem_u32(smem + OFF_S) + (uint32_t)((lane & 15) * 4 + (lane >> 4)) * 4;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      Item it;
      for (int i = pair; ok && get_item(p, steps, i, it); i += npairs) {
        const int blk = it.tile % p.tk * 2 + (int)rank;  // this CTA's 128 columns: one scale block
        const float* sp = p.d.scale + (blk < p.d.nblk ? blk : 0);
        int row = it.s0 % p.mstep;  // step within a pass
        for (int st = it.s0; st < it.s1; ++st) {
          ok = __all_sync(0xffffffffu, bar_wait(empty(s), ph ^ 1u, ab, true));
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t m = (int64_t)row * BK + h * 32 + lane;
            const bool in = blk < p.d.nblk && m < p.d.M;
            cp_async4(dst + (uint32_t)(s * S_BYTES + h * 8), sp + (in ? m * p.d.nblk : 0), in);
          }
          bar_arrive_cp_async(full_s(s));
          if (++row == p.mstep) row = 0;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      cp_async_wait_all();
    }
  } else if (warp < 4 + CONV_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    // ---------------- expand q: groups of four warps take the steps in turn, so a step's
    // expansion may last as many steps; thread (r, c) takes bytes 16c .. 16c + 15 of rows r + 16 j.
    // Threads of columns 64.. take the neighbouring row, so that eight threads' reads (64 bytes of
    // each of two rows) and writes (every other 16-byte chunk of two rows) hit distinct banks
    const int group = (warp - 4) >> 2;
    const int shift = F16 ? fp16_shift(scan_result(p, lane)) : 0;
    const float unit = exp2_int(-shift);
    const float most = exp2_int(shift + 7);  // (2^128: an infinity)
    const int terms_end = pass0 == 0 ? 3 * p.mstep : 0;  // steps before it take x2 (one pass) or x1 (two)
    const int t = threadIdx.x & 127;
    const int c = t & 7, r = (t >> 3) ^ (c >> 2);
    const uint32_t out = (uint32_t)(c >> 2) * BOX + (uint32_t)r * 128;
    const uint32_t chunk = (uint32_t)((2 * (c & 3)) ^ (r & 7)) << 4;  // of bytes 16c ..; its neighbour's: ^ 16
    int s = 0, b = 0, turn = 0, whose = 0;
    uint32_t ph = 0;
    bool ok = true;
    Item it;
    for (int i = pair; ok && get_item(p, steps, i, it); i += npairs) {
      for (int st = it.s0; st < it.s1; ++st, ++turn) {
        if (whose == group) {
          ok = bar_wait(full(s), ph, ab, true) && bar_wait(full_s(s), ph, ab, true);
          if (ok && turn >= SLOTS) {
            // the slot's last user, SLOTS steps back, was in stage s - SLOTS (this pass's or,
            // below 0, the pass before's)
            const int u = s - SLOTS;
            ok = bar_wait(empty(u < 0 ? u + STAGES : u), u < 0 ? ph ^ 1u : ph, ab, true);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* q = smem + s * STAGE_BYTES + A_BYTES + r * 128 + c * 16;
          uint8_t* o = smem + OFF_B + b * B_BYTES + out;
          const float4 sc4 = *(const float4*)(smem + OFF_S + s * S_BYTES + r * 16);
          float sc[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
          if constexpr (F16) {
            // larger finite scales are of blocks of zeros: as infinities they would make them NaN
            if (fmaxf(fmaxf(fabsf(sc[0]), fabsf(sc[1])), fmaxf(fabsf(sc[2]), fabsf(sc[3]))) > most) {
#pragma unroll
              for (int j = 0; j < 4; ++j) sc[j] = fabsf(sc[j]) > most && fabsf(sc[j]) < INFINITY ? 0.0f : sc[j];
            }
          }
          uint4 u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = *(const uint4*)(q + j * 2048);
          auto expand = [&](auto term) {
            constexpr int TERM = decltype(term)::value;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = F16 ? sc[j] * unit : sc[j];
              const f2 sc2 = f2_make(f, f);
              const uint2 x0 = expand4<T, TERM>(u[j].x, sc2), x1 = expand4<T, TERM>(u[j].y, sc2);
              const uint2 x2 = expand4<T, TERM>(u[j].z, sc2), x3 = expand4<T, TERM>(u[j].w, sc2);
              *(uint4*)(o + j * 2048 + chunk) = make_uint4(x0.x, x0.y, x1.x, x1.y);
              *(uint4*)(o + j * 2048 + (chunk ^ 16)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
            }
          };
          if (!F32 || st >= terms_end) expand(std::integral_constant<int, 0>());
          else if (st >= p.mstep) expand(std::integral_constant<int, 1>());
          else expand(std::integral_constant<int, 2>());
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(mapa(conv(b), 0));
        }
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
        if (++b == SLOTS) b = 0;
        if (++whose == CONV_GROUPS) whose = 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    // ---------------- sums and output: warp w has rows 32 (w % 4) .. of this CTA's 128 and
    // columns 128 h .. of the tile's 256
    const int w = warp - 4 - CONV_WARPS, quad = warp & 3, h = w >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(h * 128);
    const uint32_t stage = smem_u32(smem + OFF_OUT + w * OUT_BYTES);
    const float unit = F16 ? exp2_int(fp16_shift(scan_result(p, lane))) : 1.0f;
    int g = 0;
    bool ok = true;
    Item it;
    // (a pair that gave up writes NaN to the tiles that it has not finished: nobody may look at the
    // status word)
    for (int i = pair; get_item(p, steps, i, it); i += npairs) {
      const int row = (int)rank * 128 + quad * 32, col = h * 128;  // within the tile
      const int64_t n = (int64_t)(it.tile / p.tk) * TILE + row, k = (int64_t)(it.tile % p.tk) * TILE + col;
      const Out<D> out{(D*)p.d.dW + n * p.d.lddW + k, p.d.lddW, (int)min(p.d.N - n, (int64_t)32),
                       (int)min(p.d.K - k, (int64_t)128), stage};
      float acc[128];
      if (sizeof(D) == 2 && it.part < 0 && !p.d.ovw && ok) {
        if (p.access == 16) out.start(acc, lane);
        else if (p.access == 4) out.template start_narrow<4>(acc, lane);
        else out.template start_narrow<2>(acc, lane);
      } else {
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      }
      for (int st = it.s0; ok && st < it.s1; st += p.seg, ++g) {
        const int as = g & 1;
        ok = __all_sync(0xffffffffu, bar_wait(tfull(as), (uint32_t)(g >> 1) & 1u, ab, true));
        if (!ok) break;
        tc_after();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t r[16];
          tmem_ld16(taddr + (uint32_t)(as * TILE + j * 16), r);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v = __uint_as_float(r[e]);
            acc[j * 16 + e] = F16 ? fmaf(v, unit, acc[j * 16 + e]) : acc[j * 16 + e] + v;
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(mapa(tempty(as), 0));
      }
      if (!ok) {
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = NAN;
      }
      if (it.part >= 0) {
        const int64_t slot = (int64_t)(it.tile - p.whole) * p.S + it.part;
        const Out<float> part{p.part + slot * TILE * TILE + row * TILE + col, TILE, 32, 128, stage};
        part.put<true, 16>(acc, lane);
      } else if constexpr (sizeof(D) == 4) {
        if (p.access == 16) {
          if (p.d.ovw) out.template put<true, 16>(acc, lane);
          else out.template put<false, 16>(acc, lane);
        } else {
          if (p.d.ovw) out.template put<true, 4>(acc, lane);
          else out.template put<false, 4>(acc, lane);
        }
      } else {  // (with !ovw acc has the old values)
        if (p.access == 16) out.template put<true, 16>(acc, lane);
        else if (p.access == 4) out.template put<true, 4>(acc, lane);
        else out.template put<true, 2>(acc, lane);
      }
    }
  }

  // ---------------- teardown
  __syncwarp();
  tc_before();
  cluster_sync();  // no role of either CTA issues anything after this point
  if (threadIdx.x == 0 && *abort_flag) {
    // every copy issued lands before shared memory is released; without an abort all were waited for
    for (int s = 0; s < STAGES; ++s)
      if (copies[s] > 0) bar_wait(full(s), (uint32_t)(copies[s] - 1) & 1u, ab, false);
  }
  cluster_sync();
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Adds up the parts of the split tiles in part order: a thread has four columns of a row, a block
// (x, y) 8 rows from 8 y on of split tile x.
template <typename D>
__global__ void __launch_bounds__(512) k_dw_join(const __grid_constant__ Params p) {
  after_previous();
  const int tile = p.whole + (int)blockIdx.x;
  const int r = (int)blockIdx.y * 8 + (threadIdx.x >> 6), c = (threadIdx.x & 63) * 4;
  const int64_t n = (int64_t)(tile / p.tk) * TILE + r, k = (int64_t)(tile % p.tk) * TILE + c;
  if (n >= p.d.N || k >= p.d.K) return;
  const float* q = p.part + (int64_t)blockIdx.x * p.S * TILE * TILE + r * TILE + c;
  float t[4] = {};
#pragma unroll 4
  for (int s = 0; s < p.S; ++s, q += TILE * TILE) {
    const float4 v = *(const float4*)q;
    t[0] += v.x;
    t[1] += v.y;
    t[2] += v.z;
    t[3] += v.w;
  }
  D* o = (D*)p.d.dW + n * p.d.lddW + k;
  if (p.access == 16 && k + 4 <= p.d.K) {
    if constexpr (sizeof(D) == 4) {
      float4 v = p.d.ovw ? make_float4(0.f, 0.f, 0.f, 0.f) : *(float4*)o;
      *(float4*)o = make_float4(v.x + t[0], v.y + t[1], v.z + t[2], v.w + t[3]);
    } else {
      uint2 u = p.d.ovw ? make_uint2(0u, 0u) : *(uint2*)o;
      D* h = (D*)&u;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = from_f<D>(p.d.ovw ? t[i] : to_f<D>(h[i]) + t[i]);
      *(uint2*)o = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < p.d.K) o[i] = from_f<D>(p.d.ovw ? t[i] : to_f<D>(o[i]) + t[i]);
  }
}

// ------------------------------------------------------------------ staging
// dy rows that TMA cannot read in place (fp32, or a pitch that is no multiple of 16 bytes):
// copied to a 16-byte pitch; fp32 as three bf16 terms in planes of `rows` rows, each the
// leading 8 bits of what the ones before leave. Rows past M are zero. Four columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) k_stage_dy(const T* dy, int64_t lddy, int64_t M, int64_t N,
                                                  int64_t rows, void* out, int64_t ld, int vec) {
  let_next_start();
  const int64_t m = blockIdx.x, n = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
  if (n >= N) return;
  if constexpr (sizeof(T) == 4) {
    float x[4] = {};
    if (m < M) {
      const float* p = dy + m * lddy + n;
      if (vec && n + 4 <= N) {
        const float4 v = *(const float4*)p;
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) x[e] = p[e];
      }
    }
    // the pitch is a multiple of 8 columns: four are always there
    uint2* o = (uint2*)((uint16_t*)out + m * ld + n);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      uint32_t t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t hi = __float_as_uint(x[e]) & 0xffff0000u;
        const bool fin = fabsf(x[e]) < INFINITY;
        // a NaN whose set bits lie in the low half must not become an infinity
        t[e] = fin || x[e] == x[e] ? hi : 0x7fc00000u;
        x[e] = fin ? x[e] - __uint_as_float(hi) : 0.0f;
      }
      *(uint2*)((uint16_t*)o + i * rows * ld) = make_uint2(t[0] >> 16 | t[1], t[2] >> 16 | t[3]);
    }
  } else {
    const uint16_t* p = (const uint16_t*)dy + m * lddy + n;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = n + e < N ? p[e] : 0u;
    *(uint2*)((uint16_t*)out + m * ld + n) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
  after_previous();  // the next kernel waits for this one alone, and reads what the scan leaves too
}
__global__ void __launch_bounds__(256) k_stage_q(const uint8_t* __restrict__ q, int64_t ldq, int64_t K, uint8_t* out,
                                                 int64_t ld) {
  let_next_start();
  const int64_t m = blockIdx.x, k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
  if (k >= K) return;
  uint32_t w = 0;  // (the pitch is a multiple of 16)
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (k + e < K) w |= (uint32_t)q[m * ldq + k + e] << (8 * e);
  *(uint32_t*)(out + m * ld + k) = w;
}

// ------------------------------------------------------------------ plan
struct Plan8 {
  int tn, tk, steps, mstep, whole, S;
  size_t off_scan, off_part, off_dy, off_q, total;
};

// Rows that TMA cannot read in place.
bool stage_dy(const DwArgs& a, int dt) { return dt == FLCE_F32 || !rows16(a.dy, a.lddy, 2); }
// Whether the kernel needs to know the scales' range.
bool dw_tc_scans(int dt) { return dt != FLCE_BF16; }
bool stage_q(const DwArgs& a) { return !rows16(a.q, a.ldq, 1); }

// Whole tiles fill whole waves of pairs; the rest are split S ways, S minimising the steps of
// the remaining waves plus the cost of the parts in steps' time (0.34 us): the second kernel 9,
// writing and reading a part's 256 KB 0.3.
Plan8 plan(const DwArgs& a, int dt) {
  const int64_t M = a.M, N = a.N, K = a.K;
  const int pairs = num_sms() / 2;
  Plan8 p = {};
  p.tn = (int)cdiv64(N, TILE);
  p.tk = (int)cdiv64(K, TILE);
  p.mstep = (int)cdiv64(M, BK);
  const int terms = dt == FLCE_F32 ? 3 : 1;
  p.steps = terms * p.mstep;
  const int64_t tiles = (int64_t)p.tn * p.tk;
  p.whole = (int)(tiles / pairs * pairs);
  const int64_t rest = tiles - p.whole;
  p.S = 1;
  if (rest > 0) {
    double best = 0.0;
    for (int S = 1; S <= MAX_SPLIT && S <= p.steps; ++S) {
      const double waves = (double)cdiv64(rest * S, pairs) * (double)cdiv64(p.steps, S);
      const double cost = waves + (S > 1 ? 9.0 + 0.3 * (double)(rest * S) : 0.0);
      if (S == 1 || cost < best) {
        best = cost;
        p.S = S;
      }
    }
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = round_up(off + bytes, 256);
    return o;
  };
  const size_t split = p.S > 1 ? (size_t)rest : 0;
  take(256);  // the status word (Ctrl::status)
  p.off_scan = take(dw_tc_scans(dt) ? SCAN_BLOCKS * 4 : 0);
  p.off_part = take(split * p.S * TILE * TILE * 4);
  p.off_dy = take(stage_dy(a, dt) ? (size_t)terms * p.mstep * BK * round_up((size_t)N, 8) * 2 : 0);
  p.off_q = take(stage_q(a) ? (size_t)M * round_up((size_t)K, 16) : 0);
  p.total = off;
  return p;
}

template <typename T, typename D, bool F32>
cudaError_t launch(const CUtensorMap& A, const CUtensorMap& Q, const Params& p, int64_t items, bool behind,
                   cudaStream_t s) {
  auto kern = k_dw_tc8<T, D, F32>;
  // per-device cache of the pairs that fit at once; concurrent first launches may both set it
  static std::atomic<int> fit[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it starts up beside the kernel in front
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = fit[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (unsigned)(num_sms() / 2), 1, 1);
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    fit[dev].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(2 * (unsigned)(items < n ? items : n), 1, 1);
  cfg.numAttrs = behind ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, A, Q, p);
  if (e != cudaSuccess || p.S == 1) return e;
  const int64_t split = (int64_t)p.tn * p.tk - p.whole;
  return launch_after(k_dw_join<D>, dim3((unsigned)split, TILE / 8, 1), 512, 0, s, p);
}

}  // namespace

bool dw_tc_supported() { return ptx::encode_fn() != nullptr; }

size_t dw_tc_workspace(const DwArgs& a, int dt) { return plan(a, dt).total; }

cudaError_t launch_dw_tc8(const DwArgs& a, int dt, int wdt, void* workspace, int* status, uint64_t timeout_ns,
                          bool stall, cudaStream_t s) {
  const Plan8 pl = plan(a, dt);
  char* ws = (char*)workspace;
  Params p = {};
  p.d = a;
  p.tn = pl.tn;
  p.tk = pl.tk;
  p.steps = pl.steps;
  p.mstep = pl.mstep;
  p.whole = pl.whole;
  p.S = pl.S;
  p.seg = dt == FLCE_BF16 ? SEG_BF16 : SEG;
  p.part = (float*)(ws + pl.off_part);
  p.scan = (const uint32_t*)(ws + pl.off_scan);
  p.status = status;
  p.timeout_ns = timeout_ns;
  p.stall = stall;
  const int wsz = dtype_size(wdt);
  p.access = rows16(a.dW, a.lddW, wsz) ? 16 : wsz == 4 || (a.K % 2 == 0 && rows_by(a.dW, a.lddW, wsz, 4)) ? 4 : 2;
  cudaError_t e;
  if (dw_tc_scans(dt)) {
    const int64_t n = a.M * a.nblk, most = cdiv64(n, 256 * SCAN_LOADS);
    p.nscan = (int)(most < SCAN_BLOCKS ? most : SCAN_BLOCKS);
    auto scan = dt == FLCE_F16 ? k_scan_scales<true> : k_scan_scales<false>;
    scan<<<(unsigned)p.nscan, 256, 0, s>>>(a, rows16(a.q, a.ldq, 1), (uint32_t*)(ws + pl.off_scan), status);
    e = cudaGetLastError();
  } else {
    e = cudaMemsetAsync(status, 0, sizeof(int), s);
  }
  if (e != cudaSuccess) return e;

  const void* dy = a.dy;
  int64_t lddy = a.lddy, rows = a.M;
  if (stage_dy(a, dt)) {
    dy = ws + pl.off_dy;
    lddy = (int64_t)round_up((size_t)a.N, 8);
    const int64_t plane = (int64_t)pl.mstep * BK;
    const dim3 grid((unsigned)(dt == FLCE_F32 ? plane : a.M), (unsigned)cdiv64(a.N, 1024));
    if (dt == FLCE_F32) {
      // (beside the scan: fp32 1531 x 520 x 2008 31 us, 33 one after the other)
      e = launch_after(k_stage_dy<float>, grid, 256, 0, s, a.dy, a.lddy, a.M, a.N, plane, (void*)dy, lddy,
                       (int)rows16(a.dy, a.lddy, 4));
      rows = 3 * plane;
    } else {
      k_stage_dy<__half><<<grid, 256, 0, s>>>((const __half*)a.dy, a.lddy, a.M, a.N, plane, (void*)dy, lddy, 0);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  const uint8_t* q = a.q;
  int64_t ldq = a.ldq;
  if (stage_q(a)) {
    q = (const uint8_t*)(ws + pl.off_q);
    ldq = (int64_t)round_up((size_t)a.K, 16);
    k_stage_q<<<dim3((unsigned)a.M, (unsigned)cdiv64(a.K, 1024)), 256, 0, s>>>(a.q, a.ldq, a.K, (uint8_t*)q, ldq);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  CUtensorMap A, Q;
  const auto ty = dt == FLCE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!ptx::encode_2d(&A, ty, dy, a.N, rows, lddy * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !ptx::encode_2d(&Q, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, a.K, a.M, ldq, 128, BK, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int64_t items = p.whole + ((int64_t)p.tn * p.tk - p.whole) * p.S;
  const bool behind = dw_tc_scans(dt) || stage_dy(a, dt) || stage_q(a);  // another kernel of this call
  if (dt == FLCE_F16)
    return wdt == FLCE_F32 ? launch<__half, float, false>(A, Q, p, items, behind, s)
                           : launch<__half, __half, false>(A, Q, p, items, behind, s);
  if (dt == FLCE_F32) return launch<__nv_bfloat16, float, true>(A, Q, p, items, behind, s);
  if (wdt == FLCE_F32) return launch<__nv_bfloat16, float, false>(A, Q, p, items, behind, s);
  return launch<__nv_bfloat16, __nv_bfloat16, false>(A, Q, p, items, behind, s);
}

}  // namespace flce
