// Tensor-core weight gradient from 8-bit checkpoints for sm_103a:
//
//   dW[n, k] (+)= sum_m dy[m, n] * (q[m, k] * scale[m, k / 128])
//
// The scale varies along m, the axis that is summed over, so it cannot be applied to the
// product afterwards, and dy keeps its 16 bits, so the 8-bit tensor-core formats do not apply:
// the checkpoint is expanded to dy's type on the way to the tensor cores, in shared memory,
// and never in HBM. (bf16: exact where the scales are powers of two.)
//
// Shape: persistent pairs of CTAs (tcgen05 cta_group::2), a pair tile of 256 (n) x 256 (k), 64
// rows m per step. Each CTA stages its 128 columns of dy (TMA, 16 KB) and its 128 columns of
// q (TMA, 8 KB: one scale block), expands q into 16 KB of bf16 / fp16 in the swizzled MN-major
// layout that the tensor cores read, and holds a 128 x 256 fp32 accumulator in its TMEM (two,
// used in turn). The copies run up to six steps ahead, the expansion up to four.
// 640 threads:
//   warp 0   TMA producer               warps 4..11   expand q
//   warp 1   MMA issuer (leader CTA)    warps 12..19  sums and output
//   warp 2   the steps' scales (cp.async)
// A step's MMAs take 512 cycles; expanding 8192 values takes about 230 instructions of each of
// the eight warps (two per scheduler).
// The tensor cores truncate when they add to an accumulator; over M rows that adds up to an
// error of about M * 1.1e-9 relative (9e-6 at 8192 rows). So the accumulator is read out after
// every SEGMENT of rows and added, rounded to nearest, to fp32 sums in the registers of the
// output warps (128 x 256 sums over 256 threads); the other accumulator is filled meanwhile.
//
// Work split: whole tiles go round-robin over the pairs; the tiles of the last, partly filled
// wave are split along m into S parts so that they fill the pairs. Parts are left as fp32 in
// the workspace, and whichever warp finishes a tile's last part adds them up in part order
// (the same order whoever is last, so the same bits) and writes dW.
//
// fp32 dy is split into three bf16 terms beforehand (8 + 8 + 8 bits: exact), which run as
// three passes over the same checkpoint rows.
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
constexpr int OFF_BARS = OFF_S + STAGES * S_BYTES;
constexpr int BOX = 64 * 64 * 2;          // one 64 x 64 MN-major box
constexpr int THREADS = 640;
constexpr int CONV_WARPS = 8;
constexpr int SMEM = OFF_BARS + 512 + 1024;
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(STAGES > SLOTS, "the expanding warps watch a stage's barrier for their slot");
constexpr int SEG16 = 32;                 // steps per accumulator for 16-bit dy (2048 rows)
constexpr int SEG32 = 8;                  // for fp32 dy: its results are held to fp32 accuracy
constexpr int MAX_SPLIT = 16;
constexpr int PART_FLOATS = 32 * 128;     // sums of one output warp

struct Params {
  DwArgs d;
  int tn, tk;          // pair tiles along n and k
  int steps, mstep;    // steps in all, steps per term of dy (steps = terms * mstep)
  int whole;           // tiles done whole
  int S;               // parts of each other tile
  int seg;             // steps per accumulator
  float* part;         // [split tiles][S][2 CTAs][8 warps][PART_FLOATS]
  int* count;          // [split tiles][2][8] parts finished, zeroed before the launch
  int* status;
  uint64_t timeout_ns;
  int vec;             // dW rows allow 16-byte accesses
};

// Work item i: whole tile i, or part (i - whole) % S of tile whole + (i - whole) / S.
struct Item {
  int tile, part, s0, s1;
};
__device__ __forceinline__ bool get_item(const Params& p, int i, Item& it) {
  if (i < p.whole) {
    it = {i, -1, 0, p.steps};
    return true;
  }
  const int j = i - p.whole, t = p.whole + j / p.S;
  if (t >= p.tn * p.tk) return false;
  const int s = j % p.S;
  it.tile = t;
  it.part = p.S > 1 ? s : -1;
  it.s0 = (int)((int64_t)p.steps * s / p.S);
  it.s1 = (int)((int64_t)p.steps * (s + 1) / p.S);
  return true;
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four e4m3 values times a scale, as two pairs of 16-bit values (packed fp32 products).
template <typename T>
__device__ __forceinline__ uint2 expand4(uint32_t u, uint64_t sc2) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = q_unpack2(i ? u >> 16 : u);
    uint64_t a;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(sc2));
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
    o[i] = pack16<T>(lo, hi);
  }
  return make_uint2(o[0], o[1]);
}

// 16 columns of a row of dW, from p on, of which `left` exist, (+)= v; the loads go out
// together.
template <typename D>
__device__ __forceinline__ void put16(D* p, int64_t left, const float* v, int vec, int ovw) {
  if (vec && left >= 16) {
    constexpr int E = 16 / sizeof(D), NQ = 16 / E;  // elements per 16 bytes, and their number
    Raw<D, E> u[NQ];
    if (!ovw) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) u[i].load(p + i * E);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = v[i * E + e];
      if (!ovw) {
        float old[E];
        u[i].unpack(old);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += old[e];
      }
      Vec<D, E>::store(p + i * E, o);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) p[i] = from_f<D>(ovw ? v[i] : to_f<D>(p[i]) + v[i]);
}

template <typename T, typename D>
__global__ void __launch_bounds__(THREADS, 1)
    k_dw_tc8(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_q,
             const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(smem + OFF_BARS);
  const uint32_t bar0 = smem_u32(bars);
  auto full_a = [&](int s) { return bar0 + 8u * s; };                  // both CTAs' dy (leader)
  auto full_q = [&](int s) { return bar0 + 8u * (STAGES + s); };       // this CTA's q
  auto full_s = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };   // and its scales
  auto empty_a = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };  // MMAs done with the stage (and its slot)
  auto conv = [&](int s) { return bar0 + 8u * (4 * STAGES + s); };     // q expanded, both CTAs (leader)
  auto tfull = [&](int s) { return bar0 + 8u * (4 * STAGES + SLOTS + s); };       // accumulator filled
  auto tempty = [&](int s) { return bar0 + 8u * (4 * STAGES + SLOTS + 2 + s); };  // and read out (leader)
  const uint32_t drain = bar0 + 8u * (4 * STAGES + SLOTS + 4);
  constexpr int NBARS = 4 * STAGES + SLOTS + 5;
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
      bar_init(full_a(s), 1);
      bar_init(full_q(s), 1);
      bar_init(full_s(s), 32);
      bar_init(empty_a(s), 1);
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

  // Registers: 96 a thread at launch (5 warpgroups: 480 in all) = 32 + 2 * 56 + 2 * 168.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer, both CTAs
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      Item it;
      for (int i = pair; ok && get_item(p, i, it); i += npairs) {
        const int n0 = it.tile / p.tk * TILE + (int)rank * 128, k0 = it.tile % p.tk * TILE + (int)rank * 128;
        for (int st = it.s0; st < it.s1; ++st) {
          if (!bar_wait(empty_a(s), ph ^ 1u, ab, true)) {
            ok = false;
            break;
          }
          const uint32_t fa = leader ? full_a(s) : mapa(full_a(s), 0);
          if (leader) bar_expect(full_a(s), 2 * A_BYTES);
          bar_expect(full_q(s), Q_BYTES);
          const uint32_t a = smem_u32(smem + s * STAGE_BYTES);
          tma_load(a + A_BYTES, &tm_q, full_q(s), k0, st % p.mstep * BK);
          tma_load_pair(a, &tm_dy, fa, n0, st * BK);
          tma_load_pair(a + BOX, &tm_dy, fa, n0 + 64, st * BK);
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
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      Item it;
      for (int i = pair; ok && get_item(p, i, it); i += npairs) {
        for (int st = it.s0; ok && st < it.s1; ++g) {
          const int as = g & 1;
          if (!bar_wait(tempty(as), ((uint32_t)(g >> 1) & 1u) ^ 1u, ab, true)) {
            ok = false;
            break;
          }
          tc_after();
          const int end = min(st + p.seg, it.s1);
          for (bool first = true; st < end; ++st, first = false) {
            if (!bar_wait(full_a(s), ph, ab, true) || !bar_wait(conv(b), bph, ab, true)) {
              ok = false;
              break;
            }
            tc_after();
            const uint64_t da = desc0 + (uint32_t)(s * (STAGE_BYTES >> 4));
            const uint64_t db = desc0 + (uint32_t)((OFF_B + b * B_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              mma_pair(tmem + (uint32_t)(as * TILE), da + (uint64_t)(k * (2048 >> 4)), db + (uint64_t)(k * (2048 >> 4)),
                       idesc, !first || k != 0);
            mma_commit_pair(empty_a(s));
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
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
      // ---------------- scales of a step's 64 rows, that of row 8 j + r at 8 r + j
      const uint32_t dst = smem_u32(smem + OFF_S) + (uint32_t)((lane & 7) * 8 + (lane >> 3)) * 4;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      Item it;
      for (int i = pair; ok && get_item(p, i, it); i += npairs) {
        const int blk = it.tile % p.tk * 2 + (int)rank;  // this CTA's 128 columns: one scale block
        const float* sp = p.d.scale + (blk < p.d.nblk ? blk : 0);
        int row = it.s0 % p.mstep;  // step within a term of dy
        for (int st = it.s0; st < it.s1; ++st) {
          ok = __all_sync(0xffffffffu, bar_wait(empty_a(s), ph ^ 1u, ab, true));
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t m = (int64_t)row * BK + h * 32 + lane;
            const bool in = blk < p.d.nblk && m < p.d.M;
            cp_async4(dst + (uint32_t)(s * S_BYTES + h * 16), sp + (in ? m * p.d.nblk : 0), in);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ---------------- expand q: two groups of four warps take the steps in turn, so a step's
    // expansion may last two steps; thread (r, c) takes bytes 8c .. 8c + 7 of rows r + 8 j
    const int group = (warp - 4) >> 2;
    const int t = threadIdx.x & 127;
    const int c = t & 15, r = t >> 4;
    const uint32_t out = (uint32_t)(c >> 3) * BOX + (uint32_t)r * 128 + (uint32_t)(((c & 7) ^ r) << 4);
    int s = 0, b = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true;
    Item it;
    for (int i = pair; ok && get_item(p, i, it); i += npairs) {
      for (int st = it.s0; st < it.s1; ++st, ++turn) {
        if ((turn & 1) == group) {
          ok = bar_wait(full_q(s), ph, ab, true) && bar_wait(full_s(s), ph, ab, true);
          if (ok && turn >= SLOTS) {
            // the slot's last user, SLOTS steps back, was in stage s - SLOTS (this round's or,
            // below 0, the round before's)
            const int u = s - SLOTS;
            ok = bar_wait(empty_a(u < 0 ? u + STAGES : u), u < 0 ? ph ^ 1u : ph, ab, true);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* q = smem + s * STAGE_BYTES + A_BYTES + r * 128 + c * 8;
          uint8_t* o = smem + OFF_B + b * B_BYTES + out;
          const float4* sc4 = (const float4*)(smem + OFF_S + s * S_BYTES + r * 32);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 f = sc4[h];
            const float sc[4] = {f.x, f.y, f.z, f.w};
            uint2 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = *(const uint2*)(q + (4 * h + j) * 1024);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint64_t sc2;
              asm("mov.b64 %0, {%1, %1};" : "=l"(sc2) : "f"(sc[j]));
              const uint2 x = expand4<T>(u[j].x, sc2), y = expand4<T>(u[j].y, sc2);
              *(uint4*)(o + (4 * h + j) * 1024) = make_uint4(x.x, x.y, y.x, y.y);
            }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(mapa(conv(b), 0));
        }
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
        if (++b == SLOTS) b = 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // ---------------- sums and output: warp w has rows 32 (w % 4) .. of this CTA's 128 and
    // columns 128 h .. of the tile's 256
    const int w = warp - 4 - CONV_WARPS, quad = warp & 3, h = w >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(h * 128);
    int g = 0;
    bool ok = true;
    Item it;
    for (int i = pair; ok && get_item(p, i, it); i += npairs) {
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      for (int st = it.s0; st < it.s1; st += p.seg, ++g) {
        const int as = g & 1;
        ok = __all_sync(0xffffffffu, bar_wait(tfull(as), (uint32_t)(g >> 1) & 1u, ab, true));
        if (!ok) break;
        tc_after();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t r[16];
          tmem_ld16(taddr + (uint32_t)(as * TILE + j * 16), r);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[j * 16 + e] += __uint_as_float(r[e]);
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(mapa(tempty(as), 0));
      }
      if (!ok) break;
      if (it.part >= 0) {
        const int64_t slot = (int64_t)(it.tile - p.whole) * p.S;
        float4* mine = (float4*)(p.part + (((slot + it.part) * 2 + rank) * 8 + w) * PART_FLOATS) + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          mine[j * 32] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        __threadfence();
        __syncwarp();
        int done = 0;
        if (lane == 0) done = atomicAdd(p.count + ((it.tile - p.whole) * 2 + (int)rank) * 8 + w, 1);
        done = __shfl_sync(0xffffffffu, done, 0);
        if (done != p.S - 1) continue;  // another warp finishes this tile
        __threadfence();
        const float4* all = (const float4*)(p.part + ((slot * 2 + rank) * 8 + w) * PART_FLOATS) + lane;
        for (int part = 0; part < p.S; ++part, all += 2 * 8 * PART_FLOATS / 4) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float4 v = __ldcg(all + j * 32);
            acc[4 * j] = part == 0 ? v.x : acc[4 * j] + v.x;
            acc[4 * j + 1] = part == 0 ? v.y : acc[4 * j + 1] + v.y;
            acc[4 * j + 2] = part == 0 ? v.z : acc[4 * j + 2] + v.z;
            acc[4 * j + 3] = part == 0 ? v.w : acc[4 * j + 3] + v.w;
          }
        }
      }
      const int64_t n = (int64_t)(it.tile / p.tk) * TILE + rank * 128 + quad * 32 + lane;
      const int64_t k0 = (int64_t)(it.tile % p.tk) * TILE + h * 128;
      if (n < p.d.N) {
        D* row = (D*)p.d.dW + n * p.d.lddW;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (k0 + 16 * j < p.d.K) put16<D>(row + k0 + 16 * j, p.d.K - k0 - 16 * j, &acc[16 * j], p.vec, p.d.ovw);
      }
    }
  }

  // ---------------- teardown
  __syncwarp();
  tc_before();
  cluster_sync();  // no role of either CTA issues anything after this point
  if (threadIdx.x == 0) {
    // Every copy issued lands before shared memory is released. This CTA's q copies count on
    // its own barriers; the dy copies of both on the leader's, where an aborted pipeline can
    // have left the two producers one phase apart.
    for (int s = 0; s < STAGES; ++s) {
      const int mine = copies[s];
      if (mine > 0) bar_wait(full_q(s), (uint32_t)(mine - 1) & 1u, ab, false);
      if (!leader) continue;
      const int peer = (int)ld_cluster(mapa(smem_u32(&copies[s]), 1));
      int last = mine;
      if (peer > mine) {
        bar_expect(full_a(s), A_BYTES);
        last = peer;
      } else if (peer < mine) {
        bar_complete(full_a(s), A_BYTES);
      }
      if (last > 0) bar_wait(full_a(s), (uint32_t)(last - 1) & 1u, ab, false);
    }
  }
  cluster_sync();
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ------------------------------------------------------------------ staging
// dy rows that TMA cannot read in place (fp32, or a pitch that is no multiple of 16 bytes):
// copied to a 16-byte pitch; fp32 as three bf16 terms in planes of `rows` rows, each the
// leading 8 bits of what the ones before leave. Rows past M are zero.
template <typename T>
__global__ void __launch_bounds__(256) k_stage_dy(const T* __restrict__ dy, int64_t lddy, int64_t M, int64_t N,
                                                  int64_t rows, void* out, int64_t ld) {
  const int64_t m = blockIdx.x, n = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (n >= N) return;
  if constexpr (sizeof(T) == 4) {
    float x = m < M ? dy[m * lddy + n] : 0.0f;
    uint16_t* o = (uint16_t*)out + m * ld + n;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t hi = __float_as_uint(x) & 0xffff0000u;
      const bool fin = fabsf(x) < INFINITY;
      // a NaN whose set bits lie in the low half must not become an infinity
      o[i * rows * ld] = (uint16_t)((fin || x == x ? hi : 0x7fc00000u) >> 16);
      x = fin ? x - __uint_as_float(hi) : 0.0f;
    }
  } else {
    if (m < M) ((T*)out)[m * ld + n] = dy[m * lddy + n];
  }
}
__global__ void __launch_bounds__(256) k_stage_q(const uint8_t* __restrict__ q, int64_t ldq, int64_t K, uint8_t* out,
                                                 int64_t ld) {
  const int64_t m = blockIdx.x, k = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (k < K) out[m * ld + k] = q[m * ldq + k];
}

// ------------------------------------------------------------------ plan
struct Plan8 {
  int tn, tk, steps, mstep, whole, S;
  size_t off_count, off_part, off_dy, off_q, total;
  size_t count_bytes;
};

int max_pairs() { return num_sms() / 2; }

// Whole tiles fill whole waves of pairs; the rest are split S ways, S minimising the steps of
// the remaining waves plus the cost of the parts: writing and re-reading a part's 256 KB costs
// about a step's time per PART_COST parts over all pairs.
Plan8 plan(int64_t M, int64_t N, int64_t K, int dt, int pairs) {
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
      const double cost = waves + (S > 1 ? 6.0 + 0.15 * (double)(rest * S) : 0.0);
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
  p.count_bytes = split * 16 * 4;
  p.off_count = take(p.count_bytes);
  p.off_part = take(split * p.S * 16 * PART_FLOATS * 4);
  p.off_dy = take((size_t)terms * p.mstep * BK * round_up((size_t)N, 8) * 2);
  p.off_q = take((size_t)M * round_up((size_t)K, 16));
  p.total = off;
  return p;
}

template <typename T, typename D>
cudaError_t launch(const CUtensorMap& A, const CUtensorMap& Q, const Params& p, int64_t items, cudaStream_t s) {
  auto kern = k_dw_tc8<T, D>;
  // per-device cache of the pairs that fit at once; concurrent first launches may both set it
  static std::atomic<int> fit[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = fit[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (unsigned)max_pairs(), 1, 1);
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    fit[dev].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(2 * (unsigned)(items < n ? items : n), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, A, Q, p);
}

}  // namespace

bool dw_tc_supported() { return ptx::encode_fn() != nullptr; }

size_t dw_tc_workspace(int64_t M, int64_t N, int64_t K, int dt) { return plan(M, N, K, dt, max_pairs()).total; }

cudaError_t launch_dw_tc8(const DwArgs& a, int dt, int wdt, void* workspace, int* status, uint64_t timeout_ns,
                          cudaStream_t s) {
  const Plan8 pl = plan(a.M, a.N, a.K, dt, max_pairs());
  char* ws = (char*)workspace;
  Params p = {};
  p.d = a;
  p.tn = pl.tn;
  p.tk = pl.tk;
  p.steps = pl.steps;
  p.mstep = pl.mstep;
  p.whole = pl.whole;
  p.S = pl.S;
  p.seg = dt == FLCE_F32 ? SEG32 : SEG16;
  p.part = (float*)(ws + pl.off_part);
  p.count = (int*)(ws + pl.off_count);
  p.status = status;
  p.timeout_ns = timeout_ns;
  const int wsz = dtype_size(wdt);
  p.vec = rows16(a.dW, a.lddW, wsz);
  cudaError_t e = cudaSuccess;
  if (pl.count_bytes) e = cudaMemsetAsync(p.count, 0, pl.count_bytes, s);
  if (e != cudaSuccess) return e;

  const void* dy = a.dy;
  int64_t lddy = a.lddy, rows = a.M;
  if (dt == FLCE_F32 || !rows16(a.dy, a.lddy, 2)) {
    dy = ws + pl.off_dy;
    lddy = (int64_t)round_up((size_t)a.N, 8);
    const int64_t plane = (int64_t)pl.mstep * BK;
    const dim3 grid((unsigned)(dt == FLCE_F32 ? plane : a.M), (unsigned)cdiv64(a.N, 256));
    if (dt == FLCE_F32) {
      k_stage_dy<float><<<grid, 256, 0, s>>>((const float*)a.dy, a.lddy, a.M, a.N, plane, (void*)dy, lddy);
      rows = 3 * plane;
    } else {
      k_stage_dy<__half><<<grid, 256, 0, s>>>((const __half*)a.dy, a.lddy, a.M, a.N, plane, (void*)dy, lddy);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const uint8_t* q = a.q;
  int64_t ldq = a.ldq;
  if (!rows16(a.q, a.ldq, 1)) {
    q = (const uint8_t*)(ws + pl.off_q);
    ldq = (int64_t)round_up((size_t)a.K, 16);
    k_stage_q<<<dim3((unsigned)a.M, (unsigned)cdiv64(a.K, 256)), 256, 0, s>>>(a.q, a.ldq, a.K, (uint8_t*)q, ldq);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  CUtensorMap A, Q;
  const auto ty = dt == FLCE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!ptx::encode_2d(&A, ty, dy, a.N, rows, lddy * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !ptx::encode_2d(&Q, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, a.K, a.M, ldq, 128, BK, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int64_t items = p.whole + ((int64_t)p.tn * p.tk - p.whole) * p.S;
  if (dt == FLCE_F16)
    return wdt == FLCE_F32 ? launch<__half, float>(A, Q, p, items, s) : launch<__half, __half>(A, Q, p, items, s);
  if (wdt == FLCE_F32) return launch<__nv_bfloat16, float>(A, Q, p, items, s);
  return launch<__nv_bfloat16, __nv_bfloat16>(A, Q, p, items, s);
}

}  // namespace flce
