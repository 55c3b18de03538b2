// fused_tc.cu -- the fused operators' products on the 5th-generation tensor cores.
//
//   kLinear, kGated   D[n][m] = sum_k W^[n][k] x'[m][k]     (Z = X . W^T)
//   kGrad             D[k][m] = sum_n W^[n][k] dz'[m][n]    (dX = dZ . W^)
//
// Persistent CTA pairs, two SMs each, compute tiles of 256 rows x BN tokens with 256-row
// MMAs: each CTA dequantizes 128 of the rows and loads half of the tokens' activations.  A
// CTA's part of a gated tile is 64 gate rows and the 64 up rows that belong to them, so
// that act(G) * U is formed in the tile's epilogue and neither G nor U goes to memory
// (unless they are asked for).
//
// Roles (768 threads): warp 0 loads activations (TMA), warp 1 loads codes (TMA), warp 2 of
// the pair's first CTA issues the MMAs, warp 3 owns TMEM, warps 4..7 write results, warps
// 8..23 dequantize in four sets of four that take turns, a 64-deep block and an A buffer
// each.  The MMA and TMA instructions sit under elect.sync in warp-uniform code: issued
// from a thread-dependent branch, each one costs the issuing thread about 78 ns for
// operands moved to uniform registers one by one, whatever its size (measured; 4 x
// 128x256x16 in 313 ns instead of 280).
//
// Forward, the dequantized weights are the MMA's A operand in tensor memory: a thread
// owns a row, its TMEM lane.  For the gradient the contraction runs over the rows, and
// A needs W^ transposed: the threads write W^ as it lies (channels contiguous) into
// shared memory, which the MMA reads as an MN-major operand.  Both ways a word of eight
// codes takes 13 instructions: four pairs of exact 1024 + q (or 1024 + 16 q) by LOP3, an
// exact subtraction giving q - z, and one product with the scaled group scale, which is
// the only rounding (fp16, 2^-11).  bf16 operands would round to 2^-8: on top of a bf16
// output's own rounding that was half as much error again.
//
// Two accumulators in TMEM alternate between tiles, so a tile's epilogue runs under the
// next one's products; with BN <= 192 they leave room for four 64-deep A buffers.
//
// Scheduling: whole waves of tiles first, then the tiles that are left are cut along the
// contraction into one contiguous range per pair; the pieces' fp32 partials are summed, in
// order, by fused_finish, which also runs the epilogue.  No block waits for another.
//
// Bound: the tensor pipe, and for long calls the power limit.  Measured, this kernel alone:
// 191 us for 2048 x 8192 -> 8192 with residual (1440 TFLOP/s), 5.6 ms for the gated 8192 x
// 8192 -> 2 x 28672 (1370), 375 us for the gated 2048 x 4096 -> 2 x 14336 with Z saved
// (1280), 359 us for its gradient (1340), in runs of some 60 calls (the power limit takes
// more from longer ones); single CTAs with 128-row MMAs and three sets took 5 to 10 % more.  The
// epilogue is bound by instruction fetch: code added to it shows in every call (odd rows'
// columns spread over the lanes made their stores coalesced and all calls 3 to 12 %
// slower).
#include "act.cuh"
#include "common.cuh"

namespace w4 {

enum FusedMode { kLinear = 0, kGated = 1, kGrad = 2 };

struct FusedEpi {
  int64_t M, N;             // tokens, output columns of a linear / gradient call, F of a gated one
  const float *rinv;        // 1 / r per packed row
  const float *tinv;        // 1 / e per token
  const float *bias;        // forward, or NULL
  const float *colmul;      // gradient: awq_s, or NULL
  const void *residual;     // or NULL
  void *Z, *Y;              // Z or NULL
  int act, z_dtype, y_dtype, vec;  // vec: N is a multiple of 4
};

struct FusedTcParams {
  FusedEpi epi;
  const uint32_t *tab;      // [kg][rows] fp16 pairs (scale * r, 1024 + z)
  int64_t rows;             // packed rows
  int64_t kg;               // groups per packed row
  int gshift;               // log2(group)
  int bn, mt, rt, units;    // token tile, token tiles, pairs of row tiles, 128-deep units per tile
  int gt;                   // token tiles per raster block
  int full;                 // tiles computed whole
  int tiles, tail_pairs;    // all tiles (of 256 rows); CTA pairs that share the rest
  float *part;              // [2 * tail_pairs][2 CTAs][bn][128] partial tiles
};

namespace ftc {

constexpr int kSets = 4;                 // dequantizing sets of four warps, one A buffer each
constexpr int kThreads = 256 + kSets * 128;
constexpr int kCodeStages = 4, kCodeStage = 128 * 64;
constexpr int kAct = 64 * 2 / 2;         // bytes of a token's 64 channels in a stage, half of the tokens to a CTA
constexpr int kStageOut = 32 * 128 * 4;  // 32 tokens of a tile in fp32
constexpr int kGradAStage = 64 * 128 * 2;
constexpr int kMaxBn = 192;              // a multiple of 32
constexpr int kMaxActStages = 8;

__host__ __device__ constexpr int fixed_bytes(bool grad) {
  return 1024 + kCodeStages * kCodeStage + 2 * kStageOut + (grad ? kSets * kGradAStage : 0) + 256 * 4 + 512;
}
__host__ __device__ constexpr int act_stages(int bn, bool grad) {
  const int n = (227 * 1024 - fixed_bytes(grad)) / (bn * kAct);
  return n > kMaxActStages ? kMaxActStages : n;
}
// What the waits by parity rest on.  A set takes every (kSets / 2)-th unit of codes (two blocks
// each), so it comes back to a code stage at every turn of the ring, and waits for each of
// the stage's phases.  It waits for the products of its block before last, kSets blocks
// back, so a stage of activations that it arrives at has been through the turn before.
static_assert(kSets % 2 == 0 && kCodeStages % (kSets / 2) == 0, "a set visits a code stage at every turn or never");
static_assert(act_stages(kMaxBn, true) >= kSets && act_stages(kMaxBn, false) >= kSets, "a set's last block is a turn back");

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// Products of a CTA pair (M = 256: 128 rows in each CTA's tensor memory), issued by one
// thread of the pair's first CTA: D (+)= A B^T with A in tensor or shared memory.
__device__ __forceinline__ void pair_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives at the barrier of the same place in both CTAs once the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t *dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared::cluster address of the first CTA's barrier of the same place.
__device__ __forceinline__ uint32_t first_cta(const uint64_t *bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}
// (Release at the scope of the CTA: what the pair shares is tensor memory and operands read by
// the async proxy, which the fences in front order.  At cluster scope each arrive waited
// some 1,700 cycles for its warp's loads in flight.)
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// A TMA load into this CTA's memory (no multicast) that completes at a barrier of either CTA.
__device__ __forceinline__ void pair_tma_load(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// Whether the phase is complete, without waiting (try_wait may suspend the thread for
// microseconds).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by a whole warp with one answer, so that the warp-wide instructions behind it
// are reached by all lanes or by none.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, int err_bit) {
  return __all_sync(~0u, mbar_wait(bar, parity, err_bit));
}

// AND over the four epilogue warps (named barrier 1): either all of them go on or none.
__device__ __forceinline__ bool vote_epilogue(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                            *reinterpret_cast<const __half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// A volatile load, which stays where it is written: a whole block ahead of its use.
__device__ __forceinline__ uint32_t ldg_const(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// A group's constants as fp16 pairs: scale * r, 1024 + z, -(64 + z).
struct GroupK {
  uint32_t s, zlo, zhi;
  __device__ __forceinline__ void set(uint32_t w) {
    s = __byte_perm(w, w, 0x1010);
    zlo = __byte_perm(w, w, 0x3232);
    zhi = hsub2(0x63806380u, zlo);  // 960 - (1024 + z)
  }
};

// Eight codes -> pairs (0,4) (1,5) (2,6) (3,7) of fp16 (q - z) * scale * r.  1024 + q and
// 64 + q are exact in fp16, so are their differences; the product is rounded once.
__device__ __forceinline__ void dequant8(uint32_t w, const GroupK &g, uint32_t (&o)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t a = lop3_and_or(w, 0x000F000Fu, 0x64006400u), b = lop3_and_or(w, 0x00F000F0u, 0x64006400u);
  const uint32_t c = lop3_and_or(w8, 0x000F000Fu, 0x64006400u), d = lop3_and_or(w8, 0x00F000F0u, 0x64006400u);
  constexpr uint32_t k16th = 0x2C002C00u;  // 1/16
  o[0] = hmul2(hsub2(a, g.zlo), g.s);
  o[1] = hmul2(hfma2(b, k16th, g.zhi), g.s);
  o[2] = hmul2(hsub2(c, g.zlo), g.s);
  o[3] = hmul2(hfma2(d, k16th, g.zhi), g.s);
}

// A CTA pair's share of the work: tiles pair, pair + pairs, ... below `full`, then its
// range of the remaining tiles' units.  slot < 0: a whole tile.
struct Work {
  const FusedTcParams &p;
  int t;
  int64_t u, u1, base;
  int nth;
  int pair, pairs;
  __device__ __forceinline__ explicit Work(const FusedTcParams &q)
      : p(q), t(blockIdx.x >> 1), u(0), u1(0), nth(0), pair(blockIdx.x >> 1), pairs(gridDim.x >> 1) {
    if (pair < p.tail_pairs) {
      const int64_t total = (int64_t)(p.tiles - p.full) * p.units;
      u = total * pair / p.tail_pairs;
      u1 = total * (pair + 1) / p.tail_pairs;
    }
  }
  __device__ __forceinline__ bool next(int &tile, int &k0, int &k1, int &slot) {
    if (t < p.full) {
      tile = t;
      k0 = 0;
      k1 = p.units;
      slot = -1;
      t += pairs;
      return true;
    }
    if (u >= u1) return false;
    const int i = (int)(u / p.units);
    tile = p.full + i;
    k0 = (int)(u - (int64_t)i * p.units);
    k1 = (int)min((int64_t)p.units, k0 + (u1 - u));
    u += k1 - k0;
    slot = k1 - k0 == p.units ? -1 : 2 * pair + nth;
    ++nth;
    return true;
  }
};

// Raster: blocks of gt token tiles, inside a block the token tiles of one row tile side
// by side, so that the CTAs at work at one time share activations and weights in L2.
__device__ __forceinline__ void tile_at(const FusedTcParams &p, int t, int rank, int &row, int &tok) {
  const int per = p.gt * p.rt, g = t / per, r = t - g * per;
  const int w = min(p.gt, p.mt - g * p.gt);
  const int pr = r / w;
  tok = g * p.gt + r - pr * w;
  row = 2 * pr + rank;
}

// The k that tile row r of a gradient tile holds: the dequantization's pairs put code
// {0,4,1,5,2,6,3,7}[j] of a word at place j.
__device__ __forceinline__ int grad_row(int r) { return (r & ~7) | ((r & 1) << 2) | ((r >> 1) & 3); }

// 16-bit types both ways without a branch: both conversions, and the one that counts.
__device__ __forceinline__ void widen4(const uint2 &w, int dtype, float (&v)[4]) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
  const bool bf16 = dtype == 2;
  v[0] = bf16 ? __uint_as_float(w.x << 16) : a.x;
  v[1] = bf16 ? __uint_as_float(w.x & 0xFFFF0000u) : a.y;
  v[2] = bf16 ? __uint_as_float(w.y << 16) : b.x;
  v[3] = bf16 ? __uint_as_float(w.y & 0xFFFF0000u) : b.y;
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, int dtype) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return dtype == 2 ? *reinterpret_cast<const uint32_t *>(&x) : half2_bits(a, b);
}

// Stores v at columns n.. of a row that starts at element `row`; n + j < lim (a multiple of 4
// where rows start on vectors).
__device__ __forceinline__ void put4(void *p, int dtype, int64_t row, int64_t n, int64_t lim, bool vec, const float (&v)[4]) {
  const int in = (int)min((int64_t)4, lim - n);
  if (dtype != 0) {
    const uint32_t a = narrow2(v[0], v[1], dtype), b = narrow2(v[2], v[3], dtype);
    uint16_t *q = static_cast<uint16_t *>(p) + row + n;
    if (vec) {
      *reinterpret_cast<uint2 *>(q) = make_uint2(a, b);
    } else {
      q[0] = (uint16_t)a;
      if (in > 1) q[1] = (uint16_t)(a >> 16);
      if (in > 2) q[2] = (uint16_t)b;
      if (in > 3) q[3] = (uint16_t)(b >> 16);
    }
  } else {
    float *q = static_cast<float *>(p) + row + n;
    if (vec) {
      *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      q[0] = v[0];
      if (in > 1) q[1] = v[1];
      if (in > 2) q[2] = v[2];
      if (in > 3) q[3] = v[3];
    }
  }
}

// Factor and bias of four output columns (0 behind the last); first: packed row (forward) or
// channel (gradient) of the first one, column n of lim.
struct ColK {
  float f[4], b[4];
  __device__ __forceinline__ void load(const FusedEpi &e, bool grad, int64_t first, int64_t n, int64_t lim) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool ok = n + j < lim;
      f[j] = !ok ? 0.0f : grad ? (e.colmul ? e.colmul[first + j] : 1.0f) : e.rinv[first + j];
      b[j] = ok && e.bias ? e.bias[first + j] : 0.0f;
    }
  }
  // z = v * factor / e + bias
  __device__ __forceinline__ void scale(const float4 &v, float inv, float (&z)[4]) const {
    z[0] = v.x * f[0] * inv + b[0];
    z[1] = v.y * f[1] * inv + b[1];
    z[2] = v.z * f[2] * inv + b[2];
    z[3] = v.w * f[3] * inv + b[3];
  }
};

// The residual's four values at (m, n), as they lie (16 bits); 0 behind the last column.
__device__ __forceinline__ uint2 residual4(const FusedEpi &e, int64_t m, int64_t n) {
  const uint16_t *q = static_cast<const uint16_t *>(e.residual) + m * e.N + n;
  if (e.vec) return *reinterpret_cast<const uint2 *>(q);
  const int in = (int)min((int64_t)4, e.N - n);
  const uint32_t a = q[0], b = in > 1 ? q[1] : 0u, c = in > 2 ? q[2] : 0u, d = in > 3 ? q[3] : 0u;
  return make_uint2(a | b << 16, c | d << 16);
}

// `res`: the residual's values where `have`, else they are read here.
__device__ __forceinline__ void finish_linear(const FusedEpi &e, int64_t m, int64_t n, float (&z)[4], bool have, const uint2 &res) {
  const int64_t row = m * e.N;
  if (e.Z) put4(e.Z, e.z_dtype, row, n, e.N, e.vec, z);
  act_fwd4(z, e.act);
  if (have) {
    float a[4];
    widen4(res, e.y_dtype, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] += a[j];
  } else if (e.residual) {  // fp32
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      z[0] += n + j < e.N ? load_as_float(e.residual, e.y_dtype, row + n + j) : 0.0f;
      const float t = z[0];  // the four values turn round
      z[0] = z[1]; z[1] = z[2]; z[2] = z[3]; z[3] = t;
    }
  }
  put4(e.Y, e.y_dtype, row, n, e.N, e.vec, z);
}

__device__ __forceinline__ void finish_gated(const FusedEpi &e, int64_t m, int64_t f, float (&g)[4], const float (&u)[4]) {
  if (e.Z) {
    put4(e.Z, e.z_dtype, m * 2 * e.N, f, e.N, e.vec, g);
    put4(e.Z, e.z_dtype, m * 2 * e.N + e.N, f, e.N, e.vec, u);
  }
  act_fwd4(g, e.act);
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] *= u[j];
  put4(e.Y, e.y_dtype, m * e.N, f, e.N, e.vec, g);
}

}  // namespace ftc

template <int kMode>
__global__ void __launch_bounds__(ftc::kThreads, 1)
    fused_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmP,
                    const FusedTcParams p) {
  using namespace ftc;
  constexpr bool kIsGrad = kMode == kGrad;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int ns = act_stages(p.bn, kIsGrad);
  const int act_stage = p.bn * kAct;
  uint8_t *sC = smem;
  float *sOut = reinterpret_cast<float *>(sC + kCodeStages * kCodeStage);
  uint8_t *sA = reinterpret_cast<uint8_t *>(sOut) + 2 * kStageOut;
  uint8_t *sX = sA + (kIsGrad ? kSets * kGradAStage : 0);
  float *sTok = reinterpret_cast<float *>(sX + ns * act_stage);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sTok + 256);
  uint64_t *full = bars, *empty = full + kMaxActStages;
  uint64_t *cfull = empty + kMaxActStages, *cempty = cfull + kCodeStages;
  uint64_t *dfull = cempty + kCodeStages, *dempty = dfull + 2;
  uint32_t *holder = reinterpret_cast<uint32_t *>(dempty + 2);

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;

  const int rank = (int)(blockIdx.x & 1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ns; ++i) {
      mbar_init(&full[i], 1 + 8);  // the first CTA's: both boxes of activations, and a set's 4 warps in each CTA
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kCodeStages; ++i) {
      mbar_init(&cfull[i], 1);
      mbar_init(&cempty[i], 256);  // a unit's two blocks, a set each
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 8);  // the first CTA's: the epilogue's warps of both
    }
    fence_barrier_init();
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmP);
  }
  if (warp == 3) pair_tmem_alloc(holder, 512);
  tc_fence_before();
  __syncthreads();
  pair_sync();  // the other CTA's barriers are there before anything arrives at them
  tc_fence_after();
  const uint32_t tmem = *holder;
  bool ok = true;

  Work work(p);
  int tile, k0, k1, slot;
  if (warp == 0) {
    // ---- activations: a box of half the tile's tokens x 64 per stage and CTA
    grid_dependency_wait();
    int s = 0;
    uint32_t ph = 0;
    while (ok && work.next(tile, k0, k1, slot)) {
      int row, tok;
      tile_at(p, tile, rank, row, tok);
      for (int b = 2 * k0; b < 2 * k1; ++b) {
        if (!wait_all(&empty[s], ph ^ 1u, kErrTimeoutTma)) { ok = false; break; }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * act_stage));
          pair_tma_load(sX + s * act_stage, &tmX, first_cta(&full[s]), b * 64, tok * p.bn + rank * (p.bn / 2));
        }
        __syncwarp();
        if (++s == ns) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ---- codes: 128 rows x 128 channels per stage (64-byte rows, 64-byte swizzle)
    int s = 0;
    uint32_t ph = 0;
    while (ok && work.next(tile, k0, k1, slot)) {
      int row, tok;
      tile_at(p, tile, rank, row, tok);
      for (int u = k0; u < k1; ++u) {
        if (!wait_all(&cempty[s], ph ^ 1u, kErrTimeoutTma)) { ok = false; break; }
        if (elect_one()) {
          mbar_arrive_expect_tx(&cfull[s], kCodeStage);
          uint8_t *dst = sC + s * kCodeStage;
          if (kMode == kGrad) {
            tma_load_2d(dst, &tmP, &cfull[s], row * 64, u * 128);
          } else if (kMode == kLinear) {
            tma_load_2d(dst, &tmP, &cfull[s], u * 64, row * 128);
          } else {
            tma_load_2d(dst, &tmP, &cfull[s], u * 64, row * 64);
            tma_load_2d(dst + kCodeStage / 2, &tmP, &cfull[s], u * 64, (int)p.epi.N + row * 64);
          }
        }
        __syncwarp();
        if (++s == kCodeStages) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 2 && rank == 0) {
    // ---- products of both CTAs: M = 256; bit 15: A is MN-major
    const uint32_t idesc = (idesc_f16(false, p.bn) + ((uint32_t)(128 >> 4) << 24)) | (kIsGrad ? 1u << 15 : 0u);
    int s = 0, a = 0, d = 0;
    uint32_t ph = 0, dph = 0;
    bool ready = false;  // the barrier of the block at hand was seen complete while the last one was issued
    while (ok && work.next(tile, k0, k1, slot)) {
      if (!wait_all(&dempty[d], dph ^ 1u, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(d * p.bn);
      for (int b = 2 * k0; b < 2 * k1; ++b) {
        if (!ready && !wait_all(&full[s], ph, kErrTimeoutMma)) { ok = false; break; }
        tc_fence_after();
        const uint64_t bd = smem_desc_k_sw128(smem_u32(sX + s * act_stage));
        uint64_t *done = &empty[s];
        if (++s == ns) s = 0, ph ^= 1u;
        ready = __all_sync(~0u, mbar_test(&full[s], ph));
        if (elect_one()) {
          if constexpr (kIsGrad) {
            // MN-major A: 64-channel halves 8192 bytes apart (leading offset), 8-row
            // groups of the contraction 1024 bytes apart (stride offset)
            const uint64_t ad = (smem_desc_k_sw128(smem_u32(sA + a * kGradAStage)) & ~((uint64_t)0x3FFF << 16)) |
                                ((uint64_t)(8192 >> 4) << 16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              pair_mma_ss(acc, ad + (uint64_t)(128 * j), bd + (uint64_t)(2 * j), idesc, b == 2 * k0 && j == 0 ? 0u : 1u);
          } else {
            const uint32_t at = tmem + (uint32_t)(2 * p.bn + 32 * a);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              pair_mma_ts(acc, at + 8 * j, bd + (uint64_t)(2 * j), idesc, b == 2 * k0 && j == 0 ? 0u : 1u);
          }
          pair_commit(done);
          if (b == 2 * k1 - 1) pair_commit(&dfull[d]);
        }
        __syncwarp();
        if (++a == kSets) a = 0;
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
  } else if (warp >= 8) {
    // ---- dequantization: set j takes blocks j, j + kSets, ... of the CTA's whole sequence and
    // owns A buffer j, so it converts a block while the other sets' blocks are multiplied
    const int set = (warp - 8) >> 2, wq = warp & 3;
    grid_dependency_wait();  // the group constants
    // forward: this thread's packed row, TMEM lane r = 32 wq + lane
    // gradient: row nl of the block (of the contraction), channel half kh
    const int r = 32 * wq + lane, nl = 32 * (wq & 1) + lane, kh = wq >> 1;
    // The next block of this set: its constants (two 32-channel pieces) are fetched a
    // whole block of this set's ahead, across the ends of tiles.
    int b = set, b1 = 0;  // place in the current range of blocks, its end
    int64_t n = 0;
    int row = 0;
    bool row_ok = false;
    uint32_t gw[2];
    auto seek = [&]() -> bool {  // moves to the range that holds block b
      while (b >= b1) {
        b -= b1;
        if (!work.next(tile, k0, k1, slot)) return false;
        int tok;
        tile_at(p, tile, rank, row, tok);
        b += 2 * k0;
        b1 = 2 * k1;
        if constexpr (kMode == kLinear) {
          n = (int64_t)row * 128 + r;
          row_ok = n < p.rows;
        } else if constexpr (kMode == kGated) {
          const int64_t f = (int64_t)row * 64 + (r & 63);
          n = r < 64 ? f : p.epi.N + f;
          row_ok = f < p.epi.N;
        }
      }
      return true;
    };
    auto fetch = [&]() {
      if constexpr (kIsGrad) {
        n = (int64_t)b * 64 + nl;
        row_ok = n < p.rows;
      }
      const int64_t ch = kIsGrad ? (int64_t)row * 128 + 64 * kh : (int64_t)b * 64;
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // two loads even where both pieces are in one group: a
        // copy of the first one's value would wait for it here
        const int64_t g = (ch + 32 * c) >> p.gshift;
        gw[c] = row_ok && g < p.kg ? ldg_const(p.tab + g * p.rows + n) : 0u;
      }
    };
    bool more = seek();
    if (more) fetch();
    int s = set, ps = 0;  // ring stage of the block, and of this set's last one
    uint32_t sph = 0, pph = 0;
    for (int ia = set; more; ia += kSets) {
      const int cs = (ia >> 1) % kCodeStages, h = ia & 1;
      if (!wait_all(&cfull[cs], (uint32_t)((ia >> 1) / kCodeStages) & 1u, kErrTimeoutDequant)) { ok = false; break; }
      // forward: row r, chunks 2h, 2h + 1;  gradient: row 64 h + nl, chunks 2 kh, 2 kh + 1
      const int cr = kIsGrad ? 64 * h + nl : r, cc = kIsGrad ? 2 * kh : 2 * h;
      const uint32_t base = smem_u32(sC + cs * kCodeStage) + (uint32_t)(cr * 64), sw = (uint32_t)((cr >> 1) & 3);
      const uint4 q0 = lds128(base + ((((uint32_t)cc) ^ sw) << 4));
      const uint4 q1 = lds128(base + ((((uint32_t)cc + 1u) ^ sw) << 4));
      GroupK g[2];
      g[0].set(gw[0]);
      g[1].set(gw[1]);
      b += kSets;
      more = seek();
      if (more) fetch();
      const uint32_t wd[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      uint32_t out[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t o[4];
        dequant8(wd[j], g[j >> 2], o);
#pragma unroll
        for (int x = 0; x < 4; ++x) out[4 * j + x] = o[x];
      }
      // the buffer is free once this set's last block has been multiplied
      if (ia >= kSets && !wait_all(&empty[ps], pph, kErrTimeoutDequant)) { ok = false; break; }
      if constexpr (kIsGrad) {
        const uint32_t dst = smem_u32(sA + set * kGradAStage) + (uint32_t)(kh * 8192 + nl * 128);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (uint32_t)((j ^ (nl & 7)) << 4)),
                       "r"(out[4 * j]), "r"(out[4 * j + 1]), "r"(out[4 * j + 2]), "r"(out[4 * j + 3])
                       : "memory");
        fence_proxy_async_smem();
      } else {
        tc_fence_after();
        tmem_st_32x32b_x32(tmem + ((uint32_t)(32 * wq) << 16) + (uint32_t)(2 * p.bn + 32 * set), out);
        tc_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (elect_one()) arrive_cluster(first_cta(&full[s]));
      // The codes are given back only here, behind the stores that needed them: an arrive
      // right behind the loads let the loads sink below it, and now and then read the
      // stage's next contents.
      mbar_arrive(&cempty[cs]);
      ps = s;
      pph = sph;
      s += kSets;
      if (s >= ns) s -= ns, sph ^= 1u;
    }
  } else if (warp >= 4) {
    // ---- epilogue
    const int q = warp & 3, tid = threadIdx.x - 128;
    grid_dependency_wait();  // row and token factors
    const FusedEpi &e = p.epi;
    int d = 0;
    uint32_t dph = 0;
    while (work.next(tile, k0, k1, slot)) {
      int row, tok;
      tile_at(p, tile, rank, row, tok);
      const int64_t m0 = (int64_t)tok * p.bn;
      for (int t = tid; t < p.bn; t += 128) sTok[t] = m0 + t < e.M ? e.tinv[m0 + t] : 0.0f;
      // four columns of the tile (gated: and the same of the up half), and with 32 (16)
      // lanes to a token, a warp's 8 tokens of a chunk of 32
      constexpr int kLanes = kMode == kGated ? 16 : 32, kTok = 8 * kLanes / 32, kStep = 32 / kLanes;
      constexpr int kGroup4 = kMode == kLinear ? 4 : 2;
      const int col = 4 * (lane & (kLanes - 1)), t0 = 8 * q + lane / kLanes;
      const int64_t n = (int64_t)row * (kMode == kGated ? 64 : 128) + col;
      ColK c0, c1;
      if (slot < 0) {
        c0.load(e, kIsGrad, n, n, e.N);
        if (kMode == kGated) c1.load(e, false, e.N + n, n, e.N);
      }
      const bool ahead = kMode == kLinear && slot < 0 && e.residual && e.y_dtype != 0 && n < e.N;
      if (!vote_epilogue(mbar_wait(&dfull[d], dph, kErrTimeoutEpilogue))) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(d * p.bn);
      const int prow = kIsGrad ? grad_row(32 * q + lane) : 32 * q + lane;
      for (int c = 0; c * 32 < p.bn; ++c) {
        const int lim = (int)min((int64_t)p.bn, e.M - m0) - c * 32;  // valid tokens from this chunk on
        uint2 res[4];
        auto read_ahead = [&](int s0) {  // the residuals of four of this thread's tokens
          if (ahead)
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (t0 + s0 + s < lim) res[s] = residual4(e, m0 + c * 32 + t0 + s0 + s, n);
        };
        if constexpr (kMode == kLinear) read_ahead(0);  // on their way while the sums come out of tensor memory
        uint32_t v[32];
        tmem_ld_32x32b_x32(acc + (uint32_t)(c * 32), v);
        tc_wait_ld();
        if ((c + 1) * 32 >= p.bn) {
          tc_fence_before();
          __syncwarp();
          if (elect_one()) arrive_cluster(first_cta(&dempty[d]));
        }
        float *st = sOut + (c & 1) * (kStageOut / 4);
#pragma unroll
        for (int j = 0; j < 32; ++j) st[j * 128 + prow] = __uint_as_float(v[j]);
        bar_epilogue();
        if (slot >= 0) {
          float *dst = p.part + (((int64_t)slot * 2 + rank) * p.bn + c * 32) * 128;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const int t = 8 * q + s;
            if (t < lim)
              reinterpret_cast<float4 *>(dst + t * 128)[lane] = reinterpret_cast<const float4 *>(st + t * 128)[lane];
          }
        } else if (n < e.N) {
          // (loops of few tokens: a long epilogue waits for its instructions, see act_fwd4)
#pragma unroll 1
          for (int s0 = 0; s0 < kTok; s0 += kGroup4) {
            uint2 now[kGroup4];
#pragma unroll
            for (int s = 0; s < kGroup4; ++s) now[s] = res[s];
            if (kMode == kLinear && s0 + kGroup4 < kTok) read_ahead(s0 + kGroup4);
#pragma unroll
            for (int s = 0; s < kGroup4; ++s) {
              const int t = t0 + (s0 + s) * kStep;
              if (t < lim) {
                const float inv = sTok[c * 32 + t];
                float z[4];
                c0.scale(*reinterpret_cast<const float4 *>(st + t * 128 + col), inv, z);
                if constexpr (kMode == kGated) {
                  float u[4];
                  c1.scale(*reinterpret_cast<const float4 *>(st + t * 128 + 64 + col), inv, u);
                  finish_gated(e, m0 + c * 32 + t, n, z, u);
                } else {
                  finish_linear(e, m0 + c * 32 + t, n, z, ahead, now[s]);
                }
              }
            }
          }
        }
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
      bar_epilogue();  // sTok is read until here
    }
  }
  // A wait that ran out: copies of this CTA may still be in flight; give them time to land.
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {}
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // neither CTA leaves while the other's products read or arrive here
  if (warp == 3) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 512);
  }
}

// Sums the partial tiles of the tiles cut along the contraction, in order, and runs the
// epilogue: 4 outputs per thread, 8 (gated: 16) tokens per block at a time.
template <int kMode>
__global__ void __launch_bounds__(256) fused_finish(const FusedTcParams p) {
  using namespace ftc;
  grid_dependency_wait();
  constexpr int kTok = kMode == kGated ? 16 : 8, kPer = 256 / kTok;
  const FusedEpi &e = p.epi;
  const int t = blockIdx.x >> 1, rank = blockIdx.x & 1;  // among the cut tiles; the pair's CTA
  const int64_t total = (int64_t)(p.tiles - p.full) * p.units, u0 = (int64_t)t * p.units, u1 = u0 + p.units;
  // the pairs whose ranges [total c / C, total (c + 1) / C) meet [u0, u1): a pair's second
  // piece is the start of a tile, its first one the rest of the tile before
  auto begin = [&](int c) { return total * c / p.tail_pairs; };
  int c0 = (int)(u0 * p.tail_pairs / total);
  while (begin(c0 + 1) <= u0) ++c0;
  int c1 = c0;
  while (begin(c1 + 1) < u1) ++c1;
  if (c0 == c1) return;  // computed whole
  const bool second = begin(c0) < u0;  // pair c0 began in the tile before
  int row, tok;
  tile_at(p, p.full + t, rank, row, tok);
  const int col = 4 * (threadIdx.x % kPer);
  const int64_t n = kMode == kGated ? (int64_t)row * 64 + col : (int64_t)row * 128 + col;
  if (n >= e.N) return;
  ColK k, ku;
  k.load(e, kMode == kGrad, n, n, e.N);
  if (kMode == kGated) ku.load(e, false, e.N + n, n, e.N);
  const float *first = p.part + (((int64_t)2 * c0 + (second ? 1 : 0)) * 2 + rank) * p.bn * 128 + col;
  const float *rest = p.part + ((int64_t)4 * (c0 + 1) + rank) * p.bn * 128 + col;  // then every 4 bn rows
  auto add = [](float4 &a, const float4 &x) { a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w; };
  const int lim = (int)min((int64_t)p.bn, e.M - (int64_t)tok * p.bn);
#pragma unroll 2
  for (int tt = blockIdx.y * kTok + threadIdx.x / kPer; tt < lim; tt += gridDim.y * kTok) {
    const int64_t m = (int64_t)tok * p.bn + tt;
    const float *src = first + tt * 128, *more = rest + tt * 128;
    float4 v = *reinterpret_cast<const float4 *>(src), w = make_float4(0, 0, 0, 0);
    if (kMode == kGated) w = *reinterpret_cast<const float4 *>(src + 64);
#pragma unroll 2
    for (int c = c0 + 1; c <= c1; ++c, more += (int64_t)4 * p.bn * 128) {
      add(v, *reinterpret_cast<const float4 *>(more));
      if (kMode == kGated) add(w, *reinterpret_cast<const float4 *>(more + 64));
    }
    const float inv = e.tinv[m];
    float z[4];
    k.scale(v, inv, z);
    if (kMode == kGated) {
      float u[4];
      ku.scale(w, inv, u);
      finish_gated(e, m, n, z, u);
    } else {
      const bool have = e.residual && e.y_dtype != 0;
      finish_linear(e, m, n, z, have, have ? residual4(e, m, n) : make_uint2(0, 0));
    }
  }
}

template <int kMode>
cudaError_t launch_fused_tc_mode(const CUtensorMap &tmX, const CUtensorMap &tmP, const FusedTcParams &p, int pairs,
                                 cudaStream_t s) {
  static std::atomic<int> attr[kAttrDevices];
  constexpr bool grad = kMode == kGrad;
  const int smem = ftc::fixed_bytes(grad) + ftc::act_stages(p.bn, grad) * p.bn * ftc::kAct;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fused_tc_kernel<kMode>), smem, attr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(ftc::kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fused_tc_kernel<kMode>, tmX, tmP, p);
  if (e != cudaSuccess || p.full == p.tiles) return e;
  // about six blocks per SM, each at least one step of 8 (16) tokens
  const int tok = kMode == kGated ? 16 : 8, cut = 2 * (p.tiles - p.full), steps = (p.bn + tok - 1) / tok;
  int y = (12 * pairs + cut - 1) / cut;
  y = y > steps ? steps : y;
  return launch_pdl(fused_finish<kMode>, dim3((unsigned)cut, (unsigned)y), dim3(256), (size_t)0, s, p);
}

cudaError_t launch_fused_tc(int mode, const CUtensorMap &tmX, const CUtensorMap &tmP, const FusedTcParams &p, int pairs,
                            cudaStream_t s) {
  return mode == kLinear  ? launch_fused_tc_mode<kLinear>(tmX, tmP, p, pairs, s)
         : mode == kGated ? launch_fused_tc_mode<kGated>(tmX, tmP, p, pairs, s)
                          : launch_fused_tc_mode<kGrad>(tmX, tmP, p, pairs, s);
}

}  // namespace w4
