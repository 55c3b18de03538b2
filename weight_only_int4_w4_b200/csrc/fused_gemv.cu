// fused_gemv.cu -- w4a16_linear and w4a16_gated for up to 8 tokens (groups of 128), in one
// kernel without workspace: the call reads every weight once and is bound by that.
//
// A CTA (one per SM) owns an equal range of output rows, whatever its length, so that
// every SM streams the same number of bytes; the row blocks of 16 that mma.sync works on
// may end anywhere (rows behind the range are the last one again, and dropped).  Inside
// the CTA the warps split K: a warp walks over the CTA's row blocks with the activations
// of its own channels, as B fragments, in registers.  So the main loop has no barrier, no
// exchange between lanes and no traffic but the weights, which come by TMA into a ring per
// warp: 16 rows x 2 groups a piece, three or four pieces in flight.  The warps' partial
// sums meet in shared memory once, at the end, in a fixed order, where bias, activation,
// product and residual follow.
//
// Every CTA reads the activations of its channels.  Where those would be more than a
// quarter of its weights (many tokens, few rows per SM), clusters of 2 or 4 CTAs take a
// range of rows together and split K between them, and their sums meet through
// distributed shared memory.
//
// Arithmetic (exact up to fp32 sums):  a code is used as it lies, as the fp16 subnormal
// q 2^-24 (low nibbles, one AND per pair) or 16 q 2^-24 (high nibbles; their activations
// are divided by 16): five instructions per eight weights, where subtracting z from every
// pair takes nine.  Per group, with D the MMA's sum and D1 the sum that the same MMAs give
// for codes of 1 (formed once per piece of channels),
//   sum (q - z) x' = 2^24 (D - z D1).
// x' = x s 2^b, b per token and piece of channels with the largest |x'| of the piece in
// [2^13, 2^14): bf16 converts exactly down to 2^-26 and fp16 to 2^-23 of that largest value
// (of the channels divided by 16; 2^-30 and 2^-27 of the others), below it fp16's subnormals
// cut bits off; x * s is rounded to fp16 once; 2^-b follows with the scale.
//
// Fragments (g = lane / 4, t = lane % 4): lane (g, t) loads the 32 codes of channels
// 32 t .. 32 t + 31 of rows g and g + 8 of a group; word w of them feeds two MMAs, whose k
// order is the same permutation on both sides: channels 32 t + 8 w + {0, 4, 1, 5} and
// {2, 6, 3, 7}.
//
// Bound: at the start and end of a call latency; in between neither HBM nor the issue slots:
// warps wait for loads, the scales and zero points that are fetched one piece ahead among
// them.  Measured with 1 / 8 tokens, back to back in a graph: 6.8 / 9.1 us at 4096 x 4096
// (8.9 MB of weights), 18.1 / 19.5 us at 14336 -> 4096 (31 MB), 23.0 / 25.9 us for the gated
// 4096 -> 2 x 14336 (62 MB, 2.7 TB/s) and 67.9 / 72.5 us for 8192 -> 2 x 28672 (250 MB, 3.7
// TB/s).  At 62 MB counters give 48 % of the issue slots taken, and the wait for global
// loads as the largest stall.  A copy ring per lane in place of TMA, and prefetches into
// L2, were slower.
#include "act.cuh"
#include "common.cuh"

namespace w4 {

struct FusedGemvParams {
  const uint16_t *X;
  int64_t M, N, K;          // N: output columns (F for gated)
  const uint16_t *scales, *zeros;
  const float *awq_s;
  FusedEpi epi;
  int ksw;                  // warps of a CTA that split K
  int depth;                // pieces in flight per warp
  int cluster;              // CTAs that share a range of rows and split K
  int nblk;                 // row blocks of the longest CTA range (gated: gate and up)
};

namespace fgv {

constexpr int kWarps = 16;
constexpr int kMaxTokens = 8;
constexpr int kSmemMax = 226 * 1024;

constexpr int C = 2;              // groups per piece
constexpr int kPiece = C * 1024;  // 16 rows of them
// the warps' rings, their barriers, partial sums per warp, and a cluster's sums per CTA
__host__ __device__ constexpr int ring_bytes(int depth) { return kWarps * depth * (kPiece + 8) + 1024; }
__host__ __device__ constexpr int smem_bytes(int ksw, int nblk, int m, int cluster, int depth) {
  return ring_bytes(depth) + (ksw + (cluster > 1 ? 1 : 0)) * nblk * 16 * ((m + 1) & ~1) * 4;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(const float *p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// d = a * b + (first ? 0 : d)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
  if (first)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Ordered against the copies around it (a plain load may be moved across them).
__device__ __forceinline__ uint4 lds128_ordered(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}

__device__ __forceinline__ uint32_t ldg_u16(const uint16_t *p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t ldg_u32(const uint16_t *p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

}  // namespace fgv

// The activations of 32 channels of `C` groups (token row x, channels ch + 128 c ..; nothing
// where !in) as B fragments, and the factor 2^-b.  Lanes of a token (t = 0..3) share b.
template <bool kBf16>
__device__ __forceinline__ float stage_b(const uint16_t *x, const float *awq_s, bool in, int last,
                                         uint32_t (&bf)[fgv::C][16]) {
  using fgv::C;
  uint4 raw[C][4];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      raw[c][q] = in && c <= last ? *reinterpret_cast<const uint4 *>(x + c * kGroup + 8 * q) : make_uint4(0, 0, 0, 0);
    }
  float amax = 0.0f;
  if (!awq_s) {
    // |x| as bit patterns: 16-bit floats of one sign order like their bits
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        top = __vmaxu2(top, raw[c][q].x & 0x7FFF7FFFu);
        top = __vmaxu2(top, raw[c][q].y & 0x7FFF7FFFu);
        top = __vmaxu2(top, raw[c][q].z & 0x7FFF7FFFu);
        top = __vmaxu2(top, raw[c][q].w & 0x7FFF7FFFu);
      }
    top = max(top >> 16, top & 0xFFFFu);
    amax = kBf16 ? __uint_as_float(top << 16) : half_bits_to_float((uint16_t)top);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
        unpack8<kBf16>(raw[c][q], f);
        if (in && c <= last) {
          const float4 *a = reinterpret_cast<const float4 *>(awq_s + c * kGroup + 8 * q);
          const float4 u = a[0], v = a[1];
          f[0] *= u.x; f[1] *= u.y; f[2] *= u.z; f[3] *= u.w;
          f[4] *= v.x; f[5] *= v.y; f[6] *= v.z; f[7] *= v.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
      }
  }
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
  const float2 e = pow2_to(amax, 13);
  // channels 1, 3, 5, 7 sit in the high nibbles: x' / 16 (a subnormal keeps its leading
  // bits: at most 2^-25 of the piece's largest value 2^13 goes)
  const float lo = e.x, hi = e.x * 0.0625f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[8];
      unpack8<kBf16>(raw[c][q], f);
      if (awq_s && in && c <= last) {
        const float4 *a = reinterpret_cast<const float4 *>(awq_s + c * kGroup + 8 * q);
        const float4 u = a[0], v = a[1];
        f[0] *= u.x; f[1] *= u.y; f[2] *= u.z; f[3] *= u.w;
        f[4] *= v.x; f[5] *= v.y; f[6] *= v.z; f[7] *= v.w;
      }
      bf[c][4 * q + 0] = half2_bits(f[0] * lo, f[4] * lo);
      bf[c][4 * q + 1] = half2_bits(f[1] * hi, f[5] * hi);
      bf[c][4 * q + 2] = half2_bits(f[2] * lo, f[6] * lo);
      bf[c][4 * q + 3] = half2_bits(f[3] * hi, f[7] * hi);
    }
  return e.y;
}

template <bool kGated, bool kBf16>
__global__ void __launch_bounds__(fgv::kWarps * 32, 1) fused_gemv_kernel(const __grid_constant__ CUtensorMap tmP, const FusedGemvParams p) {
  using namespace fgv;
  extern __shared__ uint8_t gemv_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(gemv_smem) + 1023) & ~uintptr_t(1023));
  const int depth = p.depth;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kWarps * depth * kPiece);
  float *sPart = reinterpret_cast<float *>(bars + kWarps * depth);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int M = (int)p.M, Mp = (M + 1) & ~1;
  grid_launch_dependents();

  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t ranges = gridDim.x / p.cluster, range = blockIdx.x / p.cluster;
  const int64_t r0 = p.N * range / ranges;
  const int rows = (int)(p.N * (range + 1) / ranges - r0);
  const int nbh = (rows + 15) / 16, nb = kGated ? 2 * nbh : nbh;  // row blocks (gated: gate blocks, then up blocks)
  const int rsets = kWarps / p.ksw, kw = warp % p.ksw, rs = warp / p.ksw;
  const int Kg = (int)(p.K / kGroup), pieces = (Kg + C - 1) / C;
  // This CTA's pieces [q0, q1) go to its warps in turn, so that what the warps read at one
  // time is contiguous.
  const int q0 = (int)((int64_t)pieces * rank / p.cluster), q1 = (int)((int64_t)pieces * (rank + 1) / p.cluster);
  const int c0 = q0 + kw;
  const int mine = (nb - rs + rsets - 1) / rsets;  // this warp's row blocks
  const int total = mine > 0 && c0 < q1 ? mine * ((q1 - c0 + p.ksw - 1) / p.ksw) : 0;

  // The sequence: pieces of this warp's channels, and for each all its row blocks.  Group
  // `gr` of packed row n is number o = n Kg + gr (below 2^32): its scale and zero point
  // lie at o, its codes at 64 o.
  //
  // A piece is one TMA box of 16 rows (rows behind the range are read and dropped, bytes
  // behind a row's end are 0); its scales and zero points are loaded a piece ahead.
  uint8_t *ring = smem + warp * depth * kPiece;
  uint64_t *bar = bars + warp * depth;
  if (lane == 0)
    for (int i = 0; i < depth; ++i) mbar_init(&bar[i], 1);
  fence_barrier_init();
  __syncwarp();
  auto row_of = [&](int b) -> int {  // first packed row of a row block
    const bool up = kGated && b >= nbh;
    return (int)(r0 + (up ? p.N : 0)) + 16 * (up ? b - nbh : b);
  };
  int lblk = rs, lc = c0;  // next to load
  auto load = [&](int slot) {
    if (ftc::elect_one()) {
      mbar_arrive_expect_tx(&bar[slot], kPiece);
      tma_load_2d(ring + slot * kPiece, &tmP, &bar[slot], C * 64 * lc, row_of(lblk));
    }
    __syncwarp();
    lblk += rsets;
    if (lblk >= nb) lblk = rs, lc += p.ksw;
  };
  const bool even = (Kg & 1) == 0;
  uint32_t sz[2][2];     // scales, zeros of rows g, g + 8 of the piece: group c in half c
  const int last = rows - 1;
  auto load_sz = [&](int b, int c) {
    const int in = kGated && b >= nbh ? 16 * (b - nbh) : 16 * b;
    const uint32_t first = (uint32_t)row_of(b) * (uint32_t)Kg + (uint32_t)(C * c);
    const uint16_t *sp = p.scales + first, *zp = p.zeros + first;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r = (uint32_t)((g + 8 * h) * Kg);
      if (in + 15 > last) r = (uint32_t)(min(g + 8 * h, last - in) * Kg);  // the range ends in this block
      if (even) {
        sz[h][0] = ldg_u32(sp + r);
        sz[h][1] = ldg_u32(zp + r);
      } else {
        const uint32_t r1 = 2 * c + 1 < Kg ? r + 1 : r;
        sz[h][0] = ldg_u16(sp + r) | ldg_u16(sp + r1) << 16;
        sz[h][1] = ldg_u16(zp + r) | ldg_u16(zp + r1) << 16;
      }
    }
  };
  grid_dependency_wait();
  for (int i = 0; i < depth; ++i)
    if (i < total) load(i);
  if (total > 0) load_sz(rs, c0);

  uint32_t bf[C][16];        // B fragments
  float d1[C][2], inv[2];    // D1 and 2^-b of tokens 2t, 2t + 1
  int blk = rs, cc = c0, slot = 0;
  uint32_t ph = 0;
  bool ok = true;
  float *dst = sPart + ((size_t)(kw * p.nblk + blk) * 16 + g) * Mp + 2 * t;
  const int step = rsets * 16 * Mp;
  for (int it = 0; it < total; ++it) {
    if (blk == rs) {
      // a new piece of channels
      const int64_t ch = (int64_t)cc * C * kGroup + 32 * t;
      const float v = stage_b<kBf16>(p.X + (int64_t)g * p.K + ch, p.awq_s ? p.awq_s + ch : nullptr, g < M,
                                     Kg - 1 - C * cc, bf);
      inv[0] = __shfl_sync(~0u, v, 8 * t);
      inv[1] = __shfl_sync(~0u, v, 8 * t + 4);
      constexpr uint32_t one[4] = {0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float d[4];
#pragma unroll
        for (int q = 0; q < 8; ++q) mma(d, one, bf[c][2 * q], bf[c][2 * q + 1], q == 0);
        d1[c][0] = d[0];
        d1[c][1] = d[1];
      }
    }
    if (!ftc::wait_all(&bar[slot], ph, kErrTimeoutTma)) { ok = false; break; }
    uint4 w[C][2];
    const uint32_t at = smem_u32(ring + slot * kPiece) + g * (C * 64);  // row g + 8 has the same swizzle
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < C; ++c)
        w[c][h] = lds128_ordered(at + h * (8 * C * 64) + ((uint32_t)((4 * c + t) ^ g) << 4));
    float d[C][4], y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 u = w[c][0], v = w[c][1];
        const uint32_t l = q == 0 ? u.x : q == 1 ? u.y : q == 2 ? u.z : u.w, l8 = l >> 8;
        const uint32_t x = q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w, x8 = x >> 8;
        const uint32_t a0[4] = {l & 0x000F000Fu, x & 0x000F000Fu, l & 0x00F000F0u, x & 0x00F000F0u};
        const uint32_t a1[4] = {l8 & 0x000F000Fu, x8 & 0x000F000Fu, l8 & 0x00F000F0u, x8 & 0x00F000F0u};
        mma(d[c], a0, bf[c][4 * q], bf[c][4 * q + 1], q == 0);
        mma(d[c], a1, bf[c][4 * q + 2], bf[c][4 * q + 3], false);
      }
    // sums in units of 2^24, which the epilogue puts back
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2 sc = *reinterpret_cast<const __half2 *>(&sz[h][0]), zp = *reinterpret_cast<const __half2 *>(&sz[h][1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float v = __low2float(sc) * fmaf(-__low2float(zp), d1[0][x], d[0][2 * h + x]);
        y[2 * h + x] = fmaf(__high2float(sc), fmaf(-__high2float(zp), d1[1][x], d[1][2 * h + x]), v) * inv[x];
      }
    }
    // the slot was read (its values went through the MMAs above): refill it, and fetch the
    // next piece's constants
    if (it + depth < total) load(slot);
    if (++slot == depth) slot = 0, ph ^= 1u;
    {
      const bool turn = blk + rsets >= nb;
      if (it + 1 < total) load_sz(turn ? rs : blk + rsets, turn ? cc + p.ksw : cc);
    }
    if (2 * t < M) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 *q = reinterpret_cast<float2 *>(dst + 8 * h * Mp);
        float2 v = make_float2(y[2 * h], y[2 * h + 1]);
        if (cc != c0) {
          const float2 u = *q;
          v.x += u.x;
          v.y += u.y;
        }
        *q = v;
      }
    }
    blk += rsets;
    dst += step;
    if (blk >= nb) {
      blk = rs;
      cc += p.ksw;
      dst = sPart + ((size_t)(kw * p.nblk + blk) * 16 + g) * Mp + 2 * t;
    }
  }
  if (!ok) {  // a wait that ran out: give copies in flight time to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {}
  }
  __syncthreads();

  // ---- sums over the warps of a row block, in order (and over the cluster), and the epilogue
  const FusedEpi &e = p.epi;
  const int outs = rows * M;
  auto over_warps = [&](int tok, int r, int side) {
    const int b = (r >> 4) + side * nbh;
    const float *q = sPart + ((size_t)b * 16 + (r & 15)) * Mp + tok;
    float a = 0.0f;
    for (int k = 0; k < p.ksw; ++k) a += q[(size_t)k * p.nblk * 16 * Mp];
    return a * 16777216.0f;
  };
  float *sums = sPart + (size_t)p.ksw * p.nblk * 16 * Mp;
  if (p.cluster > 1) {
    for (int idx = threadIdx.x; idx < outs * (kGated ? 2 : 1); idx += kWarps * 32) {
      const int side = idx >= outs, i2 = side ? idx - outs : idx, tok = i2 / rows;
      sums[idx] = over_warps(tok, i2 - tok * rows, side);
    }
    cluster_sync_all();
  }
  auto total_of = [&](int idx, int tok, int r, int side) {
    if (p.cluster == 1) return over_warps(tok, r, side);
    float a = 0.0f;
    for (int c = 0; c < p.cluster; ++c) a += ld_cluster(sums + idx + side * outs, c);
    return a;
  };
  for (int idx = threadIdx.x + rank * kWarps * 32; idx < outs; idx += kWarps * 32 * p.cluster) {
    const int tok = idx / rows, r = idx - tok * rows;
    const int64_t n = r0 + r, at = (int64_t)tok * p.N + n;
    float z = total_of(idx, tok, r, 0) + (e.bias ? e.bias[n] : 0.0f);
    if constexpr (kGated) {
      const float u = total_of(idx, tok, r, 1) + (e.bias ? e.bias[p.N + n] : 0.0f);
      if (e.Z) {
        store_from_float(e.Z, e.z_dtype, (int64_t)tok * 2 * p.N + n, z);
        store_from_float(e.Z, e.z_dtype, (int64_t)tok * 2 * p.N + p.N + n, u);
      }
      z = act_fwd(z, e.act) * u;
    } else {
      if (e.Z) store_from_float(e.Z, e.z_dtype, at, z);
      z = act_fwd(z, e.act);
      if (e.residual) z += load_as_float(e.residual, e.y_dtype, at);
    }
    store_from_float(e.Y, e.y_dtype, at, z);
  }
  if (p.cluster > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
}

// Largest number of clusters of this size that one kernel of a CTA per SM can run at a time.
int fused_gemv_clusters(int cluster, int sm) {
  static std::atomic<int> known[kAttrDevices][3];
  if (cluster == 1) return sm;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kAttrDevices) return sm / cluster;
  std::atomic<int> &k = known[dev][cluster == 2 ? 0 : cluster == 4 ? 1 : 2];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm / cluster * cluster));
    cfg.blockDim = dim3(fgv::kWarps * 32);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fused_gemv_kernel<false, true>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = sm / cluster;
    }
    k.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <bool kGated, bool kBf16>
cudaError_t launch_fused_gemv_t(const CUtensorMap &tmP, const FusedGemvParams &p, int grid, cudaStream_t s) {
  static std::atomic<int> attr[kAttrDevices];
  const int smem = fgv::smem_bytes(p.ksw, p.nblk, (int)p.M, p.cluster, p.depth);
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fused_gemv_kernel<kGated, kBf16>), smem, attr);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(fgv::kWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fused_gemv_kernel<kGated, kBf16>, tmP, p);
}

cudaError_t launch_fused_gemv(const CUtensorMap &tmP, const FusedGemvParams &p, bool gated, bool bf16, int grid, cudaStream_t s) {
  return gated ? (bf16 ? launch_fused_gemv_t<true, true>(tmP, p, grid, s) : launch_fused_gemv_t<true, false>(tmP, p, grid, s))
               : (bf16 ? launch_fused_gemv_t<false, true>(tmP, p, grid, s) : launch_fused_gemv_t<false, false>(tmP, p, grid, s));
}

}  // namespace w4
