// fused_skinny.cu -- w4a16_linear and w4a16_gated for 9 to 64 tokens (groups of 128) on the
// 5th-generation tensor cores: bound by the weights' bytes.
//
// As in fused_tc.cu a weight becomes fp16 (q - z) * scale * r, rounded once (2^-11), in
// tensor memory, and the MMAs sum over all of K: 13 instructions per eight weights and
// nothing per group.  (Codes as exact subnormals, five instructions, with scale and zero
// point applied to each group's sums in fp32 took more: the sums' way out of tensor memory
// cost its warps 750 cycles a group, and at 48 tokens the whole SM's issue slots.)  What
// differs is the weights' way in:
//   * A CTA (one per SM) owns an equal range of output rows, as tiles of at most 128 rows
//     (64 gate and 64 up rows), over all of K, so that nothing is summed afterwards; where
//     that would leave most MMA rows empty, a cluster of 2, 4 or 8 CTAs shares a range and
//     splits K, and their sums meet through distributed shared memory.
//   * Codes come as 256 contiguous bytes of a row (4 groups): HBM gave 2.5 TB/s at most on
//     64-byte pieces, however many were in flight.
//   * A row's factor r (a power of two that brings its largest scale into [2^10, 2^11)) is
//     found by the threads that own the row: there is no pass over the scales before.
// An MMA of 128 rows takes 23 ns with 16 tokens and 28 ns with 64 (measured), eight of them
// a group of 128 x 128: 183 to 224 ns, where the group's bytes take 193 ns of an SM's HBM.
//
// Roles (768 threads): warp 0 loads activations (TMA), warp 1 codes (TMA), warp 2 issues the
// MMAs, warp 3 owns TMEM, warps 4..7 write results, warps 8..23 convert in four sets that
// take turns, a group and an A buffer each.
//
// Measured with 16 / 48 tokens, staging included, back to back in a graph: 11.9 / 13.8 us at
// 4096 x 4096, 22.7 / 24.4 us at 14336 -> 4096, 30.7 / 32.2 us for the gated 4096 -> 2 x
// 14336, 96 / 102 us for 8192 -> 2 x 28672 (250 MB, 2.6 TB/s).  Bound: the converting warps'
// issue slots, and the start.  At 48 tokens, gated 4096 -> 2 x 14336, counters give 33,100
// instructions to each of an SM's four schedulers in 53,800 active cycles: some 520 slots
// for each of a CTA's 64 (tile, group) blocks, waits that poll included, where the bytes of
// its 98 rows take some 280 cycles of an SM's HBM; the tensor pipe is active for 23 %.  What
// the other 20,700 cycles are (the first loads, the end, warps that all wait) was not taken
// apart.
#include "act.cuh"
#include "code_ring.cuh"
#include "common.cuh"

namespace w4 {

struct FusedSkinnyParams {
  FusedEpi epi;            // M, N (F for gated), bias, residual, Z, Y; tinv per token
  const uint16_t *scales, *zeros;
  int groups;              // K / 128
  int tile_rows;           // rows (gated: gate rows) of the longest tile
  int tiles;               // tiles of a range
  int cluster;             // CTAs that share a range and split K
  int code_stages;
};

namespace fsk {

constexpr int kThreads = 32 * (8 + 4 * kSets);
// A stage of codes: 128 rows x 4 groups, as two boxes of 128-byte rows.
constexpr int kCodeBox = 128 * 128, kCodeStage = 2 * kCodeBox;
static_assert(kCodeGroups == 4, "two boxes of two groups");
constexpr int kMaxStages = 8, kMaxCodeStages = 5;
constexpr int kMaxTokens = 64;
constexpr int kRowFactors = 16;  // tiles whose row factors are kept: conversion may be 8 groups, and so as many
                                  // tiles, in front of the products, and those 2 tiles in front of the results

__host__ __device__ constexpr int act_stage(int bn) { return bn * 256; }  // 128 channels
__host__ __device__ constexpr int stages(int bn) { return bn > 48 ? 5 : bn > 32 ? 6 : kMaxStages; }
// Everything but the codes' ring.
__host__ __device__ constexpr int fixed_bytes(int bn, int m, int tiles, int cluster) {
  return 1024 + stages(bn) * act_stage(bn) + kRowFactors * 128 * 4 + kMaxTokens * 4 + (cluster > 1 ? tiles : 1) * m * 128 * 4 +
         (2 * kMaxStages + 2 * kMaxCodeStages + 4) * 8;
}
// Stages of the codes' ring: as many as fit, since they are the bytes in flight.
__host__ __device__ constexpr int code_stages(int bn, int m, int tiles, int cluster) {
  const int n = (227 * 1024 - fixed_bytes(bn, m, tiles, cluster)) / kCodeStage;
  return n > kMaxCodeStages ? kMaxCodeStages : n;
}

}  // namespace fsk

// Blocks 0..bn-1: one token each (zeros behind the last).  x' as in fused_stage_x, as
// [K / 64][bn][64] fp16; 1 / 2^b.
template <bool kBf16>
__global__ void __launch_bounds__(1024)
    fused_stage_small(const uint16_t *X, const float *awq_s, int64_t M, int64_t K, int bn, uint16_t *xp, float *tinv) {
  grid_launch_dependents();
  __shared__ float red[32];
  const int64_t m = blockIdx.x, nv = K / 8;
  const bool real = m < M;
  const uint4 *row = reinterpret_cast<const uint4 *>(X + m * K);
  auto scaled = [&](int64_t v, float (&f)[8]) {
    unpack8<kBf16>(real ? row[v] : make_uint4(0, 0, 0, 0), f);
    if (awq_s) {
      const float4 a = reinterpret_cast<const float4 *>(awq_s)[2 * v], b = reinterpret_cast<const float4 *>(awq_s)[2 * v + 1];
      f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
      f[4] *= b.x; f[5] *= b.y; f[6] *= b.z; f[7] *= b.w;
    }
  };
  float mx = 0.0f;
  if (real)
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
      float f[8];
      scaled(v, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(f[j]));
    }
  const float2 e = pow2_to(block_max(mx, red), 13);
  if (threadIdx.x == 0) tinv[m] = e.y;
#pragma unroll 4
  for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
    float f[8];
    scaled(v, f);
    *reinterpret_cast<uint4 *>(xp + ((v >> 3) * bn + m) * 64 + (v & 7) * 8) =
        make_uint4(half2_bits(f[0] * e.x, f[4] * e.x), half2_bits(f[1] * e.x, f[5] * e.x),
                   half2_bits(f[2] * e.x, f[6] * e.x), half2_bits(f[3] * e.x, f[7] * e.x));
  }
}

// Reads 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Outputs of a tile from its sums [token][128] (of every CTA of the cluster): thread `id` of
// `n` threads.
template <bool kGated>
__device__ __forceinline__ void skinny_finish(const FusedEpi &e, const float *sums, int64_t row, int rows, int id, int n,
                                              int cluster, int remote) {
  constexpr int kRow = kGated ? 64 : 128;
  auto sum_at = [&](int i) {
    if (!remote) return sums[i];
    float a = 0.0f;
    for (int c = 0; c < cluster; ++c) a += fgv::ld_cluster(sums + i, c);
    return a;
  };
  const int r = id % kRow;
  if (r >= rows) return;
  const int64_t col = row + r;
  const float bz = e.bias ? e.bias[col] : 0.0f, bu = kGated && e.bias ? e.bias[e.N + col] : 0.0f;
#pragma unroll 4
  for (int tok = id / kRow; tok < (int)e.M; tok += n / kRow) {
    const int64_t at = (int64_t)tok * e.N + col;
    float z = sum_at(tok * 128 + r) + bz;
    if constexpr (kGated) {
      const float u = sum_at(tok * 128 + 64 + r) + bu;
      if (e.Z) {
        store_from_float(e.Z, e.z_dtype, (int64_t)tok * 2 * e.N + col, z);
        store_from_float(e.Z, e.z_dtype, (int64_t)tok * 2 * e.N + e.N + col, u);
      }
      z = act_fwd(z, e.act) * u;
    } else {
      if (e.Z) store_from_float(e.Z, e.z_dtype, at, z);
      z = act_fwd(z, e.act);
      if (e.residual) z += load_as_float(e.residual, e.y_dtype, at);
    }
    store_from_float(e.Y, e.y_dtype, at, z);
  }
}

// The largest size among `n` fp16 scales.
__device__ __forceinline__ float max_scale(const uint16_t *p, int n) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = 0;
  int i = 0;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0)
#pragma unroll 4
    for (; i + 8 <= n; i += 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + i));
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs)));
    }
  m = max(m >> 16, m & 0xFFFFu);
  for (; i < n; ++i) m = max(m, (uint32_t)__ldg(p + i) & 0x7FFFu);
  return half_bits_to_float((uint16_t)m);
}

// T: tokens / 16, rounded up.
template <int T, bool kGated>
__global__ void __launch_bounds__(fsk::kThreads, 1)
    fused_skinny_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmP,
                        const FusedSkinnyParams p) {
  using namespace fsk;
  constexpr int BN = 16 * T, NS = stages(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nc = p.code_stages;
  uint8_t *sC = smem, *sX = sC + nc * kCodeStage;
  float *sR = reinterpret_cast<float *>(sX + NS * act_stage(BN));  // 1 / r by tile and row
  float *sTok = sR + kRowFactors * 128;                            // 1 / 2^b per token
  float *sums = sTok + kMaxTokens;                                 // [tile (cluster) or one][token][128]
  const FusedEpi &e = p.epi;
  const int M = (int)e.M;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sums + (size_t)(p.cluster > 1 ? p.tiles : 1) * M * 128);
  uint64_t *full = bars, *done = full + NS;
  uint64_t *cfull = done + NS, *cempty = cfull + kMaxCodeStages;
  uint64_t *dfull = cempty + kMaxCodeStages, *dempty = dfull + 2;
  __shared__ uint32_t holder;

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1 + 128);  // activations, and the set that converts the group
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < nc; ++i) {
      mbar_init(&cfull[i], 1);
      mbar_init(&cempty[i], 128 * kSets);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 128);
    }
    fence_barrier_init();
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmP);
  }
  if (warp == 3) {
    tmem_alloc(&holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = holder;

  const int rank = p.cluster > 1 ? (int)fgv::cluster_rank() : 0;
  const int64_t ranges = gridDim.x / p.cluster, range = blockIdx.x / p.cluster;
  const int64_t r0 = e.N * range / ranges, r1 = e.N * (range + 1) / ranges;
  const int g0 = (int)((int64_t)p.groups * rank / p.cluster), g1 = (int)((int64_t)p.groups * (rank + 1) / p.cluster);
  const int ng = g1 - g0, total = ng * p.tiles;  // (tile, group) in order, tile by tile
  // First row of tile i of the range; tiles of equal length, at most tile_rows each.
  auto tile_row = [&](int i) -> int64_t { return r0 + (r1 - r0) * i / p.tiles; };
  bool ok = true;

  if (warp == 0) {
    grid_dependency_wait();
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0, g = g0; i < total; ++i) {
      if (!ftc::wait_all(&done[s], ph ^ 1u, kErrTimeoutTma)) { ok = false; break; }
      if (ftc::elect_one()) {
        mbar_arrive_expect_tx(&full[s], (uint32_t)act_stage(BN));
        tma_load_2d(sX + s * act_stage(BN), &tmX, &full[s], 0, g * 2 * BN);
      }
      __syncwarp();
      if (++s == NS) s = 0, ph ^= 1u;
      if (++g == g1) g = g0;
    }
  } else if (warp == 1) {
    // the weights do not come from the staging kernel, and what was before it has ended
    int s = 0;
    uint32_t ph = 0;
    const int box = p.tile_rows * 128, half = kGated ? 64 * 128 : 0;
    for (int tile = 0; ok && tile < p.tiles; ++tile) {
      const int row = (int)tile_row(tile);
      for (int g = g0; g < g1; g += kCodeGroups) {
        if (!ftc::wait_all(&cempty[s], ph ^ 1u, kErrTimeoutTma)) { ok = false; break; }
        const int boxes = g + 2 < g1 ? 2 : 1;
        if (ftc::elect_one()) {
          mbar_arrive_expect_tx(&cfull[s], (uint32_t)(boxes * box * (kGated ? 2 : 1)));
          uint8_t *dst = sC + s * kCodeStage;
          for (int b = 0; b < boxes; ++b) {
            tma_load_2d(dst + b * kCodeBox, &tmP, &cfull[s], (g + 2 * b) * 64, row);
            if (kGated) tma_load_2d(dst + b * kCodeBox + half, &tmP, &cfull[s], (g + 2 * b) * 64, (int)e.N + row);
          }
        }
        __syncwarp();
        if (++s == nc) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 2) {
    const uint32_t idesc = idesc_f16(false, BN);
    int s = 0, a = 0, d = 0;
    uint32_t ph = 0, dph = 0;
    bool ready = false;  // the group's barrier was seen complete while the last one was issued
    for (int tile = 0; ok && tile < p.tiles; ++tile) {
      if (!ftc::wait_all(&dempty[d], dph ^ 1u, kErrTimeoutMma)) { ok = false; break; }
      const uint32_t acc = tmem + (uint32_t)(64 * kSets + d * BN);
      for (int g = g0; g < g1; ++g) {
        if (!ready && !ftc::wait_all(&full[s], ph, kErrTimeoutMma)) { ok = false; break; }
        tc_fence_after();
        const uint64_t bd = smem_desc_k_sw128(smem_u32(sX + s * act_stage(BN)));
        uint64_t *fin = &done[s];
        if (++s == NS) s = 0, ph ^= 1u;
        ready = __all_sync(~0u, ftc::mbar_test(&full[s], ph));
        if (ftc::elect_one()) {
          const uint32_t at = tmem + (uint32_t)(64 * a);
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 64 channels per 128-byte tile of BN rows
            tc_mma_ts(acc, at + 8 * j, bd + (uint64_t)((j >> 2) * (BN * 128 / 16) + 2 * (j & 3)), idesc,
                      g > g0 || j > 0 ? 1u : 0u);
          tc_commit(fin);
          if (g == g1 - 1) tc_commit(&dfull[d]);
        }
        __syncwarp();
        if (++a == kSets) a = 0;
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
  } else if (warp >= 8) {
    // ---- conversion: set j takes groups j, j + 4, ... of the CTA's sequence
    const int set = (warp - 8) >> 2, wq = warp & 3, r = 32 * wq + lane;
    const uint32_t at = tmem + ((uint32_t)(32 * wq) << 16) + (uint32_t)(64 * set);
    const uint32_t sw = (uint32_t)(r & 7);
    int s = set, ps = 0;
    uint32_t pph = 0, sph = 0;
    CodeWalk walk(set, ng, nc);
    int tile = -1;
    float rf = 0.0f;
    const uint16_t *sp = p.scales, *zp = p.zeros;
    uint32_t scn = 0, zn = 0;
    for (int i = set; i < total; i += kSets, walk.next()) {
      const int gi = walk.group;
      if (walk.tile != tile) {
        // this thread's row of the tile: its factor, and where its constants lie
        tile = walk.tile;
        const int64_t row = tile_row(tile);
        const int rows = (int)(tile_row(tile + 1) - row), f = kGated ? r & 63 : r;
        const int64_t n = row + (f < rows ? f : 0) + (kGated && r >= 64 ? e.N : 0);
        sp = p.scales + n * p.groups + g0;
        zp = p.zeros + n * p.groups + g0;
        scn = fgv::ldg_u16(sp + gi);
        zn = fgv::ldg_u16(zp + gi);
        const float2 rr = pow2_to(max_scale(sp, ng), 10);
        rf = rr.x;
        // (whichever set starts a tile writes the same values)
        sR[(tile % kRowFactors) * 128 + r] = rr.y;
      }
      if (!walk.reach([&](int c, uint32_t ph) { return ftc::wait_all(&cfull[c], ph, kErrTimeoutDequant); },
                      [&](int c) { mbar_arrive(&cempty[c]); })) { ok = false; break; }
      const int sub = gi % kCodeGroups;
      const uint32_t base = smem_u32(sC + walk.slot * kCodeStage + (sub >> 1) * kCodeBox) + (uint32_t)(r * 128);
      const uint32_t c0 = (uint32_t)(4 * (sub & 1));
      ftc::GroupK k;
      {
        const __half2 h = __floats2half2_rn(half_bits_to_float((uint16_t)scn) * rf, 1024.0f + half_bits_to_float((uint16_t)zn));
        k.set(*reinterpret_cast<const uint32_t *>(&h));
      }
      if (gi + kSets < ng) {
        scn = fgv::ldg_u16(sp + gi + kSets);
        zn = fgv::ldg_u16(zp + gi + kSets);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q0 = lds128(base + (((c0 + 2 * h) ^ sw) << 4)), q1 = lds128(base + (((c0 + 2 * h + 1) ^ sw) << 4));
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t out[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t o[4];
          ftc::dequant8(w[j], k, o);
#pragma unroll
          for (int x = 0; x < 4; ++x) out[4 * j + x] = o[x];
        }
        // the buffer is free once this set's last group has been multiplied
        if (h == 0 && i >= kSets && !ftc::wait_all(&done[ps], pph, kErrTimeoutDequant)) { ok = false; break; }
        if (h == 0) tc_fence_after();
        tmem_st_32x32b_x32(at + 32 * h, out);
      }
      if (!ok) break;
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&full[s]);
      mbar_arrive(&cempty[walk.slot]);
      walk.leave();
      ps = s;
      pph = sph;
      s += kSets;
      if (s >= NS) s -= NS, sph ^= 1u;
    }
  } else if (warp >= 4) {
    // ---- results: the tile's sums into shared memory as [token][row], and (without a
    // cluster) its epilogue
    const int r = 32 * (warp & 3) + lane;
    grid_dependency_wait();
    if (r < M) sTok[r] = e.tinv[r];
    int d = 0;
    uint32_t dph = 0;
    for (int tile = 0; tile < p.tiles; ++tile) {
      ok = ftc::vote_epilogue(mbar_wait(&dfull[d], dph, kErrTimeoutEpilogue));
      if (!ok) break;
      tc_fence_after();
      const float rinv = sR[(tile % kRowFactors) * 128 + r];
      float *to = sums + (size_t)(p.cluster > 1 ? tile : 0) * M * 128 + r;
      const uint32_t src = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(64 * kSets + d * BN);
#pragma unroll
      for (int c = 0; c < T; ++c) {
        uint32_t v[16];
        tmem_ld_cols(src + 16 * c, v);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (16 * c + j < M) to[(16 * c + j) * 128] = __uint_as_float(v[j]) * rinv * sTok[16 * c + j];
      }
      tc_fence_before();
      mbar_arrive(&dempty[d]);
      // (the last tile, whose results nothing hides: by all threads, below)
      if (p.cluster == 1 && tile < p.tiles - 1) {
        ftc::bar_epilogue();
        const int64_t row = tile_row(tile);
        skinny_finish<kGated>(e, sums, row, (int)(tile_row(tile + 1) - row), (int)threadIdx.x - 128, 128, 1, 0);
        ftc::bar_epilogue();  // the sums are read until here
      }
      d ^= 1;
      if (d == 0) dph ^= 1u;
    }
  }
  if (!ok) {  // a wait that ran out: give copies in flight time to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {}
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (p.cluster == 1) {
    const int64_t row = tile_row(p.tiles - 1);
    skinny_finish<kGated>(e, sums, row, (int)(r1 - row), (int)threadIdx.x, kThreads, 1, 0);
    return;
  }
  fgv::cluster_sync_all();
  for (int tile = 0; tile < p.tiles; ++tile) {
    const int64_t row = tile_row(tile);
    skinny_finish<kGated>(e, sums + (size_t)tile * M * 128, row, (int)(tile_row(tile + 1) - row),
                          rank * kThreads + (int)threadIdx.x, p.cluster * kThreads, p.cluster, 1);
  }
  fgv::cluster_sync_all();  // no CTA leaves while another reads its sums
}

cudaError_t launch_fused_stage_small(const void *X, bool bf16, const float *awq_s, int64_t M, int64_t K, int bn, uint16_t *xp,
                                     float *tinv, cudaStream_t s) {
  const uint16_t *x = static_cast<const uint16_t *>(X);
  const int threads = K >= 8192 ? 1024 : K >= 4096 ? 512 : 256;  // two vectors or so to a thread
  if (bf16) fused_stage_small<true><<<bn, threads, 0, s>>>(x, awq_s, M, K, bn, xp, tinv);
  else fused_stage_small<false><<<bn, threads, 0, s>>>(x, awq_s, M, K, bn, xp, tinv);
  return cudaGetLastError();
}

template <int T, bool kGated>
cudaError_t launch_fused_skinny_t(const CUtensorMap &tmX, const CUtensorMap &tmP, const FusedSkinnyParams &p, int grid,
                                  cudaStream_t s) {
  static std::atomic<int> attr[kAttrDevices];
  const int smem = fsk::fixed_bytes(16 * T, (int)p.epi.M, p.tiles, p.cluster) + p.code_stages * fsk::kCodeStage;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fused_skinny_kernel<T, kGated>), smem, attr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(fsk::kThreads);
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
  return cudaLaunchKernelEx(&cfg, fused_skinny_kernel<T, kGated>, tmX, tmP, p);
}

cudaError_t launch_fused_skinny(const CUtensorMap &tmX, const CUtensorMap &tmP, const FusedSkinnyParams &p, bool gated,
                                int grid, cudaStream_t s) {
  switch ((p.epi.M + 15) / 16) {
    case 1: return gated ? launch_fused_skinny_t<1, true>(tmX, tmP, p, grid, s) : launch_fused_skinny_t<1, false>(tmX, tmP, p, grid, s);
    case 2: return gated ? launch_fused_skinny_t<2, true>(tmX, tmP, p, grid, s) : launch_fused_skinny_t<2, false>(tmX, tmP, p, grid, s);
    case 3: return gated ? launch_fused_skinny_t<3, true>(tmX, tmP, p, grid, s) : launch_fused_skinny_t<3, false>(tmX, tmP, p, grid, s);
    default: return gated ? launch_fused_skinny_t<4, true>(tmX, tmP, p, grid, s) : launch_fused_skinny_t<4, false>(tmX, tmP, p, grid, s);
  }
}

}  // namespace w4
