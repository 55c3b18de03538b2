// fused_gemv.cu -- w4a16_linear and w4a16_gated for up to 16 tokens (groups of 128), in one
// kernel without workspace: the call reads every weight once and is bound by that.
//
// A CTA (one per SM) owns an equal range of output rows, whatever its length, so that
// every SM streams the same number of bytes; the row blocks of 16 that mma.sync works on
// may end anywhere (rows behind the range are the last one again, and dropped).  Inside
// the CTA the warps split K: a warp walks over the CTA's row blocks with the activations
// of its own channels, as B fragments, in registers.  So the main loop has no barrier, no
// shared memory and no traffic but the weights: 16-byte loads from global memory straight
// into the A fragments' owners, two (row block, 256-channel) pieces ahead, 64 KB in
// flight per SM.  The warps' partial sums meet in shared memory once, at the end, in a
// fixed order, where bias, activation, product and residual follow.
//
// Arithmetic (exact up to fp32 sums):  a code is used as it lies, as the fp16 subnormal
// q 2^-24 (low nibbles, one AND per pair) or 16 q 2^-24 (high nibbles; their activations
// are divided by 16).  Per group, with D the MMA's sum and S the sum of the activations,
//   sum (q - z) x' = 2^24 (D - z 2^-24 S),   y += (scale 2^24) (D - (z 2^-24) S),
// five instructions per eight weights where subtracting z from every pair takes nine.
// x' = x s 2^b, b per token and warp with the largest |x'| of the warp's channels in
// [2^13, 2^14): bf16 and fp16 convert exactly, x * s is rounded to fp16 once.
//
// Fragments (g = lane / 4, t = lane % 4): lane (g, t) loads the 32 codes of channels
// 32 t .. 32 t + 31 of rows g and g + 8 of a group; word w of them feeds two MMAs, whose k
// order is the same permutation on both sides: channels 32 t + 8 w + {0, 4, 1, 5} and
// {2, 6, 3, 7}.
#include "act.cuh"
#include "common.cuh"

namespace w4 {

struct FusedGemvParams {
  const uint16_t *X;
  int64_t M, N, K;          // N: output columns (F for gated)
  const uint8_t *packed;
  const uint16_t *scales, *zeros;
  const float *awq_s;
  FusedEpi epi;
  int ksw;                  // warps that split K
  int nblk;                 // row blocks of the longest CTA range (gated: gate and up)
};

namespace fgv {

constexpr int kWarps = 16;
constexpr int kMaxTokens = 16;
constexpr int kSmemMax = 220 * 1024;

__host__ __device__ constexpr int smem_bytes(int ksw, int nblk, int m) {
  return ksw * nblk * 16 * m * 4 + kWarps * kMaxTokens * 4;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t ldg_u16(const uint16_t *p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

}  // namespace fgv

// T octets of tokens; C groups per piece (C = 2 for one octet, so that its B fragments, 32
// registers, and two pieces of weights in flight fit 128 registers; C = 1 for two octets).
template <int T, bool kGated, bool kBf16>
__global__ void __launch_bounds__(fgv::kWarps * 32, 1) fused_gemv_kernel(const FusedGemvParams p) {
  using namespace fgv;
  constexpr int C = T == 1 ? 2 : 1;
  constexpr int P = T == 1 ? 2 : 4;  // pieces in flight
  extern __shared__ __align__(16) float sPart[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int M = (int)p.M;
  float *sInv = sPart + (size_t)p.ksw * p.nblk * 16 * M;  // [warp][token] 2^-b
  grid_launch_dependents();

  const int64_t r0 = p.N * blockIdx.x / gridDim.x, r1 = p.N * (blockIdx.x + 1) / gridDim.x;
  const int nb = (int)((r1 - r0 + 15) / 16) * (kGated ? 2 : 1);  // row blocks (gated: gate, up, gate, ...)
  const int rsets = kWarps / p.ksw, kw = warp % p.ksw, rs = warp / p.ksw;
  const int Kg = (int)(p.K / kGroup), pieces = (Kg + C - 1) / C;
  const int c0 = (int)((int64_t)pieces * kw / p.ksw), c1 = (int)((int64_t)pieces * (kw + 1) / p.ksw);
  const int mine = (nb - rs + rsets - 1) / rsets;  // this warp's row blocks
  const int total = mine > 0 ? mine * (c1 - c0) : 0;

  // Packed rows g and g + 8 of row block `blk`.
  auto row_of = [&](int blk, int half) -> int64_t {
    const int j = kGated ? blk >> 1 : blk;
    int64_t r = r0 + 16 * j + g + 8 * half;
    r = r < r1 ? r : r1 - 1;
    return kGated && (blk & 1) ? p.N + r : r;
  };
  const int64_t rowb = p.K / 2;
  // The sequence: pieces of this warp's channels, and for each all its row blocks.
  uint4 w[P][C][2];
  uint32_t sz[P][C][2][2];  // scale, zero of rows g, g + 8
  int li = 0, lc = c0;      // next to load
  auto load = [&](int slot) {
    const int blk = rs + li * rsets;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = row_of(blk, h);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int gr = min(C * lc + c, Kg - 1);  // behind the last group: that one again, its activations are 0
        w[slot][c][h] = ldg_nc_v4(p.packed + n * rowb + gr * 64 + t * 16);
        sz[slot][c][h][0] = ldg_u16(p.scales + n * Kg + gr);
        sz[slot][c][h][1] = ldg_u16(p.zeros + n * Kg + gr);
      }
    }
    if (++li == mine) li = 0, ++lc;
  };
  // While the kernel before this one ends: the first pieces on their way into L2 (a hint,
  // which reads nothing; what that kernel writes is read behind the wait only).
  if (total > 0)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.packed + row_of(rs, 0) * rowb + (int64_t)c0 * C * 64 + t * 16));
  grid_dependency_wait();
#pragma unroll
  for (int s = 0; s < P; ++s)
    if (s < total) load(s);

  // ---- activations: the power of two of each token over this warp's channels
  float scl[T];
#pragma unroll
  for (int o = 0; o < T; ++o) {
    const int tok = 8 * o + g;
    float mx = 0.0f;
    if (tok < M)
      for (int ch = c0 * C * kGroup + 8 * t; ch < min(c1 * C, Kg) * kGroup; ch += 32) {
        float f[8];
        unpack8<kBf16>(*reinterpret_cast<const uint4 *>(p.X + tok * p.K + ch), f);
        if (p.awq_s) {
          const float4 a = *reinterpret_cast<const float4 *>(p.awq_s + ch), b = *reinterpret_cast<const float4 *>(p.awq_s + ch + 4);
          f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
          f[4] *= b.x; f[5] *= b.y; f[6] *= b.z; f[7] *= b.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(f[j]));
      }
    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
    const float2 e = pow2_to(mx, 13);
    scl[o] = e.x;
    if (t == 0) sInv[warp * kMaxTokens + tok] = e.y;
  }

  uint32_t bf[C][T][16];  // B fragments: [word][MMA of the word][register]
  float S[C][T][2];       // sums of x' of tokens 2t, 2t + 1 over the group
  int i = 0, cc = c0;
  for (int it = 0; it < total; it += P) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      if (it + s >= total) break;
      if (i == 0) {
        // a new piece of channels: its activations become B fragments
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int o = 0; o < T; ++o) {
            const int tok = 8 * o + g, gr = C * cc + c;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float f[8] = {};
              if (tok < M && gr < Kg) {
                const int64_t ch = (int64_t)gr * kGroup + 32 * t + 8 * q;
                unpack8<kBf16>(*reinterpret_cast<const uint4 *>(p.X + tok * p.K + ch), f);
                if (p.awq_s) {
                  const float4 a = *reinterpret_cast<const float4 *>(p.awq_s + ch),
                               b = *reinterpret_cast<const float4 *>(p.awq_s + ch + 4);
                  f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
                  f[4] *= b.x; f[5] *= b.y; f[6] *= b.z; f[7] *= b.w;
                }
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                f[j] = __half2float(__float2half_rn(f[j] * scl[o]));
                sum += f[j];
              }
              // odd channels sit in the high nibbles: x' / 16 (a subnormal keeps its
              // leading bits: at most 2^-25 of the token's largest value 2^13 goes)
              bf[c][o][4 * q + 0] = half2_bits(f[0], f[4]);
              bf[c][o][4 * q + 1] = half2_bits(f[1] * 0.0625f, f[5] * 0.0625f);
              bf[c][o][4 * q + 2] = half2_bits(f[2], f[6]);
              bf[c][o][4 * q + 3] = half2_bits(f[3] * 0.0625f, f[7] * 0.0625f);
            }
            sum += __shfl_xor_sync(~0u, sum, 1);
            sum += __shfl_xor_sync(~0u, sum, 2);
            S[c][o][0] = __shfl_sync(~0u, sum, 8 * t);
            S[c][o][1] = __shfl_sync(~0u, sum, 8 * t + 4);
          }
      }
      float y[T][4] = {};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t wl[4] = {w[s][c][0].x, w[s][c][0].y, w[s][c][0].z, w[s][c][0].w};
        const uint32_t wh[4] = {w[s][c][1].x, w[s][c][1].y, w[s][c][1].z, w[s][c][1].w};
        float d[T][4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t l8 = wl[q] >> 8, h8 = wh[q] >> 8;
          const uint32_t a0[4] = {wl[q] & 0x000F000Fu, wh[q] & 0x000F000Fu, wl[q] & 0x00F000F0u, wh[q] & 0x00F000F0u};
          const uint32_t a1[4] = {l8 & 0x000F000Fu, h8 & 0x000F000Fu, l8 & 0x00F000F0u, h8 & 0x00F000F0u};
#pragma unroll
          for (int o = 0; o < T; ++o) {
            mma(d[o], a0, bf[c][o][4 * q], bf[c][o][4 * q + 1]);
            mma(d[o], a1, bf[c][o][4 * q + 2], bf[c][o][4 * q + 3]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sc = half_bits_to_float((uint16_t)sz[s][c][h][0]) * 16777216.0f;
          const float z = half_bits_to_float((uint16_t)sz[s][c][h][1]) * -5.9604644775390625e-8f;
#pragma unroll
          for (int o = 0; o < T; ++o) {
            y[o][2 * h] = fmaf(sc, fmaf(z, S[c][o][0], d[o][2 * h]), y[o][2 * h]);
            y[o][2 * h + 1] = fmaf(sc, fmaf(z, S[c][o][1], d[o][2 * h + 1]), y[o][2 * h + 1]);
          }
        }
      }
      if (it + s + P < total) load(s);
      const int blk = rs + i * rsets;
      float *dst = sPart + (size_t)(kw * p.nblk + blk) * 16 * M;
#pragma unroll
      for (int o = 0; o < T; ++o)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int tok = 8 * o + 2 * t + x;
            if (tok < M) {
              float *q = dst + tok * 16 + g + 8 * h;
              *q = cc == c0 ? y[o][2 * h + x] : *q + y[o][2 * h + x];
            }
          }
      if (++i == mine) i = 0, ++cc;
    }
  }
  __syncthreads();

  // ---- sums over the warps of a row block, in order, and the epilogue
  const FusedEpi &e = p.epi;
  const int rows = (int)(r1 - r0);
  for (int idx = threadIdx.x; idx < rows * M; idx += kWarps * 32) {
    const int tok = idx / rows, r = idx - tok * rows;
    auto total_of = [&](int side) {
      const int blk = kGated ? 2 * (r >> 4) + side : r >> 4, set = blk % rsets;
      float a = 0.0f;
      for (int k = 0; k < p.ksw; ++k)
        a += sPart[((size_t)(k * p.nblk + blk) * M + tok) * 16 + (r & 15)] * sInv[(set * p.ksw + k) * kMaxTokens + tok];
      return a;
    };
    const int64_t n = r0 + r, at = (int64_t)tok * p.N + n;
    float z = total_of(0) + (e.bias ? e.bias[n] : 0.0f);
    if constexpr (kGated) {
      const float u = total_of(1) + (e.bias ? e.bias[p.N + n] : 0.0f);
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
}

template <int T, bool kGated, bool kBf16>
cudaError_t launch_fused_gemv_t(const FusedGemvParams &p, int grid, cudaStream_t s) {
  static std::atomic<int> attr[kAttrDevices];
  const int smem = fgv::smem_bytes(p.ksw, p.nblk, (int)p.M);
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fused_gemv_kernel<T, kGated, kBf16>), smem, attr);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(fused_gemv_kernel<T, kGated, kBf16>, dim3((unsigned)grid), dim3(fgv::kWarps * 32), (size_t)smem, s, p);
}

cudaError_t launch_fused_gemv(const FusedGemvParams &p, bool gated, bool bf16, int grid, cudaStream_t s) {
  if (p.M <= 8)
    return gated ? (bf16 ? launch_fused_gemv_t<1, true, true>(p, grid, s) : launch_fused_gemv_t<1, true, false>(p, grid, s))
                 : (bf16 ? launch_fused_gemv_t<1, false, true>(p, grid, s) : launch_fused_gemv_t<1, false, false>(p, grid, s));
  return gated ? (bf16 ? launch_fused_gemv_t<2, true, true>(p, grid, s) : launch_fused_gemv_t<2, true, false>(p, grid, s))
               : (bf16 ? launch_fused_gemv_t<2, false, true>(p, grid, s) : launch_fused_gemv_t<2, false, false>(p, grid, s));
}

}  // namespace w4
