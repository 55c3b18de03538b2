// fused_stage.cu -- operand preparation of the fused tensor-core products, and dbias.
//
// The products run on fp16 operands with powers of two taken out, so that neither side
// can leave fp16's range and no bits but the last rounding are lost:
//   rows    r[n] = 2^a with a such that the row's largest scale * r lies in [2^10, 2^11):
//           (q - z) * (scale r) is at most 15 * 2^11 < 65504, and full precision reaches
//           down to groups whose scale is 2^-24 of the row's largest.
//   tokens  e[m] = 2^b with the token's largest |value| * e in [2^13, 2^14).
// Both are undone in fp32 in the product's epilogue.  Activations convert exactly down to
// 2^-30 (bf16, 8 significant bits) or 2^-27 (fp16, 11) of their token's largest, below which
// fp16's subnormals cut bits off: an error of 2^-38 of the largest at most.  With AWQ, x * s
// is rounded to fp16 once.
//
// Bound: HBM and the latency of a token's largest value, which has to be known before its
// first store.  Measured: 66 us for 2644 tokens of 17792 and the factors of 12850 rows
// (216 MB read and written, 3.3 TB/s); 20 us for 2048 tokens of 8192 and the factors of 8192
// rows (3.4 TB/s of activations); 93 us alone and 104 us in front of the product for dZ of
// 2048 tokens of 2 x 14336 (294 MB, 2.8 to 3.2 TB/s), where the exchange between a cluster's
// CTAs (memory barrier and cluster barrier for every token) is what warps wait for most.
#include "act.cuh"
#include "common.cuh"

namespace w4 {

// 2^k as a float, k in [-149, 127]
__device__ __forceinline__ float pow2f(int k) {
  return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(1u << (k + 149));
}

// The factor 2^b that brings `amax` into [2^t, 2^(t+1)), and its inverse.  0, infinity
// and NaN get 1 (a token with a non-finite value has non-finite outputs anyway).
__device__ __forceinline__ float2 pow2_to(float amax, int t) {
  if (!(amax > 0.0f) || amax > 3.4028235e38f) return make_float2(1.0f, 1.0f);
  int b = t - ilogbf(amax);
  b = b > 126 ? 126 : b;  // subnormal amax: 2^126 is enough to keep its few bits
  return make_float2(pow2f(b), pow2f(-b));
}

__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (unsigned i = 1; i < blockDim.x / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

// Row factors and group constants of 32 packed rows (256 threads): rinv[n] = 1 / r and,
// transposed to [group][row], the fp16 pair (scale * r, 1024 + z).  Rows are the lanes of
// every kernel that dequantizes, so a warp then reads its constants as one 128-byte line;
// straight from scales [n][g] each lane touched a line of its own, and the lines of a
// tile did not fit L1.
constexpr int kPrepRows = 32;

__device__ __forceinline__ void prep_rows(const uint16_t *scales, const uint16_t *zeros, int64_t kg, int64_t N, int64_t n0,
                                          float *rinv, uint32_t *tab) {
  __shared__ uint32_t tile[kPrepRows][33];
  __shared__ float rr[kPrepRows];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + 4 * w + i;
    float mx = 0.0f;
    if (n < N)
      for (int64_t g = lane; g < kg; g += 32) mx = fmaxf(mx, fabsf(half_bits_to_float(scales[n * kg + g])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float2 f = pow2_to(mx, 10);
    if (lane == 0) rr[4 * w + i] = f.x;
    if (lane == 0 && n < N) rinv[n] = f.y;
  }
  __syncwarp();  // a warp converts the rows whose factors it found
  for (int64_t g0 = 0; g0 < kg; g0 += 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + 4 * w + i, g = g0 + lane;
      if (n < N && g < kg) {
        const __half2 h = __floats2half2_rn(half_bits_to_float(scales[n * kg + g]) * rr[4 * w + i],
                                            1024.0f + half_bits_to_float(zeros[n * kg + g]));
        tile[4 * w + i][lane] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    __syncthreads();
    for (int gi = w; gi < 32; gi += 8)
      if (g0 + gi < kg && n0 + lane < N) tab[(g0 + gi) * N + n0 + lane] = tile[lane][gi];
    __syncthreads();
  }
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Blocks 0..M-1: x' = fp16(x s e) of one token, in the order the dequantization yields
// (0, 4, 1, 5, 2, 6, 3, 7 of every 8 channels), and 1 / e.  The blocks behind them:
// row factors and group constants of 32 packed rows each.  A token is read once: each thread keeps up
// to 4 vectors (K <= 8192 at 256 threads) between the maximum and the conversion; deeper
// layers read the rest again, from L1 or L2.
constexpr int kStageThreads = 256;
constexpr int kStageKeep = 4;

template <bool kBf16>
__global__ void __launch_bounds__(kStageThreads)
    fused_stage_x(const uint16_t *X, const float *awq_s, int64_t M, int64_t K, const uint16_t *scales,
                  const uint16_t *zeros, int64_t kg, int64_t N, uint16_t *xp, float *tinv, float *rinv, uint32_t *tab) {
  grid_launch_dependents();
  if (blockIdx.x >= M) {
    prep_rows(scales, zeros, kg, N, ((int64_t)blockIdx.x - M) * kPrepRows, rinv, tab);
    return;
  }
  __shared__ float red[kStageThreads / 32];
  const int64_t m = blockIdx.x, nv = K / 8;
  const uint4 *row = reinterpret_cast<const uint4 *>(X + m * K);
  auto scaled = [&](const uint4 &w, int64_t v, float (&f)[8]) {
    unpack8<kBf16>(w, f);
    if (awq_s) {
      const float4 a = reinterpret_cast<const float4 *>(awq_s)[2 * v], b = reinterpret_cast<const float4 *>(awq_s)[2 * v + 1];
      f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
      f[4] *= b.x; f[5] *= b.y; f[6] *= b.z; f[7] *= b.w;
    }
  };
  uint4 keep[kStageKeep];
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < kStageKeep; ++i) {
    const int64_t v = threadIdx.x + (int64_t)i * kStageThreads;
    keep[i] = v < nv ? row[v] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kStageKeep; ++i) {
    const int64_t v = threadIdx.x + (int64_t)i * kStageThreads;
    if (v >= nv) break;
    float f[8];
    scaled(keep[i], v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(f[j]));
  }
  for (int64_t v = threadIdx.x + (int64_t)kStageKeep * kStageThreads; v < nv; v += kStageThreads) {
    float f[8];
    scaled(row[v], v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(f[j]));
  }
  const float2 e = pow2_to(block_max(mx, red), 13);
  if (threadIdx.x == 0) tinv[m] = e.y;
  uint4 *out = reinterpret_cast<uint4 *>(xp + m * K);
  auto put = [&](const uint4 &w, int64_t v) {
    float f[8];
    scaled(w, v, f);
    out[v] = make_uint4(half2_bits(f[0] * e.x, f[4] * e.x), half2_bits(f[1] * e.x, f[5] * e.x),
                        half2_bits(f[2] * e.x, f[6] * e.x), half2_bits(f[3] * e.x, f[7] * e.x));
  };
#pragma unroll
  for (int i = 0; i < kStageKeep; ++i) {
    const int64_t v = threadIdx.x + (int64_t)i * kStageThreads;
    if (v < nv) put(keep[i], v);
  }
  for (int64_t v = threadIdx.x + (int64_t)kStageKeep * kStageThreads; v < nv; v += kStageThreads) put(row[v], v);
}

__global__ void __launch_bounds__(kStageThreads)
    fused_prep(const uint16_t *scales, const uint16_t *zeros, int64_t kg, int64_t N, float *rinv, uint32_t *tab) {
  prep_rows(scales, zeros, kg, N, (int64_t)blockIdx.x * kPrepRows, rinv, tab);
  grid_launch_dependents();  // only here: clusters that start among these blocks do not pack, and one left over
                             // takes as long again (twice the time at M = 7355, N = 37373, in every second call)
}

// dZ of `kVec` consecutive rows n.. of token m (gated: n.. lies on one side of F).
template <bool kGated, int kVec>
__device__ __forceinline__ void dz_at(const void *dY, const void *Z, int dtype, int act, int64_t N, int64_t m, int64_t n,
                                      float (&d)[kVec]) {
  const int64_t F = kGated ? N / 2 : N, f = kGated && n >= F ? n - F : n;
  float g[kVec], a[kVec], u[kVec];
  auto get = [&](const void *p, int64_t i, float (&v)[kVec]) {
    if constexpr (kVec == 8) {
      const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
      if (dtype == 2) unpack8<true>(w, v);
      else unpack8<false>(w, v);
    } else {
      v[0] = load_as_float(p, dtype, i);
    }
  };
  get(dY, m * F + f, g);
  if (Z) get(Z, m * N + f, a);
  if (kGated && n < F) get(Z, m * N + F + f, u);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    float y = 0.0f, s = 1.0f;
    if (Z) act_both(a[j], act, y, s);
    d[j] = !kGated ? g[j] * s : n < F ? g[j] * u[j] * s : g[j] * y;
  }
}

// dz' = fp16(dZ / r[n] * e), natural order, and 1 / e.  A cluster of CTAs takes tokens in turn,
// each CTA the same vectors of 8 outputs f (V to a thread) (of a gated call: rows f and F + f, which
// share their inputs) of every token: dZ stays in registers while the CTAs exchange the
// token's largest value, the next token's inputs are on their way meanwhile, and dbias's
// sums over the cluster's tokens, to part [cluster][N], cost nothing but additions.
// V = 1 where a cluster of 8 reaches over F with it (more CTAs then hide each other's
// exchanges), else 2, with 512 threads where one row factor per column leaves the shared
// memory for it.  kVec: rows start on 16 bytes; else elements one at a time.
__host__ __device__ constexpr int dz_threads(bool gated, int v) { return v == 1 || gated ? 256 : 512; }
__host__ __device__ constexpr int dz_per_sm(bool gated, int v) { return v == 1 ? 3 : gated ? 2 : 1; }

template <bool kGated, bool kBias, bool kVec, int V>
__global__ void __launch_bounds__(dz_threads(kGated, V), dz_per_sm(kGated, V))
    fused_stage_dz(const uint16_t *dY, const uint16_t *Z, int bf16, int act, int64_t M, int64_t N, int64_t ld,
                   const float *rinv, uint16_t *dzp, float *tinv, float *part) {
  constexpr int R = kGated ? 2 : 1, kDzThreads = dz_threads(kGated, V), kSlice = kDzThreads * V * 8;
  __shared__ __align__(16) float srinv[R][kSlice];
  __shared__ float red[kDzThreads / 32];
  __shared__ float peers[2][8];
  const int slices = gridDim.x, slice = blockIdx.x;  // a cluster is a row of the grid
  const int64_t F = kGated ? N / 2 : N;
  grid_launch_dependents();
  grid_dependency_wait();  // the row factors
  // A thread's outputs: at(i, j) of the slice, its 8 V values V vectors where rows start on
  // 16 bytes; else a warp's 32 threads read 32 neighbours.
  auto at = [&](int i, int j) {
    return kVec ? (i * kDzThreads + (int)threadIdx.x) * 8 + j : (i * 8 + j) * kDzThreads + (int)threadIdx.x;
  };
  const int64_t first = (int64_t)slice * kSlice;
  int64_t f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = first + at(i, 0);
  for (int j = threadIdx.x; j < kSlice; j += kDzThreads) {
    const int64_t n = (int64_t)slice * kSlice + j;
#pragma unroll
    for (int h = 0; h < R; ++h) srinv[h][j] = n < F ? rinv[h * F + n] : 0.0f;
  }
  __syncthreads();
  if (slices > 1)  // every CTA of the cluster runs before one writes to another
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  // The thread's values i of a row.  Behind F: 0, or where elements are read one at a time the
  // last one again, whose row factor is 0 (reads under a condition are not moved up, and each
  // pair waits for the one before: 2,800 instead of 990 us at M = 7355, N = 37373).
  auto get = [&](const uint16_t *row, int i) -> uint4 {
    if constexpr (kVec) {
      return f[i] < F ? *reinterpret_cast<const uint4 *>(row + f[i]) : make_uint4(0, 0, 0, 0);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = row[min(first + at(i, j), F - 1)];
      return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
  };
  uint4 raw[V][1 + R];  // dY; Z (gated: G, U)
  auto fetch = [&](int64_t m) {
    m = min(m, M - 1);  // (the last fetch is not used)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      raw[i][0] = get(dY + m * F, i);
      raw[i][1] = get(Z ? Z + m * N : dY + m * F, i);  // (unused without Z)
      if constexpr (kGated) raw[i][2] = get(Z + m * N + F, i);
    }
  };
  auto widen = [&](const uint4 &w, float (&v)[8]) {
    if (bf16) unpack8<true>(w, v);
    else unpack8<false>(w, v);
  };
  float acc[kBias ? V : 1][R][8] = {};
  fetch(blockIdx.y);
  int par = 0;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y, par ^= 1) {
    float d[V][R][8];
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float g[8], a[8], y[8], s[8];
      widen(raw[i][0], g);
      widen(raw[i][1], a);
      act_both8(a, Z ? act : (int)kActNone, y, s);
      if constexpr (kGated) {
        float u[8];
        widen(raw[i][R], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[i][0][j] = g[j] * u[j] * s[j];
          d[i][R - 1][j] = g[j] * y[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][0][j] = g[j] * s[j];
      }
#pragma unroll
      for (int h = 0; h < R; ++h) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          float r4[4];
          if constexpr (kVec) {
            const float4 x = *reinterpret_cast<const float4 *>(srinv[h] + at(i, j));
            r4[0] = x.x, r4[1] = x.y, r4[2] = x.z, r4[3] = x.w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) r4[k] = srinv[h][at(i, j + k)];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kBias) acc[i][h][j + k] += d[i][h][j + k];
            d[i][h][j + k] *= r4[k];
            mx = fmaxf(mx, fabsf(d[i][h][j + k]));
          }
        }
      }
    }
    fetch(m + gridDim.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = red[0];
#pragma unroll
    for (int i = 1; i < kDzThreads / 32; ++i) mx = fmaxf(mx, red[i]);
    if (slices > 1) {
      if (threadIdx.x < slices) {  // this CTA's largest value to every CTA of the cluster
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&peers[par][slice])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(mx) : "memory");
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      for (int i = 0; i < slices; ++i) mx = fmaxf(mx, peers[par][i]);
    } else {
      __syncthreads();  // red is read until here
    }
    const float2 e = pow2_to(mx, 13);
    if (slice == 0 && threadIdx.x == 0) tinv[m] = e.y;
    if (!kVec && slice == 0 && threadIdx.x < ld - N) dzp[m * ld + N + threadIdx.x] = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (f[i] < F)
#pragma unroll
        for (int h = 0; h < R; ++h) {
          const float(&x)[8] = d[i][h];
          const uint4 w = make_uint4(half2_bits(x[0] * e.x, x[1] * e.x), half2_bits(x[2] * e.x, x[3] * e.x),
                                     half2_bits(x[4] * e.x, x[5] * e.x), half2_bits(x[6] * e.x, x[7] * e.x));
          uint16_t *to = dzp + m * ld + h * F + first;
          if constexpr (kVec) {
            *reinterpret_cast<uint4 *>(to + at(i, 0)) = w;
          } else {
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (first + at(i, j) < F) to[at(i, j)] = (uint16_t)(q[j >> 1] >> (16 * (j & 1)));
          }
        }
  }
  if constexpr (kBias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int h = 0; h < R; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (first + at(i, j) < F) part[(int64_t)blockIdx.y * N + h * F + first + at(i, j)] = acc[i][h][j];
  }
  if (slices > 1)  // no CTA leaves while another may write to it
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same for rows longer than a cluster's slices: one token per block, in two passes (the
// second finds its inputs in L2); columns N.. up to the row stride `ld` become 0.
template <bool kGated, int kVec>
__global__ void __launch_bounds__(512)
    fused_stage_dz_rows(const void *dY, const void *Z, int dtype, int act, int64_t N, int64_t ld, const float *rinv,
                        uint16_t *dzp, float *tinv) {
  grid_launch_dependents();
  grid_dependency_wait();  // the row factors
  __shared__ float red[16];
  const int64_t m = blockIdx.x;
  float mx = 0.0f;
  for (int64_t n = (int64_t)threadIdx.x * kVec; n < N; n += 512 * kVec) {
    float d[kVec];
    dz_at<kGated, kVec>(dY, Z, dtype, act, N, m, n, d);
#pragma unroll
    for (int j = 0; j < kVec; ++j) mx = fmaxf(mx, fabsf(d[j] * rinv[n + j]));
  }
  const float2 e = pow2_to(block_max(mx, red), 13);
  if (threadIdx.x == 0) tinv[m] = e.y;
  for (int64_t n = (int64_t)threadIdx.x * kVec; n < ld; n += 512 * kVec) {
    float d[kVec] = {};
    if (n < N) {
      dz_at<kGated, kVec>(dY, Z, dtype, act, N, m, n, d);
#pragma unroll
      for (int j = 0; j < kVec; ++j) d[j] = d[j] * rinv[n + j] * e.x;
    }
    if constexpr (kVec == 8)
      *reinterpret_cast<uint4 *>(dzp + m * ld + n) = make_uint4(half2_bits(d[0], d[1]), half2_bits(d[2], d[3]),
                                                                half2_bits(d[4], d[5]), half2_bits(d[6], d[7]));
    else
      dzp[m * ld + n] = __half_as_ushort(__float2half_rn(d[0]));
  }
}

// dbias: sums of dZ over the tokens.  A block takes 32 * kVec columns and a range of
// tokens, 8 tokens at a time (one per warp); the ranges' sums go to part [ranges][N] and
// a second kernel adds them in order, so the result does not depend on timing.
template <bool kGated, int kVec>
__global__ void __launch_bounds__(256)
    fused_dbias_part(const void *dY, const void *Z, int dtype, int act, int64_t M, int64_t N, int64_t per, float *part) {
  __shared__ float sum[8][32 * kVec];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = ((int64_t)blockIdx.x * 32 + lane) * kVec;
  const int64_t m1 = min(M, ((int64_t)blockIdx.y + 1) * per);
  float acc[kVec] = {};
  if (n < N)
    for (int64_t m = (int64_t)blockIdx.y * per + w; m < m1; m += 8) {
      float d[kVec];
      dz_at<kGated, kVec>(dY, Z, dtype, act, N, m, n, d);
#pragma unroll
      for (int j = 0; j < kVec; ++j) acc[j] += d[j];
    }
#pragma unroll
  for (int j = 0; j < kVec; ++j) sum[w][lane * kVec + j] = acc[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * kVec; c += 256) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sum[i][c];
    const int64_t col = (int64_t)blockIdx.x * 32 * kVec + c;
    if (col < N) part[blockIdx.y * N + col] = s;
  }
}

__global__ void __launch_bounds__(256) fused_dbias_sum(const float *part, int ranges, int64_t N, float *dbias) {
  __shared__ float sum[8][32];  // 32 columns, every eighth range to a warp
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (n < N)
#pragma unroll 8
    for (int i = w; i < ranges; i += 8) s += part[i * N + n];
  sum[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sum[i][lane];
    dbias[n] = s;
  }
}

// ------------------------------------------------------------------ launches
template <typename... Args>
cudaError_t launch_pdl(void (*kern)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       typename std::common_type<Args>::type... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_fused_stage_x(const void *X, bool bf16, const float *awq_s, int64_t M, int64_t K,
                                 const uint16_t *scales, const uint16_t *zeros, int64_t kg, int64_t N, uint16_t *xp,
                                 float *tinv, float *rinv, uint32_t *tab, cudaStream_t s) {
  const unsigned grid = (unsigned)(M + (N + kPrepRows - 1) / kPrepRows);
  const uint16_t *x = static_cast<const uint16_t *>(X);
  if (bf16) fused_stage_x<true><<<grid, kStageThreads, 0, s>>>(x, awq_s, M, K, scales, zeros, kg, N, xp, tinv, rinv, tab);
  else fused_stage_x<false><<<grid, kStageThreads, 0, s>>>(x, awq_s, M, K, scales, zeros, kg, N, xp, tinv, rinv, tab);
  return cudaGetLastError();
}

// Vectors per thread with which clusters of 8 reach over a token, 0 where they do not.
int fused_dz_vecs(int64_t N, bool gated) {
  const int64_t F = gated ? N / 2 : N;
  return F <= 8 * 8 * dz_threads(gated, 1) ? 1 : F <= 8 * 16 * dz_threads(gated, 2) ? 2 : 0;
}
// Clusters, at most: as many as the SMs hold, one per token.
int64_t fused_dz_grid(int64_t M, int64_t N, bool gated, int sm) {
  const int v = fused_dz_vecs(N, gated);
  const int64_t F = gated ? N / 2 : N, slice = dz_threads(gated, v) * 8 * v, slices = (F + slice - 1) / slice;
  const int64_t n = dz_per_sm(gated, v) * (int64_t)sm / slices;
  return M < n ? M : n < 1 ? 1 : n;
}
// Rows of dbias's partial sums: clusters, or ranges of tokens (about four blocks per SM, at
// least 8 tokens each).
int64_t fused_dbias_parts(int64_t M, int64_t N, bool gated, int sm) {
  if (fused_dz_vecs(N, gated)) return fused_dz_grid(M, N, gated, sm);
  const bool vec = (gated ? N / 2 : N) % 8 == 0;
  const int64_t cols = (N + (vec ? 256 : 32) - 1) / (vec ? 256 : 32);
  int64_t r = (600 + cols - 1) / cols;
  r = r > (M + 7) / 8 ? (M + 7) / 8 : r;
  return r < 1 ? 1 : r;
}

cudaError_t launch_fused_stage_dz(const void *dY, const void *Z, int dtype, int act, bool gated, int64_t M, int64_t N,
                                  int64_t ld, const uint16_t *scales, const uint16_t *zeros, int64_t kg, uint16_t *dzp,
                                  float *tinv, float *rinv, uint32_t *tab, float *part, float *dbias, int sm,
                                  int64_t *sums, cudaStream_t s) {
  const bool vec = (gated ? N / 2 : N) % 8 == 0;
  const int clusters = fused_dz_vecs(N, gated);
  *sums = 0;
  int64_t parts = dbias ? fused_dbias_parts(M, N, gated, sm) : 0;
  if (dbias && !clusters) {
    const int64_t per = (M + parts - 1) / parts;
    parts = (M + per - 1) / per;
    const dim3 grid((unsigned)((N + (vec ? 256 : 32) - 1) / (vec ? 256 : 32)), (unsigned)parts);
    auto k = gated ? (vec ? fused_dbias_part<true, 8> : fused_dbias_part<true, 1>)
                   : (vec ? fused_dbias_part<false, 8> : fused_dbias_part<false, 1>);
    k<<<grid, 256, 0, s>>>(dY, Z, dtype, act, M, N, per, part);
    fused_dbias_sum<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(part, (int)parts, N, dbias);
  }
  fused_prep<<<(unsigned)((N + kPrepRows - 1) / kPrepRows), kStageThreads, 0, s>>>(scales, zeros, kg, N, rinv, tab);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (!clusters) {
    auto k = gated ? (vec ? fused_stage_dz_rows<true, 8> : fused_stage_dz_rows<true, 1>)
                   : (vec ? fused_stage_dz_rows<false, 8> : fused_stage_dz_rows<false, 1>);
    return launch_pdl(k, dim3((unsigned)M), dim3(512), 0, s, dY, Z, dtype, act, N, ld, (const float *)rinv, dzp, tinv);
  }
  const int64_t F = gated ? N / 2 : N, slice = dz_threads(gated, clusters) * 8 * clusters;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((F + slice - 1) / slice), 1);
  cfg.blockDim = dim3(dz_threads(gated, clusters));
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cfg.gridDim.x;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cfg.gridDim.x > 1 ? 2 : 1;
  auto pick = [&](auto g, auto b, auto v) {
    constexpr bool G = decltype(g)::value, B = decltype(b)::value, C = decltype(v)::value;
    return clusters == 1 ? fused_stage_dz<G, B, C, 1> : fused_stage_dz<G, B, C, 2>;
  };
  using T = std::true_type;
  using U = std::false_type;
  const bool bias = dbias != nullptr;
  auto k = gated ? (bias ? (vec ? pick(T{}, T{}, T{}) : pick(T{}, T{}, U{})) : (vec ? pick(T{}, U{}, T{}) : pick(T{}, U{}, U{})))
                 : (bias ? (vec ? pick(U{}, T{}, T{}) : pick(U{}, T{}, U{})) : (vec ? pick(U{}, U{}, T{}) : pick(U{}, U{}, U{})));
  // No more clusters than run at a time (a few left over would take as long again): what the
  // device holds of this kernel and cluster size, asked once.
  static std::atomic<int> known[kAttrDevices][16][8];
  int dev = 0, most = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  std::atomic<int> *kn = dev >= 0 && dev < kAttrDevices
                             ? &known[dev][8 * gated + 4 * bias + 2 * vec + (clusters == 1)][cfg.gridDim.x - 1] : nullptr;
  if (kn) most = kn->load(std::memory_order_relaxed);
  if (most == 0) {
    cudaLaunchConfig_t q = cfg;
    q.gridDim.y = 1024;
    q.attrs = at + 1;
    q.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&most, k, &q) != cudaSuccess || most < 1) {
      cudaGetLastError();
      most = sm / (int)cfg.gridDim.x > 0 ? sm / (int)cfg.gridDim.x : 1;
    }
    if (kn) kn->store(most, std::memory_order_relaxed);
  }
  const int64_t want = fused_dz_grid(M, N, gated, sm);
  *sums = want < most ? want : most;
  cfg.gridDim.y = (unsigned)*sums;
  return cudaLaunchKernelEx(&cfg, k, static_cast<const uint16_t *>(dY), static_cast<const uint16_t *>(Z), dtype == 2 ? 1 : 0,
                            act, M, N, ld, (const float *)rinv, dzp, tinv, part);
}

// Behind the product (which does not wait for it): dbias from the clusters' sums.
cudaError_t launch_fused_dbias_sum(int64_t N, int64_t sums, const float *part, float *dbias, cudaStream_t s) {
  if (sums == 0) return cudaSuccess;  // summed already
  fused_dbias_sum<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(part, (int)sums, N, dbias);
  return cudaGetLastError();
}

}  // namespace w4
