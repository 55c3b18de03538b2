// fused_simple.cu -- plain CUDA-core kernels of the fused operators: right for every
// size and type, 64 x 64 tiles in shared memory, fp32 throughout.
#include "act.cuh"
#include "common.cuh"

namespace w4 {

struct FusedParams {
  const void *X;  // activations (or dZ fp32 for the gradient)
  int x_dtype;
  int64_t M, N, K;  // N: rows of the packed matrix (2F for gated)
  int group;
  const uint8_t *packed;
  const uint16_t *scales, *zeros;
  const float *awq_s, *bias;
  int act;
  const void *residual;
  void *Z, *Y;
  int y_dtype;
};

__device__ __forceinline__ float weight_at(const FusedParams &p, int64_t n, int64_t k) {
  const uint8_t b = p.packed[n * (p.K / 2) + k / 2];
  const int64_t g = n * (p.K / p.group) + k / p.group;
  const float q = (float)((k & 1) ? b >> 4 : b & 15);
  const float w = (q - half_bits_to_float(p.zeros[g])) * half_bits_to_float(p.scales[g]);
  return p.awq_s ? w * p.awq_s[k] : w;
}

// Y tile of 64 tokens x 64 outputs; gated: the tile's up rows are F = N / 2 below its gate rows.
template <bool kGated>
__global__ void __launch_bounds__(256) fused_simple_fwd(FusedParams p) {
  __shared__ float sX[64][17], sW[kGated ? 2 : 1][64][17];
  const int64_t F = kGated ? p.N / 2 : p.N;
  const int64_t n0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, accu[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, c = i & 15;
      sX[r][c] = m0 + r < p.M ? load_as_float(p.X, p.x_dtype, (m0 + r) * p.K + k0 + c) : 0.0f;
      sW[0][r][c] = n0 + r < F ? weight_at(p, n0 + r, k0 + c) : 0.0f;
      if constexpr (kGated) sW[1][r][c] = n0 + r < F ? weight_at(p, F + n0 + r, k0 + c) : 0.0f;
    }
    __syncthreads();
    for (int c = 0; c < 16; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
          acc[i][j] += sX[ty * 4 + i][c] * sW[0][tx * 4 + j][c];
          if constexpr (kGated) accu[i][j] += sX[ty * 4 + i][c] * sW[1][tx * 4 + j][c];
        }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= F) continue;
      float z = acc[i][j] + (p.bias ? p.bias[n] : 0.0f), y;
      if constexpr (kGated) {
        const float u = accu[i][j] + (p.bias ? p.bias[F + n] : 0.0f);
        if (p.Z) {
          store_from_float(p.Z, p.x_dtype, m * p.N + n, z);
          store_from_float(p.Z, p.x_dtype, m * p.N + F + n, u);
        }
        y = act_fwd(z, p.act) * u;
      } else {
        if (p.Z) store_from_float(p.Z, p.x_dtype, m * p.N + n, z);
        y = act_fwd(z, p.act);
        if (p.residual) y += load_as_float(p.residual, p.y_dtype, m * p.N + n);
      }
      store_from_float(p.Y, p.y_dtype, m * F + n, y);
    }
}

// dZ [M][N] fp32 from dY (and the pre-activations).
__global__ void fused_simple_dz(const void *dY, int dtype, const void *Z, int act, bool gated, int64_t M, int64_t N,
                                float *dZ) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= M * N) return;
  const int64_t m = i / N, n = i % N;
  float y, d;
  if (gated) {
    const int64_t F = N / 2, f = n < F ? n : n - F;
    act_both(load_as_float(Z, dtype, m * N + f), act, y, d);
    const float dh = load_as_float(dY, dtype, m * F + f);
    dZ[i] = n < F ? dh * load_as_float(Z, dtype, m * N + F + f) * d : dh * y;
  } else {
    d = 1.0f;
    if (Z) act_both(load_as_float(Z, dtype, i), act, y, d);
    dZ[i] = load_as_float(dY, dtype, i) * d;
  }
}

// dX [M][K] = dZ . W^, 64 x 64 tiles over (tokens, channels), contraction over the N rows.
__global__ void __launch_bounds__(256) fused_simple_dx(FusedParams p) {
  __shared__ float sZ[64][17], sW[16][65];
  const int64_t k0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * 64;
  const float *dZ = static_cast<const float *>(p.X);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t n0 = 0; n0 < p.N; n0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, c = i & 15, wr = i >> 6, wc = i & 63;
      sZ[r][c] = m0 + r < p.M && n0 + c < p.N ? dZ[(m0 + r) * p.N + n0 + c] : 0.0f;
      sW[wr][wc] = n0 + wr < p.N && k0 + wc < p.K ? weight_at(p, n0 + wr, k0 + wc) : 0.0f;
    }
    __syncthreads();
    for (int c = 0; c < 16; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += sZ[ty * 4 + i][c] * sW[c][tx * 4 + j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (m < p.M && k < p.K) store_from_float(p.Y, p.y_dtype, m * p.K + k, acc[i][j]);
    }
}

__global__ void fused_simple_dbias(const float *dZ, int64_t M, int64_t N, float *dbias) {
  const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= N) return;
  float a = 0.0f;
  for (int64_t m = 0; m < M; ++m) a += dZ[m * N + n];
  dbias[n] = a;
}

cudaError_t launch_fused_simple(const FusedParams &p, bool gated, cudaStream_t s) {
  const dim3 grid((unsigned)(((gated ? p.N / 2 : p.N) + 63) / 64), (unsigned)((p.M + 63) / 64));
  if (gated) fused_simple_fwd<true><<<grid, 256, 0, s>>>(p);
  else fused_simple_fwd<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fused_grad_simple(const FusedParams &p, bool gated, const void *dY, const void *Z, float *dZ,
                                     float *dbias, cudaStream_t s) {
  fused_simple_dz<<<(unsigned)((p.M * p.N + 255) / 256), 256, 0, s>>>(dY, p.x_dtype, Z, p.act, gated, p.M, p.N, dZ);
  if (dbias) fused_simple_dbias<<<(unsigned)((p.N + 255) / 256), 256, 0, s>>>(dZ, p.M, p.N, dbias);
  FusedParams q = p;
  q.X = dZ;
  fused_simple_dx<<<dim3((unsigned)((p.K + 63) / 64), (unsigned)((p.M + 63) / 64)), 256, 0, s>>>(q);
  return cudaGetLastError();
}

}  // namespace w4
