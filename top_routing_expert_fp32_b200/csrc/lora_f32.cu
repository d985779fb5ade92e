// fp32 form of the shared projection with per-row adapters for more than 64 rows (see lora.cu),
// on the CUDA cores: S = scale (X A), then 64 x 64 tiles of X W whose epilogue adds S B and the
// addend. Sums are kept in runs of 64 terms that are added up afterwards, so the rounding error
// grows with the run length, not with K.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kShrinkThreads = 128;
constexpr int kTile = 64, kDepth = 16, kRun = 64, kThreads = 256;

// One block per row: 4 ranks per thread, the rest of the threads over k.
__global__ void __launch_bounds__(kShrinkThreads)
    shrink_f32_kernel(const float* __restrict__ X, const float* __restrict__ A,
                      const int32_t* __restrict__ adapter, const float* __restrict__ scale,
                      float* __restrict__ S, int K, int L, int rank, int* err) {
  __shared__ float red[kShrinkThreads * 4];
  const int64_t m = blockIdx.x;
  const int ad = adapter[m];
  if (ad < -1 || ad >= L) {
    if (threadIdx.x == 0) record_error(err, MOE_DEVERR_BAD_INDEX);
    return;
  }
  if (ad < 0) return;
  const int per_row = rank / 4, subs = kShrinkThreads / per_row;
  const int tid = static_cast<int>(threadIdx.x), v = tid % per_row, sub = tid / per_row;
  if (sub < subs) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = sub; k0 < K; k0 += subs * kRun) {
      float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
      const int k1 = min(K, k0 + subs * kRun);
#pragma unroll 4
      for (int k = k0; k < k1; k += subs) {
        const float x = X[m * K + k];
        const float4 w = __ldg(reinterpret_cast<const float4*>(
            A + (static_cast<int64_t>(ad) * K + k) * rank + v * 4));
        run.x = fmaf(x, w.x, run.x);
        run.y = fmaf(x, w.y, run.y);
        run.z = fmaf(x, w.z, run.z);
        run.w = fmaf(x, w.w, run.w);
      }
      acc.x += run.x;
      acc.y += run.y;
      acc.z += run.z;
      acc.w += run.w;
    }
    *reinterpret_cast<float4*>(&red[sub * rank + v * 4]) = acc;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < rank; r += kShrinkThreads) {
    float s = 0.f;
    for (int q = 0; q < subs; ++q) s += red[q * rank + r];
    S[m * rank + r] = scale != nullptr ? s * scale[ad] : s;
  }
}

__global__ void __launch_bounds__(kThreads)
    project_f32_kernel(const float* __restrict__ X, const float* __restrict__ W,
                       const float* __restrict__ B, const int32_t* __restrict__ adapter,
                       const float* __restrict__ S, const float* addend, float* Y, int64_t M,
                       int K, int N, int L, int rank) {
  __shared__ float xs[kDepth][kTile + 4];
  __shared__ float ws[kDepth][kTile];
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int n0 = static_cast<int>(blockIdx.x) * kTile;
  const int tr = static_cast<int>(threadIdx.x) / 16, tc = static_cast<int>(threadIdx.x) % 16;
  float acc[4][4] = {}, run[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kDepth) {
    {  // 64 rows x 16 k of X, 16 k x 64 columns of W: one float4 each
      const int r = static_cast<int>(threadIdx.x) / 4, k = (static_cast<int>(threadIdx.x) % 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m0 + r < M && k0 + k < K)
        x = *reinterpret_cast<const float4*>(X + (m0 + r) * K + k0 + k);
      xs[k][r] = x.x;
      xs[k + 1][r] = x.y;
      xs[k + 2][r] = x.z;
      xs[k + 3][r] = x.w;
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + tr < K && n0 + tc * 4 < N)
        w = __ldg(reinterpret_cast<const float4*>(W + static_cast<int64_t>(k0 + tr) * N + n0 +
                                                  tc * 4));
      *reinterpret_cast<float4*>(&ws[tr][tc * 4]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = xs[k][tr * 4 + i];
      const float4 w = *reinterpret_cast<const float4*>(&ws[k][tc * 4]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        run[i][0] = fmaf(x[i], w.x, run[i][0]);
        run[i][1] = fmaf(x[i], w.y, run[i][1]);
        run[i][2] = fmaf(x[i], w.z, run[i][2]);
        run[i][3] = fmaf(x[i], w.w, run[i][3]);
      }
    }
    __syncthreads();
    if ((k0 / kDepth) % (kRun / kDepth) == kRun / kDepth - 1 || k0 + kDepth >= K) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] += run[i][j];
          run[i][j] = 0.f;
        }
    }
  }
  const int n = n0 + tc * 4;
  if (n >= N) return;
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + tr * 4 + i;
    if (m >= M) break;
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
    const int ad = adapter[m];
    if (ad >= 0 && ad < L) {
      const float* s = S + m * rank;
      const float* b = B + static_cast<int64_t>(ad) * rank * N + n;
#pragma unroll 4
      for (int r = 0; r < rank; ++r) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(b + static_cast<int64_t>(r) * N));
        d.x = fmaf(s[r], w.x, d.x);
        d.y = fmaf(s[r], w.y, d.y);
        d.z = fmaf(s[r], w.z, d.z);
        d.w = fmaf(s[r], w.w, d.w);
      }
    }
    float4 y = make_float4(acc[i][0] + d.x, acc[i][1] + d.y, acc[i][2] + d.z, acc[i][3] + d.w);
    if (addend != nullptr) {
      const float4 q = *reinterpret_cast<const float4*>(addend + m * N + n);
      y.x += q.x;
      y.y += q.y;
      y.z += q.z;
      y.w += q.w;
    }
    *reinterpret_cast<float4*>(Y + m * N + n) = y;
  }
}

}  // namespace

size_t lora_f32_workspace_bytes(const moe_lora_problem& p) {
  return sizeof(float) * static_cast<size_t>(p.M) * p.rank;
}

cudaError_t launch_lora_f32(const moe_lora_problem& p, const LoraTensors& t, void* scratch,
                            int* err, cudaStream_t stream) {
  float* S = static_cast<float*>(scratch);
  shrink_f32_kernel<<<static_cast<unsigned>(p.M), kShrinkThreads, 0, stream>>>(
      static_cast<const float*>(t.X), static_cast<const float*>(t.A), t.adapter, t.scale, S,
      static_cast<int>(p.K), p.adapters, p.rank, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Rows in grid.y: at most 65535 tiles a launch.
  const int64_t rows_per_launch = int64_t(65535) * kTile;
  for (int64_t m = 0; m < p.M; m += rows_per_launch) {
    const int64_t rows = std::min(rows_per_launch, p.M - m);
    const dim3 grid(static_cast<unsigned>((p.N + kTile - 1) / kTile),
                    static_cast<unsigned>((rows + kTile - 1) / kTile));
    project_f32_kernel<<<grid, kThreads, 0, stream>>>(
        static_cast<const float*>(t.X) + m * p.K, static_cast<const float*>(t.W),
        static_cast<const float*>(t.B), t.adapter + m, S + m * p.rank,
        t.addend != nullptr ? static_cast<const float*>(t.addend) + m * p.N : nullptr,
        static_cast<float*>(t.Y) + m * p.N, rows, static_cast<int>(p.K), static_cast<int>(p.N),
        p.adapters, p.rank);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
