// fp32 form of the shared projection with per-row adapters for more than 64 rows (see lora.cu),
// on the CUDA cores: S = scale (X A), then 128 x 64 tiles of X W whose epilogue adds S B and the
// addend. Bound by the FMA and shared-memory pipes for many tiles; few tiles cut K over the blocks
// of a cluster, whose sums meet in distributed shared memory (128 rows, 4096 x 512: 52 us, without
// the cut and the prefetch 241). Sums are kept in runs of 64 terms that are added up afterwards:
// the rounding error of K terms grows like that of 64 + K / 64 of them in one chain. (A tile has
// 128 rows: just above 64 rows two calls of lora.cu's kernel take less, 65 rows of 4096 x 14336
// 358 us as 64 and 1 against 485 here; 128 rows 594 as two against 497.)
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kShrinkThreads = 512;
constexpr int kRows = 128, kTile = 64, kDepth = 16, kRun = 64, kThreads = 256;
constexpr int kMaxSplits = 8;

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
      constexpr int kAtOnce = 8;  // k whose loads are on their way at once
      for (int kk = k0; kk < k1; kk += kAtOnce * subs) {
        float x[kAtOnce];
        float4 w[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int k = kk + u * subs;
          const bool in = k < k1;
          x[u] = in ? X[m * K + k] : 0.f;
          w[u] = in ? __ldg(reinterpret_cast<const float4*>(
                          A + (static_cast<int64_t>(ad) * K + k) * rank + v * 4))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          run.x = fmaf(x[u], w[u].x, run.x);
          run.y = fmaf(x[u], w[u].y, run.y);
          run.z = fmaf(x[u], w[u].z, run.z);
          run.w = fmaf(x[u], w[u].w, run.w);
        }
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

// Two fp32 values in one register pair, for the two-wide fused multiply-add.
__device__ __forceinline__ uint64_t both(float v) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// Tile (blockIdx.y, blockIdx.x), share blockIdx.z of K; the shares of a tile are one cluster.
__global__ void __launch_bounds__(kThreads)
    project_f32_kernel(const float* __restrict__ X, const float* __restrict__ W,
                       const float* __restrict__ B, const int32_t* __restrict__ adapter,
                       const float* __restrict__ S, const float* addend, float* Y, int64_t M,
                       int K, int N, int L, int rank) {
  struct Stage {
    float x[kDepth][kRows + 4];
    float w[kDepth][kTile];
  };
  __shared__ __align__(16) union {
    Stage stages[2];
    float sums[kRows * kTile];
  } sh;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kRows;
  const int n0 = static_cast<int>(blockIdx.x) * kTile;
  const int tid = static_cast<int>(threadIdx.x), tr = tid / 16, tc = tid % 16;
  const int splits = static_cast<int>(gridDim.z), split = static_cast<int>(blockIdx.z);
  const int chunk = (K + splits * kRun - 1) / (splits * kRun) * kRun;
  const int k_begin = min(K, split * chunk), k_end = min(K, k_begin + chunk);

  // 128 rows x 16 k of X, 16 k x 64 columns of W: two float4 and one per thread.
  const int lr = tid / 4, lk = tid % 4 * 4;
  float4 x[2], w;
  auto load = [&](int k0) {
    x[0] = x[1] = w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (m0 + h * 64 + lr < M && k0 + lk < k_end)
        x[h] = *reinterpret_cast<const float4*>(X + (m0 + h * 64 + lr) * K + k0 + lk);
    if (k0 + tr < k_end && n0 + tc * 4 < N)
      w = __ldg(reinterpret_cast<const float4*>(W + static_cast<int64_t>(k0 + tr) * N + n0 +
                                                tc * 4));
  };
  auto put = [&](Stage& st) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      st.x[lk][h * 64 + lr] = x[h].x;
      st.x[lk + 1][h * 64 + lr] = x[h].y;
      st.x[lk + 2][h * 64 + lr] = x[h].z;
      st.x[lk + 3][h * 64 + lr] = x[h].w;
    }
    *reinterpret_cast<float4*>(&st.w[tr][tc * 4]) = w;
  };
  // Eight rows by four columns per thread, two columns per instruction.
  float acc[8][4] = {};
  uint64_t run[8][2] = {};
  load(k_begin);
  put(sh.stages[0]);
  __syncthreads();
  int cur = 0;
  for (int k0 = k_begin; k0 < k_end; k0 += kDepth, cur ^= 1) {
    const bool more = k0 + kDepth < k_end;
    if (more) load(k0 + kDepth);  // under way during this stage's products
    const Stage& st = sh.stages[cur];
#pragma unroll 4
    for (int k = 0; k < kDepth; ++k) {
      const float4 x0 = *reinterpret_cast<const float4*>(&st.x[k][tr * 8]);
      const float4 x1 = *reinterpret_cast<const float4*>(&st.x[k][tr * 8 + 4]);
      const ulonglong2 wv = *reinterpret_cast<const ulonglong2*>(&st.w[k][tc * 4]);
      const float xs[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t xx = both(xs[i]);
        fma_pair(run[i][0], xx, wv.x);
        fma_pair(run[i][1], xx, wv.y);
      }
    }
    if (((k0 - k_begin) / kDepth) % (kRun / kDepth) == kRun / kDepth - 1 || !more) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 v = halves(run[i][j]);
          acc[i][2 * j] += v.x;
          acc[i][2 * j + 1] += v.y;
          run[i][j] = 0u;
        }
    }
    if (more) put(sh.stages[cur ^ 1]);  // last read before the barrier of the step before
    __syncthreads();
  }

  // The block's sums in place of the stages; each block then finishes its share of the rows.
  float* sums = sh.sums;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(sums + (tr * 8 + i) * kTile + tc * 4) =
        make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  cluster_sync_all();
  const int rows = kRows / splits;
  for (int item = tid; item < rows * (kTile / 4); item += kThreads) {
    const int r0 = split * rows + item / (kTile / 4), c4 = item % (kTile / 4) * 4;
    const int64_t m = m0 + r0;
    const int n = n0 + c4;
    if (m >= M || n >= N) continue;
    const uint32_t here = smem_u32(sums + r0 * kTile + c4);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < splits; ++b) {
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(mapa_shared(here, static_cast<uint32_t>(b)))
                   : "memory");
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    const int ad = adapter[m];
    if (ad >= 0 && ad < L) {
      const float* s = S + m * rank;
      const float* b = B + static_cast<int64_t>(ad) * rank * N + n;
      for (int r0 = 0; r0 < rank; r0 += kRun) {
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
        const int r1 = min(rank, r0 + kRun);
#pragma unroll 4
        for (int r = r0; r < r1; ++r) {
          const float4 bv =
              __ldg(reinterpret_cast<const float4*>(b + static_cast<int64_t>(r) * N));
          d.x = fmaf(s[r], bv.x, d.x);
          d.y = fmaf(s[r], bv.y, d.y);
          d.z = fmaf(s[r], bv.z, d.z);
          d.w = fmaf(s[r], bv.w, d.w);
        }
        y.x += d.x;
        y.y += d.y;
        y.z += d.z;
        y.w += d.w;
      }
    }
    if (addend != nullptr) {
      const float4 q = *reinterpret_cast<const float4*>(addend + m * N + n);
      y.x += q.x;
      y.y += q.y;
      y.z += q.z;
      y.w += q.w;
    }
    *reinterpret_cast<float4*>(Y + m * N + n) = y;
  }
  cluster_sync_all();  // no block leaves while another reads its sums
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
  const int64_t rows_per_launch = int64_t(65535) * kRows;
  for (int64_t m = 0; m < p.M; m += rows_per_launch) {
    const int64_t rows = std::min(rows_per_launch, p.M - m);
    const int64_t tiles = (p.N + kTile - 1) / kTile * ((rows + kRows - 1) / kRows);
    // K over a cluster's blocks until the device has four blocks per SM, 128 k each at least.
    int splits = 1;
    while (splits < kMaxSplits && tiles * splits * 2 <= 4 * num_sms() && p.K >= 256 * splits)
      splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + kTile - 1) / kTile),
                       static_cast<unsigned>((rows + kRows - 1) / kRows),
                       static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = static_cast<unsigned>(splits);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float* addend =
        t.addend != nullptr ? static_cast<const float*>(t.addend) + m * p.N : nullptr;
    e = cudaLaunchKernelEx(&cfg, project_f32_kernel, static_cast<const float*>(t.X) + m * p.K,
                           static_cast<const float*>(t.W), static_cast<const float*>(t.B),
                           t.adapter + m, static_cast<const float*>(S) + m * p.rank, addend,
                           static_cast<float*>(t.Y) + m * p.N, rows, static_cast<int>(p.K),
                           static_cast<int>(p.N), static_cast<int>(p.adapters),
                           static_cast<int>(p.rank));
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
