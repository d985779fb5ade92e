// Weight streaming for products with few rows: a persistent block per SM reads its share of a
// matrix through a ring of shared-memory stages filled by TMA, and multiplies it by the few
// activation rows, which come from L2 straight into registers. What bounds such a product is
// the one pass over the weights, so
//   - the work is cut into equal runs of stages, one per block, whatever the tile count
//     (SplitK): a tile whose reduction is shared by several blocks is summed by the last of
//     them to finish, in block order, so the result does not depend on timing;
//   - the loads run ahead of the arithmetic by the whole ring (160 KB and more per SM, above the
//     44 KB per SM that 6.5 TB/s times a microsecond of latency needs), also across grid
//     barriers: weights do not depend on what the barrier waits for.
// 16-bit weights [k][n] (n contiguous) become the row operand of mma.m16n8k16 through transposed
// ldmatrix (16 output columns x 16 k per instruction), the activation rows its 8 columns: one
// instruction per 512 bytes of weights and 8 rows, far from the tensor cores' limit, where the
// tcgen05 tiles of 64 or 128 rows would mostly multiply padding.
#pragma once

#include "common.cuh"

namespace moe {
namespace stream {

enum WeightKind { kBF16 = 0, kF32 = 1, kW8 = 2 };

constexpr int kConsumerWarps = 8;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kThreads = kConsumers + 32;  // + the producer warp
constexpr int kBoxBytes = 8192;            // one TMA box
constexpr int kStageBytes = 2 * kBoxBytes;
constexpr int kMaxRows = 64;               // activation rows of one product
constexpr int kMaxGrid = 148;              // blocks (one per SM)
constexpr int kBarConsumers = 1, kBarAll = 2;  // named barriers

// A box is kBoxRows k-rows by kCols output columns (128-byte rows; 64-byte rows for 8-bit
// weights). Warp w of a stage takes box w/4 and the (w%4)-th quarter of its rows.
template <int WK>
struct Box;
template <>
struct Box<kBF16> {
  static constexpr int kCols = 64, kRows = 64, kK16 = 1;
};
template <>
struct Box<kF32> {
  static constexpr int kCols = 32, kRows = 64, kK16 = 1;
};
template <>
struct Box<kW8> {
  static constexpr int kCols = 64, kRows = 128, kK16 = 2;
};

// Equal runs of the `total` stages of a product over `grid` blocks: block c takes
// [start(c), start(c+1)).
struct SplitK {
  long long total;
  int grid;
  __device__ long long start(int c) const { return total * c / grid; }
  // The block that takes stage s (the largest c with start(c) <= s).
  __device__ int owner(long long s) const {
    return static_cast<int>(((s + 1) * grid - 1) / total);
  }
};

struct Ring {
  uint32_t base;  // shared address of stage 0 (1024-byte aligned)
  uint64_t* full;
  uint64_t* empty;
  int stages;
};

struct Cursor {
  int stage = 0;
  uint32_t phase = 0;
  __device__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two int8 values in the low bytes of the two halves -> two bf16, exactly. For a byte b,
// bf16 0x4300 | (b & 127) is 128 + (b & 127) and 0x4300 | (b & 128) is 128 or, for negative b,
// 256; their difference is b.
__device__ __forceinline__ uint32_t i8x2_to_bf16x2(uint32_t v) {
  const uint32_t lo = (v & 0x007F007Fu) | 0x43004300u;
  const uint32_t hi = (v & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo),
                                   *reinterpret_cast<const __nv_bfloat162*>(&hi));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// fp32 sums of this warp's k-quarter: kCols columns by 8*NT rows.
//   mma kinds: v[((m * NT) + j) * 4 + c] for the 16-column group m and row tile j.
//   fp32:      v[row], column = lane.
template <int WK, int NT>
struct Acc {
  static constexpr int kSize = WK == kF32 ? 8 * NT : 16 * NT;
  float v[kSize];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kSize; ++i) v[i] = 0.0f;
  }
};

// The activation operand of one stage: NT row tiles, kK16 k-steps of 16; with SPLIT each value
// is the sum of two bf16 terms (words 0-1 and 2-3).
template <int WK, int NT, bool SPLIT>
struct Frag {
  uint32_t r[Box<WK>::kK16][NT][SPLIT ? 4 : 2];
};

// acc += (this warp's quarter of the box)^T x rows. `box`: shared address of the box, `quarter`:
// 0..3.
template <int WK, int NT, bool SPLIT>
__device__ __forceinline__ void multiply(Acc<WK, NT>& acc, uint32_t box, int quarter, int lane,
                                         const Frag<WK, NT, SPLIT>& f) {
  const int b = lane >> 3, i = lane & 7;
  if constexpr (WK == kBF16) {
    // 8x8 blocks (columns lo/hi) x (k lo/hi) of a 16 x 16 piece, 128-byte swizzled rows.
    const uint32_t row = box + static_cast<uint32_t>(quarter * 16 + (b >> 1) * 8 + i) * 128;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t a[4];
      ldsm_x4_trans(row + static_cast<uint32_t>(((m * 2 + (b & 1)) ^ i) << 4), a);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16(&acc.v[(m * NT + j) * 4], a, f.r[0][j][0], f.r[0][j][1]);
        if constexpr (SPLIT) mma_bf16(&acc.v[(m * NT + j) * 4], a, f.r[0][j][2], f.r[0][j][3]);
      }
    }
  } else {
    // 16-byte blocks of 8 k-rows: as 16-bit elements, a transposed 8x8 block gives each thread
    // the bytes of columns 2g and 2g+1 at k = 2t and 2t+1; the even columns take the
    // instruction's rows 0-7 and the odd ones rows 8-15.
    const uint32_t row = static_cast<uint32_t>(quarter * 32 + b * 8 + i);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t q[4];
      ldsm_x4_trans(box + row * 64 + ((static_cast<uint32_t>(m) ^ ((row >> 1) & 3u)) << 4), q);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = q[2 * s + h];
          a[2 * h] = i8x2_to_bf16x2(v & 0x00FF00FFu);
          a[2 * h + 1] = i8x2_to_bf16x2((v >> 8) & 0x00FF00FFu);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_bf16(&acc.v[(m * NT + j) * 4], a, f.r[s][j][0], f.r[s][j][1]);
          if constexpr (SPLIT)
            mma_bf16(&acc.v[(m * NT + j) * 4], a, f.r[s][j][2], f.r[s][j][3]);
        }
      }
    }
  }
}

// fp32 weights on the CUDA cores: acc.v[r] += sum over the quarter's 16 k of W[k][lane] x_r[k].
// row(r): row r's values (global memory), k0: its first k here, K: the reduction length.
template <int NT, typename RowPtr>
__device__ __forceinline__ void multiply_f32(Acc<kF32, NT>& acc, uint32_t box, int quarter,
                                             int lane, int n_rows, int k0, int K, RowPtr row) {
  float w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t r = static_cast<uint32_t>(quarter * 16 + i);
    const uint32_t at = box + r * 128 + (((static_cast<uint32_t>(lane) >> 2) ^ (r & 7u)) << 4) +
                        (static_cast<uint32_t>(lane) & 3u) * 4;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[i]) : "r"(at) : "memory");
  }
#pragma unroll
  for (int r = 0; r < 8 * NT; ++r) {
    if (r < n_rows) {
      const float* x = row(r) + k0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (k0 + 4 * q < K) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(x + 4 * q));
          acc.v[r] = fmaf(w[4 * q], v.x, acc.v[r]);
          acc.v[r] = fmaf(w[4 * q + 1], v.y, acc.v[r]);
          acc.v[r] = fmaf(w[4 * q + 2], v.z, acc.v[r]);
          acc.v[r] = fmaf(w[4 * q + 3], v.w, acc.v[r]);
        }
      }
    }
  }
}

// The warps' sums of one row tile meet in shared memory: red[warp][8 rows][kRedPitch]. The
// pitch keeps both the fragment-shaped writes and the row-shaped reads free of bank conflicts.
constexpr int kRedPitch = 68;
constexpr int kRedFloats = kConsumerWarps * 8 * kRedPitch;

template <int WK, int NT>
__device__ __forceinline__ void put_tile(float* red, const Acc<WK, NT>& acc, int j, int warp,
                                         int lane) {
  float* mine = red + warp * 8 * kRedPitch;
  if constexpr (WK == kF32) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float v = 0.0f;
#pragma unroll
      for (int jj = 0; jj < NT; ++jj)
        if (jj == j) v = acc.v[8 * jj + r];
      mine[r * kRedPitch + lane] = v;
    }
  } else {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int jj = 0; jj < NT; ++jj) {
        if (jj == j) {
          const float* c = &acc.v[(m * NT + jj) * 4];
          const int lo = WK == kW8 ? 16 * m + 2 * g : 16 * m + g;
          const int hi = WK == kW8 ? lo + 1 : lo + 8;
          mine[(2 * t) * kRedPitch + lo] = c[0];
          mine[(2 * t + 1) * kRedPitch + lo] = c[1];
          mine[(2 * t) * kRedPitch + hi] = c[2];
          mine[(2 * t + 1) * kRedPitch + hi] = c[3];
        }
      }
    }
  }
}

// Sum of warps [w0, w1) at (row, columns 2 pair and 2 pair + 1), in warp order.
__device__ __forceinline__ float2 take_pair(const float* red, int w0, int w1, int row, int pair) {
  float2 s = make_float2(0.0f, 0.0f);
  for (int w = w0; w < w1; ++w) {
    const float2 v =
        *reinterpret_cast<const float2*>(red + (w * 8 + row) * kRedPitch + 2 * pair);
    s.x += v.x;
    s.y += v.y;
  }
  return s;
}

// A thread's place in an epilogue pass over 8 rows by kCols columns.
template <int WK>
struct Place {
  static constexpr int kPairs = Box<WK>::kCols / 2;
  int row, pair;
  bool active;
  __device__ explicit Place(int tid)
      : row(tid / kPairs), pair(tid % kPairs), active(tid < 8 * kPairs) {}
};

// All consumer threads of every block: arrive, wait until `target` arrivals (bounded). The
// block's earlier global writes are visible to the others afterwards. False: the wait ran out.
__device__ __forceinline__ bool grid_barrier(int* bar, int target, int tid, int* flag,
                                             uint64_t timeout_ns, int* err) {
  named_bar_sync(kBarConsumers, kConsumers);
  if (tid == 0) {
    __threadfence();
    atomicAdd(bar, 1);
    int ok = 1;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
      int v;
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
      if (v >= target) break;
      if (globaltimer_ns() - t0 > timeout_ns) {
        ok = 0;
        record_error(err, MOE_DEVERR_WAIT_TIMEOUT);
        break;
      }
    }
    __threadfence();
    *flag = ok;
  }
  named_bar_sync(kBarConsumers, kConsumers);
  const bool ok = *flag != 0;
  return ok;
}

// One arrival per block that shares a tile; true in the block that arrives last (its threads
// then see what the others wrote before arriving).
__device__ __forceinline__ bool last_to_finish(int* counter, int parts, int tid, int* flag) {
  __threadfence();
  named_bar_sync(kBarConsumers, kConsumers);
  if (tid == 0) {
    const int old = atomicAdd(counter, 1);
    __threadfence();
    *flag = old == parts - 1;
  }
  named_bar_sync(kBarConsumers, kConsumers);
  const bool last = *flag != 0;
  return last;
}

// Producer side of one stage: wait for it to be free, then announce its bytes.
__device__ __forceinline__ bool acquire_stage(const Ring& ring, const Cursor& c,
                                              uint64_t timeout_ns) {
  if (!mbar_wait(&ring.empty[c.stage], c.phase ^ 1u, timeout_ns)) return false;
  mbar_arrive_expect_tx(&ring.full[c.stage], kStageBytes);
  return true;
}

// Before the block ends: every copy issued into the ring has landed (bounded).
__device__ __forceinline__ void drain(const Ring& ring, const Cursor& end, long long issued,
                                      uint64_t timeout_ns) {
  Cursor c = end;
  const long long n = issued < ring.stages ? issued : ring.stages;
  for (long long i = 0; i < n; ++i) {
    if (c.stage == 0) {
      c.stage = ring.stages - 1;
      c.phase ^= 1u;
    } else {
      --c.stage;
    }
    if (!mbar_wait(&ring.full[c.stage], c.phase, timeout_ns)) return;
  }
}

// 3-D map over stacked weights [count][rows][cols] (cols contiguous) in boxes of Box<kind>;
// elements past the edges read as zero. Defined in few.cu.
}  // namespace stream

bool make_stream_map(CUtensorMap* m, const void* ptr, int kind, uint64_t cols, uint64_t rows,
                     uint64_t count);

}  // namespace moe
