// Weight streaming for products with few rows: a persistent block per SM reads its share of a
// matrix through a ring of shared-memory stages filled by TMA, and multiplies it by the few
// activation rows. What bounds such a product is
// the one pass over the weights, so
//   - the work is cut into equal runs of stages, one per block, whatever the tile count
//     (SplitK): a tile whose reduction is shared by several blocks is summed by the last of
//     them to finish, in block order, so the result does not depend on timing;
//   - a stage's rows are 256 contiguous bytes (two 128-byte boxes side by side): with 128 bytes
//     the same loop without arithmetic read 5.5 TB/s, with 256 bytes 6.4 TB/s (2.6 GB of weights);
//   - the loads run ahead of the arithmetic by the whole ring, also across grid barriers
//     (weights do not depend on what the barrier waits for), but at most kInFlight stages are
//     under way at once: 96 KB per SM cover the latency, and more only queue in the memory
//     system, where the activation rows then queue behind them (Mixtral-shaped layer, 8 tokens,
//     with rows loaded by the consumers: 192 KB in flight 506 us, 128 KB 455, 96 KB 423, 64 KB
//     463);
//   - the activation rows of a stage come through the same ring, fetched once per block by a
//     second producer warp, so that the consumers never wait for an L2 access. It copies them
//     16 bytes per lane (cp.async): one bulk copy per row took about 110 cycles of the warp,
//     more than a stage's 1424 cycles of HBM time from 13 rows on.
// 16-bit weights [k][n] (n contiguous) become the row operand of mma.m16n8k16 through transposed
// ldmatrix (16 output columns x 16 k per instruction), the activation rows its 8 columns: one
// instruction per 512 bytes of weights and 8 rows, far from the tensor cores' limit: the stream
// bounds the 16-bit layer, so that tcgen05, with the weights' columns as its 128 rows, has nothing
// to win there (not tried for 33 to 64 rows of adapters, which the stream does not bound). The rows
// come through plain ldmatrix, 32 k of 8 rows per instruction, their pitch 16 bytes modulo the 128
// of all banks.
#pragma once

#include "common.cuh"

namespace moe {
namespace stream {

enum WeightKind { kBF16 = 0, kF32 = 1, kW8 = 2 };

constexpr int kBoxRows = 64;               // one TMA box: 64 k-rows of 128 bytes, swizzled
constexpr int kBoxBytes = kBoxRows * 128;
constexpr int kStageBytes = 4 * kBoxBytes;
constexpr int kMaxStages = 6;
constexpr int kInFlight = 3;               // stages of weights under way at once
// Activation rows of a stage, per tile of 8 rows. One matrix pair: 64 k-values of the rows
// themselves, rows kRowPitch bytes apart (no bank conflicts). One matrix: 128 k-values, 16-bit
// ones in operand order (two planes of four 512-byte groups), fp32 plain.
constexpr int kTileBytes = 4096;
constexpr int kRowPitch = 144, kRowPitchF32 = 256;
constexpr int kMaxRows = 64;     // activation rows of one call
constexpr int kMaxGrid = 148;    // blocks (one per SM)
constexpr int kBarConsumers = 1, kBarAll = 2, kBarRows = 3, kBarSide = 4;  // named barriers

// A stage is four boxes: two side by side (kCols output columns) times either two matrices with
// the same 64 k-rows, or 128 k-rows of one matrix. Where the reduction is cut over the warps, a
// box's warps each take 32 of its k-rows and a segment of kSeg columns: two warps for 16- and 32-bit
// weights, four for 8-bit ones, whose conversion to bf16 is what their warps spend their time on
// (Mixtral-shaped layer, 8 tokens: 300 us with 8 warps, 245 with 16).
// kPieceRows: activation rows of one product (tiles of 8); an expert with more rows is streamed
// again for the next piece. It is what the registers hold, but for a few words: a spill costs an L2
// access here, since the ring leaves the L1 cache almost nothing (8-bit weights, 32 tokens: 1300 us
// with pieces of 32 rows, 359 us of 16, whose kernel still spills 40 bytes of a thread).
template <int WK>
struct Shape;
template <>
struct Shape<kBF16> {
  static constexpr int kCols = 128, kBoxCols = 64, kSeg = 64, kBoxWarps = 2, kPieceRows = 32;
};
template <>
struct Shape<kF32> {
  static constexpr int kCols = 64, kBoxCols = 32, kSeg = 32, kBoxWarps = 2, kPieceRows = 32;
};
template <>
struct Shape<kW8> {
  static constexpr int kCols = 256, kBoxCols = 128, kSeg = 64, kBoxWarps = 4, kPieceRows = 16;
};

// The block: consumer warps, then a warpgroup whose first two warps produce weights and rows. The
// register file is shared out again after the start: the producers' warpgroup hands some of its
// registers to the consumers (threads x registers at the start = the two parts' sum).
template <int WK>
struct Team {
  static constexpr int kWarps = 4 * Shape<WK>::kBoxWarps;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kWeightWarp = kWarps, kRowWarp = kWarps + 1;
  static constexpr int kThreads = kConsumers + 128;
  static constexpr int kStartRegs = kWarps == 8 ? 168 : 96;
  static constexpr int kConsumerRegs = kWarps == 8 ? 216 : 104;
  static constexpr int kProducerRegs = kWarps == 8 ? 72 : 64;
  static_assert(kConsumers * kConsumerRegs + 128 * kProducerRegs <= kStartRegs * kThreads &&
                kStartRegs * kThreads <= 65536, "registers");
};

// A consumer warp's box, its first k-row there (0 or 32) and its segment of the box's columns.
template <int WK>
__device__ __forceinline__ int box_of(int warp) {
  return warp / Shape<WK>::kBoxWarps;
}
template <int WK>
__device__ __forceinline__ int warp_row(int warp) {
  return (WK == kW8 ? (warp >> 1) & 1 : warp & 1) * 32;
}
template <int WK>
__device__ __forceinline__ int warp_seg(int warp) {
  return WK == kW8 ? warp & 1 : 0;
}

// The stages of a product, `tiles` of `steps` each, over at most `blocks` blocks: block c takes
// [start(c), start(c+1)). Equal runs of stages, or runs of whole tiles where those are hardly
// longer: sharing a tile costs a block about as much as kShareStages stages (its sums to L2 and
// back, and an arrival that everybody's writes wait for).
constexpr int kShareStages = 4;
struct SplitK {
  long long units;  // stages or whole tiles
  int unit;         // stages of a unit
  int grid;
  __device__ SplitK(long long tiles, int steps, int blocks) {
    const long long total = tiles * steps;
    const long long whole = (tiles + blocks - 1) / blocks * steps;
    const bool by_tile = whole <= (total + blocks - 1) / blocks + kShareStages;
    units = by_tile ? tiles : total;
    unit = by_tile ? steps : 1;
    grid = static_cast<int>(units < blocks ? units : blocks);
  }
  __device__ long long start(int c) const { return units * c / grid * unit; }
  // The block that takes stage s, by stages (the largest c with start(c) <= s).
  __device__ int owner(long long s) const {
    return static_cast<int>(((s + 1) * grid - 1) / units);
  }
};

// Barriers of whole warps of the block. The instruction is for warps whose lanes are together, and
// lanes leave a wait or a loop one by one: the warp barrier before it brings them back.
__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t count) {
  __syncwarp();
  named_bar_sync(id, count);
}
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t count) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct Ring {
  uint8_t* weights;  // stage 0 (1024-byte aligned), kStageBytes each
  uint8_t* rows;     // stage 0, row_bytes each
  uint64_t* full;    // weights have landed
  uint64_t* rows_full;
  uint64_t* empty;
  int stages, row_bytes;
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

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (v & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_difference(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
// Four int8 values -> bf16, exactly: bytes 0 and 2 to `even`, bytes 1 and 3 to `odd`. For a byte
// b, bf16 0x4300 | (b & 127) is 128 + (b & 127) and 0x4300 | (b & 128) is 128 or, for negative b,
// 256; their difference is b.
__device__ __forceinline__ void i8x4_to_bf16(uint32_t v, uint32_t& even, uint32_t& odd) {
  const uint32_t u = v >> 8;
  even = bf16x2_difference(and_or(v, 0x007F007Fu, 0x43004300u),
                           and_or(v, 0x00800080u, 0x43004300u));
  odd = bf16x2_difference(and_or(u, 0x007F007Fu, 0x43004300u),
                          and_or(u, 0x00800080u, 0x43004300u));
}

// fp32 sums of one warp: kSeg columns by 8*NT rows.
//   mma kinds: v[(m * NT + j) * 4 + c] for the 16-column group m and row tile j.
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

// One thread's activation values of 32 k: for each row tile its pairs k = 8 q + 2 t + {0, 1} of
// row g (lane = 4 g + t); with SPLIT each value is the sum of two bf16 terms (planes 0 and 1).
template <int NT, bool SPLIT>
struct Frag {
  uint32_t r[NT][SPLIT ? 2 : 1][4];

  // From operand order: `rows` of the stage, 32-value group 0..3.
  __device__ __forceinline__ void load_ordered(const uint8_t* rows, int group, int lane) {
    static_assert(SPLIT, "two planes");
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(rows + j * kTileBytes + group * 1024 +
                                                        q * 512 + lane * 16);
        r[j][q][0] = v.x;
        r[j][q][1] = v.y;
        r[j][q][2] = v.z;
        r[j][q][3] = v.w;
      }
  }

  // From plain rows: 32-value group `group`; k0: its first k within the reduction of K (past its
  // end nothing was copied: zeros; K is a multiple of 8).
  __device__ __forceinline__ void load_rows(const uint8_t* rows, int row_pitch, int group, int k0,
                                            int K, int lane) {
    static_assert(!SPLIT, "one plane");
    const uint32_t at = smem_u32(rows) + static_cast<uint32_t>((lane & 7) * row_pitch +
                                                               group * 64 + (lane >> 3) * 16);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      ldsm_x4(at + static_cast<uint32_t>(8 * j * row_pitch), r[j][0]);
    if (k0 + 32 > K) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (k0 + 8 * q >= K) {
#pragma unroll
          for (int j = 0; j < NT; ++j) r[j][0][q] = 0u;
        }
    }
  }
};

// A warp's weights of one stage, as the transposed loads deliver them: registers, so that the
// stage can be handed back before the arithmetic.
template <int WK>
struct Weights {
  uint32_t r[WK == kBF16 ? 8 : 4][4];
  // `box`: shared address of the warp's box.
  __device__ __forceinline__ void load(uint32_t box, int warp, int lane) {
    const int b = lane >> 3, i = lane & 7;
    const uint32_t rows = box + static_cast<uint32_t>(warp_row<WK>(warp)) * 128;
    if constexpr (WK == kBF16) {
      // Matrices of one load: (column halves lo, hi) x (blocks 2s, 2s + 1).
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t k = static_cast<uint32_t>(16 * s + (b >> 1) * 8 + i);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          ldsm_x4_trans(rows + k * 128 + ((static_cast<uint32_t>(m * 2 + (b & 1)) ^ (k & 7u)) << 4),
                        r[s * 4 + m]);
      }
    } else {
      // One load takes 16 columns (bytes) of all four blocks.
      const uint32_t k = static_cast<uint32_t>(lane);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        ldsm_x4_trans(rows + k * 128 +
                          ((static_cast<uint32_t>(warp_seg<WK>(warp) * 4 + m) ^ (k & 7u)) << 4),
                      r[m]);
    }
  }
};

// acc += weights^T x rows.
template <int WK, int NT, bool SPLIT>
__device__ __forceinline__ void multiply(Acc<WK, NT>& acc, const Weights<WK>& w,
                                         const Frag<NT, SPLIT>& f) {
  constexpr int kPlanes = SPLIT ? 2 : 1;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if constexpr (WK == kBF16) {
#pragma unroll
      for (int q = 0; q < kPlanes; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mma_bf16(&acc.v[(m * NT + j) * 4], w.r[s * 4 + m], f.r[j][q][2 * s],
                     f.r[j][q][2 * s + 1]);
    } else {
      // As 16-bit elements, a transposed 8x8 matrix gives each thread the bytes of columns 2g and
      // 2g+1 at its pair of k; the even columns take the instruction's rows 0-7 and the odd ones
      // rows 8-15.
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) i8x4_to_bf16(w.r[m][2 * s + h], a[2 * h], a[2 * h + 1]);
#pragma unroll
        for (int q = 0; q < kPlanes; ++q)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_bf16(&acc.v[(m * NT + j) * 4], a, f.r[j][q][2 * s], f.r[j][q][2 * s + 1]);
      }
    }
  }
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// fp32 weights on the CUDA cores: acc.v[r] += sum over the warp's 32 k-rows of W[k][lane] x_r[k].
// `rows`: shared address of the stage's rows at this warp's first k, pitch bytes apart; k0: that k
// within K.
template <int NT>
__device__ __forceinline__ void multiply_f32(Acc<kF32, NT>& acc, uint32_t box, int warp, int lane,
                                             uint32_t rows, int pitch, int n_rows, int k0,
                                             int K) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t r = static_cast<uint32_t>((warp & 1) * 32 + h * 16 + i);
      const uint32_t at = box + r * 128 + (((static_cast<uint32_t>(lane) >> 2) ^ (r & 7u)) << 4) +
                          (static_cast<uint32_t>(lane) & 3u) * 4;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[i]) : "r"(at) : "memory");
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j >= n_rows) continue;
      // Eight rows at a time, 16 terms on their own: independent chains, and short ones, which
      // keep the rounding error low. (Rows past the last are read from the ring and dropped.)
      float s[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) s[r] = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (k0 + h * 16 + 4 * q < K) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 v = ld_shared_f4(rows + (8 * j + r) * static_cast<uint32_t>(pitch) +
                                          h * 64 + q * 16);
            s[r] = fmaf(w[4 * q], v.x, s[r]);
            s[r] = fmaf(w[4 * q + 1], v.y, s[r]);
            s[r] = fmaf(w[4 * q + 2], v.z, s[r]);
            s[r] = fmaf(w[4 * q + 3], v.w, s[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) acc.v[8 * j + r] += s[r];
    }
  }
}

// The warps' sums of one row tile meet in shared memory: red[warp][8 rows][kRedPitch]. The
// pitch keeps both the fragment-shaped writes and the row-shaped reads free of bank conflicts.
// With eight warps two such buffers in turn: one barrier per row tile, since a thread that writes
// a buffer again has passed the barrier of the other one, and with it every read of this one.
// Sixteen warps have one buffer of the same bytes and a second barrier after the reads.
constexpr int kRedPitch = 68;
constexpr size_t kRedBytes = 16 * 8 * kRedPitch * sizeof(float);
template <int WK>
struct RedTurn {
  float* base;
  int turn = 0;
  __device__ float* next() {
    if (Team<WK>::kWarps == 8) turn ^= 1;
    return base + turn * (8 * 8 * kRedPitch);
  }
  __device__ void done() {
    if (Team<WK>::kWarps != 8) bar_sync(kBarConsumers, Team<WK>::kConsumers);
  }
};

template <int WK, int NT>
__device__ __forceinline__ void put_tile(float* red, const Acc<WK, NT>& acc, int j, int warp,
                                         int lane) {
  float* mine = red + warp * 8 * kRedPitch;
#pragma unroll
  for (int jj = 0; jj < NT; ++jj) {
    if (jj != j) continue;
    if constexpr (WK == kF32) {
#pragma unroll
      for (int r = 0; r < 8; ++r) mine[r * kRedPitch + lane] = acc.v[8 * jj + r];
    } else {
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
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

// A thread's places in an epilogue pass over 8 rows by kCols columns, two columns at a time:
// i = tid, tid + kConsumers, ... < Places<WK>::kCount.
template <int WK>
struct Places {
  static constexpr int kPairs = Shape<WK>::kCols / 2;
  static constexpr int kCount = 8 * kPairs;
  static constexpr int kMine = (kCount + Team<WK>::kConsumers - 1) / Team<WK>::kConsumers;
  __device__ static int row(int i) { return i / kPairs; }
  __device__ static int col(int i) { return 2 * (i % kPairs); }
};

// Sum, in warp order, of the warps that hold columns col and col + 1 of `row`: of the matrix
// `branch` (0, 1) of a two-matrix stage, or of all (branch < 0).
template <int WK>
__device__ __forceinline__ float2 take_pair(const float* red, int branch, int row, int col) {
  const int box = col / Shape<WK>::kBoxCols, seg = col % Shape<WK>::kBoxCols / Shape<WK>::kSeg;
  const int in = col % Shape<WK>::kSeg;
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (branch >= 0 && half != branch) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // the two halves of the box's k-rows
      const int w = (half * 2 + box) * Shape<WK>::kBoxWarps + (WK == kW8 ? q * 2 + seg : q);
      const float2 v = *reinterpret_cast<const float2*>(red + (w * 8 + row) * kRedPitch + in);
      s.x += v.x;
      s.y += v.y;
    }
  }
  return s;
}

// Arrivals at a counter in global memory. Release and acquire at gpu scope: what the thread, and
// through the block barrier before it the whole block, wrote is visible to whoever sees the
// arrival (a full fence on either side took a microsecond).
__device__ __forceinline__ void arrive_global(int* counter) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(counter) : "memory");
}
__device__ __forceinline__ int count_global(int* counter) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
               : "=r"(old)
               : "l"(counter)
               : "memory");
  return old;
}

// A warp's arrival at a counter that `parts` warps share; true in the one that arrives last, whose
// lanes then see what all lanes of the others wrote before they arrived. The warp barriers make
// lane 0's release and acquire the whole warp's: a shuffle orders no memory.
__device__ __forceinline__ bool last_warp_to_arrive(int* counter, int parts, int lane) {
  __syncwarp();
  int old = 0;
  if (lane == 0) old = count_global(counter);
  old = __shfl_sync(0xFFFFFFFFu, old, 0);
  __syncwarp();
  return old == parts - 1;
}

// One thread: wait until `target` blocks have arrived at *bar (bounded).
__device__ __forceinline__ bool spin_until(int* bar, int target, uint64_t timeout_ns, int* err) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if (v >= target) break;
    if (globaltimer_ns() - t0 > timeout_ns) {
      record_error(err, MOE_DEVERR_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

// All consumer threads of every block: arrive, wait until `target` arrivals (bounded). The
// block's earlier global writes are visible to the others afterwards. False: the wait ran out.
template <int kConsumers>
__device__ __forceinline__ bool grid_barrier(int* bar, int target, int tid, int* flag,
                                             uint64_t timeout_ns, int* err) {
  bar_sync(kBarConsumers, kConsumers);
  if (tid == 0) {
    arrive_global(bar);
    *flag = spin_until(bar, target, timeout_ns, err) ? 1 : 0;
  }
  __syncwarp();
  bar_sync(kBarConsumers, kConsumers);
  return *flag != 0;
}

// One arrival per block that shares a tile; true in the block that arrives last (its threads
// then see what the others wrote before arriving).
template <int kConsumers>
__device__ __forceinline__ bool last_to_finish(int* counter, int parts, int tid, int* flag) {
  bar_sync(kBarConsumers, kConsumers);
  if (tid == 0) *flag = count_global(counter) == parts - 1;
  __syncwarp();
  bar_sync(kBarConsumers, kConsumers);
  const bool last = *flag != 0;
  return last;
}

// v[c] += the shares that blocks first..last hold of place i0 + c * kConsumers (< limit), in block
// order. `part`: [grid][2][part_floats]; a tile's first block holds its share in the second
// half. Four blocks' loads are on their way at once: an L2 latency for four of them, not one each.
template <int kConsumers, int C>
__device__ __forceinline__ void add_shares(float2 (&v)[C], const float* part, int64_t part_floats,
                                           int first, int last, int i0, int limit) {
  constexpr int kAtOnce = 4;
  for (int b0 = first; b0 <= last; b0 += kAtOnce) {
    float2 w[kAtOnce][C];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int b = b0 + u;
      const float2* p = reinterpret_cast<const float2*>(
          part + (static_cast<int64_t>(b) * 2 + (b == first ? 1 : 0)) * part_floats);
#pragma unroll
      for (int c = 0; c < C; ++c)
        w[u][c] = b <= last && i0 + c * kConsumers < limit ? __ldcg(p + i0 + c * kConsumers)
                                                           : make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[c].x += w[u][c].x;
        v[c].y += w[u][c].y;
      }
    }
  }
}

// The sum of p[q * stride] for q = first, first + step, ... below n, in that order. kAtOnce loads
// are on their way at once, the last ones too: an unrolled loop would take its remainder one L2
// latency at a time, longer than everything else here.
template <int kAtOnce>
__device__ __forceinline__ float sum_partials(const float* p, int64_t stride, int first, int step,
                                              int n) {
  float s = 0.0f;
  for (int q0 = first; q0 < n; q0 += kAtOnce * step) {
    float v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      v[u] = q0 + u * step < n ? __ldcg(p + (q0 + u * step) * stride) : 0.0f;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) s += v[u];
  }
  return s;
}

// Weight producer, before it fills the stage at `c` (the issued-th overall): the stage is free
// and at most kInFlight - 1 earlier ones are still under way; then announce its bytes.
__device__ __forceinline__ bool acquire_weights(const Ring& ring, const Cursor& c,
                                                long long issued, uint64_t timeout_ns) {
  if (!mbar_wait(&ring.empty[c.stage], c.phase ^ 1u, timeout_ns)) return false;
  if (issued >= kInFlight && ring.stages >= kInFlight) {
    int s = c.stage - kInFlight;
    uint32_t phase = c.phase;
    if (s < 0) {
      s += ring.stages;
      phase ^= 1u;
    }
    if (!mbar_wait(&ring.full[s], phase, timeout_ns)) return false;
  }
  mbar_arrive_expect_tx(&ring.full[c.stage], kStageBytes);
  return true;
}

// Before the block ends: every copy counted on `full` has landed (bounded).
__device__ __forceinline__ void drain(uint64_t* full, int stages, const Cursor& end,
                                      long long issued, uint64_t timeout_ns) {
  Cursor c = end;
  const long long n = issued < stages ? issued : stages;
  for (long long i = 0; i < n; ++i) {
    if (c.stage == 0) {
      c.stage = stages - 1;
      c.phase ^= 1u;
    } else {
      --c.stage;
    }
    if (!mbar_wait(&full[c.stage], c.phase, timeout_ns)) return;
  }
}

// A lane's 16 bytes global -> shared, and its arrival on `bar` (initialised for 32 lanes) once its
// copies so far have landed.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Generic-proxy writes of global memory before bulk copies of it, and the other way round.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

}  // namespace stream

// 3-D map over stacked weights [count][rows][cols] (cols contiguous) of a stream::WeightKind in
// boxes of box_rows rows x 128 bytes, 128-byte swizzle; elements past the edges read as zero.
bool make_stream_map(CUtensorMap* m, const void* ptr, int kind, uint64_t cols, uint64_t rows,
                     uint64_t count, uint32_t box_rows = stream::kBoxRows);

}  // namespace moe
