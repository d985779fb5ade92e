// A projection shared by all rows beside the low-rank adapter of each row's own request:
//   Y[m] = addend[m] + X[m] W + scale[a] (X[m] A[a]) B[a],   a = adapter[m] (-1: none)
// for at most 64 rows, in one cooperative kernel (more rows: lora_sm100.cu, lora_f32.cu).
//
// What bounds it: one pass over W (and over the used adapters). W runs through the ring of
// stream.cuh in equal shares per block, as the few-token layer's down projection does; on top come
// the launch, the first stage's latency (4 us) and the last tiles' sums (3 us). The adapters' part
// hides behind the stream:
//   1. Shrink. Beside the stream, two warps compute S = X A: block (row, slice of K), a 16-byte
//      piece of an A row per thread, fp32 partial sums to L2. They arrive at the grid barrier,
//      wait for it, add everybody's partial sums up in shared memory and tell the consumers.
//   2. Expand. The different adapters of the batch (slots) follow W in the same ring: a stage
//      then holds 8 pieces of 16 ranks x the tile's columns of some B[a], and a tile's reduction
//      is its k-stages and then those. A warp multiplies a piece into fresh registers, for the
//      row tiles that have the adapter, and adds the sums of those rows only, so that a row
//      never meets another adapter's values, whatever they hold. S enters as two bf16 terms (16
//      bits of mantissa; fp32 weights: as it is). (The rows' expand products on the CUDA cores,
//      row by row out of L2, took longer than the stream: 48 rows of 48 adapters 71 us.)
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "stream.cuh"

namespace moe {

namespace {

using namespace stream;

// bf16 and fp32 weights: eight consumer warps; the two producers' neighbours compute S.
using LoraTeam = Team<kBF16>;
static_assert(Team<kF32>::kThreads == LoraTeam::kThreads, "one team");
constexpr int kConsumers = LoraTeam::kConsumers, kThreads = LoraTeam::kThreads;

constexpr int kMaxRank = 128;
// 128 values of a row: bf16 with 16 bytes against bank conflicts, fp32 (read as broadcasts) plain.
constexpr int kRowPitch128 = 272, kRowPitch128F32 = 512;

struct LoraArgs {
  const void* X;
  const void* A;
  const float* scale;
  const int32_t* adapter;
  const void* addend;
  void* Y;
  float* part_s;   // [slices][M][rank]
  float* part;     // [grid][2][part_floats]: sums of shared tiles
  int* counters;   // [kMaxGrid][kWarps]: the warps' arrivals at shared tiles
  int* bar;        // [3] workspace header ints, zero at rest: blocks that started, blocks that
                   // have their partial S out, blocks that finished
  int* err;
  int64_t part_floats;
  uint64_t timeout_ns;
  int M, K, N, L, rank, slices;
};

constexpr int kSideThreads = 64;  // the two warps that compute S

struct LoraTables {
  uint64_t full[kMaxStages];
  uint64_t rows_full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t s_ready;              // S is complete, the grid barrier passed
  float scratch[kSideThreads * 8];
  uint64_t slot_rows[kMaxRows];  // rows of each slot's adapter
  int slot[kMaxRows];            // the batch's different adapters
  int adapter[kMaxRows];         // of each row; -1: none
  float scale[kMaxRows];         // and its scale
  uint32_t firsts[2];
};

constexpr int kPieceRanks = 16;
constexpr int kStagePieces = 2 * kBoxRows / kPieceRanks;  // 8
__host__ __device__ constexpr int pieces_of(int rank) {
  return (rank + kPieceRanks - 1) / kPieceRanks;
}

constexpr size_t kMaxSmem = 232448;
static_assert(2 * LoraTeam::kWarps * 16 * 32 * sizeof(float) <= kRedBytes, "the parts' sums");
// S: whole row tiles of whole pieces, fp32 or two bf16 terms, zeros beyond M and the rank.
__host__ __device__ constexpr size_t s_bytes(int M, int rank) {
  return sizeof(float) * static_cast<size_t>((M + 7) / 8 * 8) * pieces_of(rank) * kPieceRanks;
}
// The consumers' sums: fp32 as in the few-token layer; bf16 per warp, or pair of warps, 16 columns
// of the rows at kStripPitch floats a row, or the sums that a pair exchanges.
constexpr int kStripPitch = 18;
__host__ __device__ constexpr int row_tiles_of(int M) {  // kernels are made for these
  const int n = (M + 7) / 8;
  return n <= 4 ? n : n <= 6 ? 6 : 8;
}
__host__ __device__ constexpr size_t sum_bytes(int M, bool f32) {
  return f32 ? kRedBytes
             : sizeof(float) * LoraTeam::kWarps * row_tiles_of(M) * 8 * kStripPitch;
}
__host__ __device__ constexpr size_t lora_ring_bytes(int M, int rank, bool f32) {
  return (kMaxSmem - 1024 - sum_bytes(M, f32) - s_bytes(M, rank) - sizeof(LoraTables)) &
         ~size_t(1023);
}
// A stage's rows, whole tiles of 8.
__host__ __device__ constexpr int lora_row_bytes(int M, bool f32) {
  return (M + 7) / 8 * 8 * (f32 ? kRowPitch128F32 : kRowPitch128);
}
__host__ __device__ constexpr int lora_stages(int M, int rank, bool f32) {
  const int s = static_cast<int>(lora_ring_bytes(M, rank, f32) /
                                 (kStageBytes + static_cast<size_t>(lora_row_bytes(M, f32))));
  return s < kMaxStages ? s : kMaxStages;
}
static_assert(lora_stages(kMaxRows, kMaxRank, false) >= kInFlight, "ring");
static_assert(lora_stages(kMaxRows, kMaxRank, true) >= 2, "ring");

// 16 bytes: four fp32 or eight bf16 values.
template <bool F32>
__device__ __forceinline__ void unpack16(const uint4& a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
      v[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
    }
  }
}

// The side warps' partial S of one row and slice of K (item: row + M * slice); kVec values of a row
// of A per thread (16 bytes).
template <bool F32>
__device__ void shrink(const LoraArgs& a, LoraTables& tb, int sid, int item) {
  constexpr int kVec = F32 ? 4 : 8;
  const int m = item % a.M, slice = item / a.M;
  const int ad = tb.adapter[m];
  if (ad < 0) return;  // nobody reads this row's sums
  const int per_row = a.rank / kVec, subs = kSideThreads / per_row;
  const int chunk = (a.K + a.slices - 1) / a.slices;
  const int k0 = min(a.K, slice * chunk), k1 = min(a.K, k0 + chunk);
  const int v = sid % per_row, sub = sid / per_row;
  if (sub < subs) {
    const int64_t x0 = static_cast<int64_t>(m) * a.K;
    const int64_t a0 = static_cast<int64_t>(ad) * a.K * a.rank + v * kVec;
    // Runs of 64 terms, added up in shared memory: the rounding error of one chain grows with its
    // length, 1024 terms for 64 rows of 4096 at rank 128.
    constexpr int kRun = 64;
    float* sums = tb.scratch + sub * a.rank + v * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) sums[i] = 0.0f;
    // Four k at a time, all their loads on their way before the first product of the four before:
    // beside the stream a load takes about 2 us (a row of 4096: the partial sums were out after 9.8
    // us one by one, 4.6 us by fours). Each row reads its own adapter, also where rows share one:
    // 64 rows of 4096 x 4096, 64 adapters of rank 128, take 136 us, most of it here.
    constexpr int kAtOnce = 4;
    static_assert(kRun % kAtOnce == 0, "whole runs");
    float x[kAtOnce];
    uint4 w[kAtOnce];
    auto load = [&](int k) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int at = k + u * subs;
        if (at < k1) {
          x[u] = F32 ? __ldg(static_cast<const float*>(a.X) + x0 + at)
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.X)[x0 + at]);
          w[u] = __ldg(reinterpret_cast<const uint4*>(
              static_cast<const uint8_t*>(a.A) +
              (a0 + static_cast<int64_t>(at) * a.rank) * (F32 ? 4 : 2)));
        }
      }
    };
    load(k0 + sub);
    for (int run = k0 + sub; run < k1; run += kRun * subs) {
      float acc[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
      const int end = min(k1, run + kRun * subs);
      for (int k = run; k < end; k += kAtOnce * subs) {
        float cx[kAtOnce];
        uint4 cw[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          cx[u] = x[u];
          cw[u] = w[u];
        }
        load(k + kAtOnce * subs);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          if (k + u * subs >= end) break;
          float v8[kVec];
          unpack16<F32>(cw[u], v8);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = fmaf(cx[u], v8[i], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) sums[i] += acc[i];
    }
  }
  bar_sync(kBarSide, kSideThreads);
  for (int r = sid; r < a.rank; r += kSideThreads) {
    float s = 0.0f;
#pragma unroll 4
    for (int q = 0; q < subs; ++q) s += tb.scratch[q * a.rank + r];
    a.part_s[(static_cast<int64_t>(slice) * a.M + m) * a.rank + r] = s;
  }
}

// S of one row and rank, scaled, as the expand reads it.
template <bool F32>
__device__ __forceinline__ void put_s(const LoraArgs& a, const LoraTables& tb, uint8_t* S, int i,
                                      float s) {
  const int m = i / a.rank, r = i - m * a.rank, ad = tb.adapter[m];
  const int at = m * pieces_of(a.rank) * kPieceRanks + r;
  if (ad < 0) return;
  s *= tb.scale[m];
  if constexpr (F32) {
    reinterpret_cast<float*>(S)[at] = s;
  } else {
    __nv_bfloat16* hi = reinterpret_cast<__nv_bfloat16*>(S) + at;
    const __nv_bfloat16 h = __float2bfloat16_rn(s);
    *hi = h;
    // A value that is infinite, or becomes so in bf16, has no remainder.
    const float rest = s - __bfloat162float(h);
    hi[(a.M + 7) / 8 * 8 * pieces_of(a.rank) * kPieceRanks] =
        __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.0f);
  }
}

// The side warps, after the grid barrier: all of S from everybody's partial sums.
template <bool F32>
__device__ void gather_s(const LoraArgs& a, LoraTables& tb, uint8_t* S, int sid) {
  const int n = a.M * a.rank;
  int per = 1;  // threads per value, over the slices
  while (per * 2 <= a.slices && per * 2 * n <= kSideThreads) per *= 2;
  if (per > 1) {
    const int i = sid % n, part = sid / n;
    if (part < per)
      tb.scratch[part * n + i] = sum_partials<8>(a.part_s + i, n, part, per, a.slices);
    bar_sync(kBarSide, kSideThreads);
    if (sid < n) {
      float s = 0.0f;
      for (int q = 0; q < per; ++q) s += tb.scratch[q * n + sid];
      put_s<F32>(a, tb, S, sid, s);
    }
    return;
  }
  // Four values by four slices on their way at once.
  constexpr int kAtOnce = 4, kSlices = 4;
  for (int i0 = sid; i0 < n; i0 += kAtOnce * kSideThreads) {
    float s[kAtOnce] = {};
    for (int q0 = 0; q0 < a.slices; q0 += kSlices) {
      float v[kSlices][kAtOnce];
#pragma unroll
      for (int q = 0; q < kSlices; ++q)
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int i = i0 + u * kSideThreads;
          v[q][u] = q0 + q < a.slices && i < n
                        ? __ldcg(a.part_s + static_cast<int64_t>(q0 + q) * n + i) : 0.0f;
        }
#pragma unroll
      for (int q = 0; q < kSlices; ++q)
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) s[u] += v[q][u];
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i0 + u * kSideThreads < n) put_s<F32>(a, tb, S, i0 + u * kSideThreads, s[u]);
  }
}

// ---- fp32 consumers, on the CUDA cores. A warp has eight rows, both 32-column boxes of the tile
// (a lane one column of each) and 1 / kParts of a stage's k; where there are fewer row tiles than
// warps, the parts' sums meet in shared memory. The loops are rolled: with the rows of all tiles
// unrolled in every warp a short call spent 11 us fetching instructions (64 rows, K = 64).
template <int NT>
struct RowsF32 {
  static constexpr int kParts = LoraTeam::kWarps / NT;
  static constexpr int kMine = 16 / kParts;  // of the (box, row) sums of a row tile, per warp
  float v[2][8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[0][r] = v[1][r] = 0.0f;
  }
};

__device__ __forceinline__ float ld_weight_f32(uint32_t box, int row, int lane) {
  const uint32_t r = static_cast<uint32_t>(row), l = static_cast<uint32_t>(lane);
  float w;
  asm volatile("ld.shared.f32 %0, [%1];"
               : "=f"(w)
               : "r"(box + r * 128 + (((l >> 2) ^ (r & 7u)) << 4) + (l & 3u) * 4)
               : "memory");
  return w;
}

// acc += the warp's k of a stage. `x`: shared address of its first row. 16 terms at a time on their
// own, which keeps the rounding error low.
template <int NT>
__device__ __forceinline__ void stage_f32(RowsF32<NT>& acc, uint32_t stage, uint32_t x, int part,
                                          int lane, int k0, int K) {
  constexpr int kDepth = 2 * kBoxRows / RowsF32<NT>::kParts;
#pragma unroll 1
  for (int k = part * kDepth; k < (part + 1) * kDepth && k0 + k < K; k += 16) {
    const uint32_t box = stage + static_cast<uint32_t>(k / kBoxRows) * 2 * kBoxBytes;
    float s[2][8];
#pragma unroll
    for (int r = 0; r < 8; ++r) s[0][r] = s[1][r] = 0.0f;
#pragma unroll 1
    for (int q = k; q < k + 16 && k0 + q < K; q += 4) {
      float w[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          w[c][i] = ld_weight_f32(box + c * kBoxBytes, q % kBoxRows + i, lane);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 v = ld_shared_f4(x + static_cast<uint32_t>(r * kRowPitch128F32 + q * 4));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s[c][r] = fmaf(w[c][0], v.x, s[c][r]);
          s[c][r] = fmaf(w[c][1], v.y, s[c][r]);
          s[c][r] = fmaf(w[c][2], v.z, s[c][r]);
          s[c][r] = fmaf(w[c][3], v.w, s[c][r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      acc.v[0][r] += s[0][r];
      acc.v[1][r] += s[1][r];
    }
  }
}

// acc += S x (every kParts-th of the pieces, from piece0 on, of an adapters' stage).
template <int NT>
__device__ __forceinline__ void expand_f32(RowsF32<NT>& acc, uint32_t stage, int tile, int part,
                                           int lane, const LoraTables& tb, const uint8_t* S,
                                           int piece0, int n_pieces, int per_slot) {
  const int ranks = per_slot * kPieceRanks;
#pragma unroll 1
  for (int h = part; h < kStagePieces; h += RowsF32<NT>::kParts) {
    const int piece = piece0 + h;
    if (piece >= n_pieces) return;
    const int slot = piece / per_slot, r0 = (piece - slot * per_slot) * kPieceRanks;
    const uint32_t mine = static_cast<uint32_t>(tb.slot_rows[slot] >> (8 * tile)) & 0xFFu;
    if (mine == 0) continue;
    const uint32_t box = stage + static_cast<uint32_t>(h >> 2) * 2 * kBoxBytes;
    float w[2][kPieceRanks];
#pragma unroll
    for (int i = 0; i < kPieceRanks; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        w[c][i] = ld_weight_f32(box + c * kBoxBytes, (h & 3) * kPieceRanks + i, lane);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if ((mine >> r) & 1u) {
        const float* s = reinterpret_cast<const float*>(S) + (8 * tile + r) * ranks + r0;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kPieceRanks; ++i) {
          s0 = fmaf(w[0][i], s[i], s0);
          s1 = fmaf(w[1][i], s[i], s1);
        }
        acc.v[0][r] += s0;
        acc.v[1][r] += s1;
      }
    }
  }
}

// Y of kMine sums of one lane: those from `first` on of its (box, row) pairs, box-major. An
// element's addend is read by the lane that writes it, before it does.
template <int NT>
__device__ __forceinline__ void store_f32(const LoraArgs& a, const float (&v)[RowsF32<NT>::kMine],
                                          int first, int tile, int n0, int lane) {
  const float* addend = static_cast<const float*>(a.addend);
  int64_t at[RowsF32<NT>::kMine];
  float e[RowsF32<NT>::kMine];
#pragma unroll
  for (int q = 0; q < RowsF32<NT>::kMine; ++q) {
    const int i = first + q, m = 8 * tile + (i & 7), n = n0 + (i >> 3) * 32 + lane;
    at[q] = m < a.M && n < a.N ? static_cast<int64_t>(m) * a.N + n : -1;
    e[q] = addend != nullptr && at[q] >= 0 ? addend[at[q]] : 0.0f;
  }
#pragma unroll
  for (int q = 0; q < RowsF32<NT>::kMine; ++q)
    if (at[q] >= 0) static_cast<float*>(a.Y)[at[q]] = v[q] + e[q];
}

// A tile's end: the parts' sums together, then Y, or the warp's share of a tile that blocks
// first..last share, whose last arrival adds the shares up in block order.
template <int NT>
__device__ __forceinline__ void finish_f32(const LoraArgs& a, const RowsF32<NT>& acc, float* red,
                                           int n0, int tid, bool whole, bool is_first, int first,
                                           int last) {
  using R = RowsF32<NT>;
  const int lane = tid & 31, warp = tid >> 5, tile = warp % NT, part = warp / NT;
  const int mine = part * R::kMine;  // the first of the warp's sums
  float v[R::kMine];
  if constexpr (R::kParts == 1) {
#pragma unroll
    for (int q = 0; q < R::kMine; ++q) v[q] = acc.v[q >> 3][q & 7];
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) red[(warp * 16 + q) * 32 + lane] = acc.v[q >> 3][q & 7];
    bar_sync(kBarConsumers, kConsumers);
#pragma unroll
    for (int q = 0; q < R::kMine; ++q) {
      v[q] = 0.0f;
#pragma unroll
      for (int p = 0; p < R::kParts; ++p)
        v[q] += red[((p * NT + tile) * 16 + mine + q) * 32 + lane];
    }
  }
  if (8 * tile >= a.M) return;
  if (!whole) {
    auto share = [&](int b, bool head) {
      return a.part + (static_cast<int64_t>(b) * 2 + (head ? 1 : 0)) * a.part_floats +
             warp * (R::kMine * 32) + lane;
    };
    float* out = share(static_cast<int>(blockIdx.x), is_first);
#pragma unroll
    for (int q = 0; q < R::kMine; ++q) out[q * 32] = v[q];
    if (!last_warp_to_arrive(a.counters + first * LoraTeam::kWarps + warp, last - first + 1, lane))
      return;
    // (The sums of four blocks are on their way at once.)
#pragma unroll
    for (int q = 0; q < R::kMine; ++q) v[q] = 0.0f;
    for (int b0 = first; b0 <= last; b0 += 4) {
      float w[4][R::kMine];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < R::kMine; ++q)
          w[u][q] = b0 + u <= last ? __ldcg(share(b0 + u, b0 + u == first) + q * 32) : 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < R::kMine; ++q) v[q] += w[u][q];
    }
  }
  store_f32<NT>(a, v, mine, tile, n0, lane);
}

// ---- bf16 consumers. A warp owns 16 columns of the tile and all of the reduction, so its sums are
// final in its registers: it needs neither the other warps nor a barrier to write them, or its
// share of them, and goes on with the next tile while others still multiply. It pays with
// shared-memory reads, since every warp reads all the activation rows: above 32 rows a pair of
// warps owns 32 columns, half of the reduction each, and the second hands its sums to the first.
// Against the few-token layer's way (the reduction over four warps, whose sums meet in shared
// memory eight rows at a time): 1 row of 4096 x 4096 13.2 us against 13.6, 32 rows of
// 4096 x 14336 with their adapters 33.8 against 35.2, 48 rows 42.7 against 43.2 (45.0 without
// the pairs).
constexpr int halves_of(int NT) { return NT > 4 ? 2 : 1; }

// Sums v[h][j][c]: row 8 j + 2 t + (c & 1), column 16 h + g + 8 (c >> 1) of the warp's, where
// lane = 4 g + t.
template <int NT>
struct Strip {
  static constexpr int kHalves = halves_of(NT);  // of the reduction; groups of 16 columns
  float v[kHalves][NT][4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[h][j][c] = 0.0f;
  }
};

// A warp's place: its columns' number among the tile's, its half of the reduction, the box of a
// side-by-side pair and the first 16-byte piece of the box's rows.
template <int NT>
struct Place {
  static constexpr int kHalves = halves_of(NT);
  static constexpr int kOwners = LoraTeam::kWarps / kHalves;  // warps that write sums
  int owner, half, side, piece;
  __device__ explicit Place(int warp)
      : owner(warp % kOwners), half(warp / kOwners), side(owner / (kOwners / 2)),
        piece(owner % (kOwners / 2) * 2 * kHalves) {}
  // Shared address of the 16 bytes that lane l of a transposed load addresses: 16 k-rows from row0
  // of the box on, column group h.
  __device__ __forceinline__ uint32_t weights(uint32_t box, int row0, int h, int lane) const {
    const uint32_t r = static_cast<uint32_t>(row0 + (lane >> 4) * 8 + (lane & 7));
    const uint32_t chunk = static_cast<uint32_t>(piece + h * 2 + ((lane >> 3) & 1));
    return box + r * 128 + ((chunk ^ (r & 7u)) << 4);
  }
};

// acc += a stage of 128 k. `release` hands the stage back once it is read.
template <int NT, class F>
__device__ __forceinline__ void strip_stage(Strip<NT>& acc, const Place<NT>& at, uint32_t stage,
                                            const uint8_t* rows, int lane, int k0, int K,
                                            F release) {
  constexpr int H = halves_of(NT), kGroups = 4 / H;  // of 32 k
  uint32_t w[kGroups][2][H][4];
#pragma unroll
  for (int q = 0; q < kGroups; ++q) {
    const int k32 = at.half * kGroups + q;
    const uint32_t box = stage + static_cast<uint32_t>((k32 >> 1) * 2 + at.side) * kBoxBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < H; ++h)
        ldsm_x4_trans(at.weights(box, (k32 & 1) * 32 + 16 * s, h, lane), w[q][s][h]);
  }
#pragma unroll
  for (int q = 0; q < kGroups; ++q) {
    const int k32 = at.half * kGroups + q;
    Frag<NT, false> f;
    f.load_rows(rows, kRowPitch128, k32, k0 + k32 * 32, K, lane);
    if (q == kGroups - 1) release();
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mma_bf16(acc.v[h][j], w[q][s][h], f.r[j][0][2 * s], f.r[j][0][2 * s + 1]);
  }
}

// acc += S x (the warp's pieces, of those from piece0 on, of an adapters' stage).
template <int NT>
__device__ __forceinline__ void strip_expand(Strip<NT>& acc, const Place<NT>& at, uint32_t stage,
                                             int lane, const LoraTables& tb, const uint8_t* S,
                                             int M, int piece0, int n_pieces, int per_slot) {
  constexpr int H = halves_of(NT), kPieces = kStagePieces / H;
  const int ranks = per_slot * kPieceRanks, g = lane >> 2, t = lane & 3;
  const uint32_t* hi = reinterpret_cast<const uint32_t*>(S);
  const uint32_t* lo = hi + (M + 7) / 8 * 8 * ranks / 2;
  piece0 += at.half * kPieces;
  int slot = piece0 / per_slot, part = piece0 - slot * per_slot;
#pragma unroll 2
  for (int i = 0; i < kPieces; ++i) {
    if (piece0 + i >= n_pieces) return;
    const uint64_t rows = tb.slot_rows[slot];
    const int in_stage = at.half * kPieces + i;
    const uint32_t box = stage + static_cast<uint32_t>((in_stage >> 2) * 2 + at.side) * kBoxBytes;
    uint32_t w[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
      ldsm_x4_trans(at.weights(box, (in_stage & 3) * kPieceRanks, h, lane), w[h]);
    const int r0 = part * kPieceRanks;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t mine = static_cast<uint32_t>(rows >> (8 * j)) & 0xFFu;
      if (mine == 0) continue;
      const int s = ((8 * j + g) * ranks + r0) / 2 + t;
      const uint32_t h0 = hi[s], h1 = hi[s + 4], l0 = lo[s], l1 = lo[s + 4];
      const bool even = (mine >> (2 * t)) & 1u, odd = (mine >> (2 * t + 1)) & 1u;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_bf16(c, w[h], h0, h1);
        mma_bf16(c, w[h], l0, l1);
        acc.v[h][j][0] += even ? c[0] : 0.0f;
        acc.v[h][j][1] += odd ? c[1] : 0.0f;
        acc.v[h][j][2] += even ? c[2] : 0.0f;
        acc.v[h][j][3] += odd ? c[3] : 0.0f;
      }
    }
    if (++part == per_slot) {
      part = 0;
      ++slot;
    }
  }
}

// The two warps of a pair, at a tile's end: the second's sums through shared memory (`strip`,
// owned by the pair) to the first, which goes on to write them. True in the first. Barriers
// kBarPair + owner: the sums are there; + kOwners: the strip is free again (also before its first
// use, so the first arrives there at the start and after each write).
constexpr int kBarPair = 5;
template <int NT>
__device__ __forceinline__ bool strip_meet(Strip<NT>& acc, const Place<NT>& at, float* strip,
                                           int lane) {
  constexpr int H = halves_of(NT);
  static_assert(H == 1 || sizeof(float4) * 32 * H * NT <=
                              sizeof(float) * 2 * NT * 8 * kStripPitch, "strip");
  if constexpr (H == 2) {
    float4* x = reinterpret_cast<float4*>(strip) + lane;
    if (at.half == 1) {
      bar_sync(kBarPair + Place<NT>::kOwners + at.owner, 64);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          x[(h * NT + j) * 32] = make_float4(acc.v[h][j][0], acc.v[h][j][1], acc.v[h][j][2],
                                             acc.v[h][j][3]);
      bar_arrive(kBarPair + at.owner, 64);
      return false;
    }
    bar_sync(kBarPair + at.owner, 64);
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float4 v = x[(h * NT + j) * 32];
        acc.v[h][j][0] += v.x;
        acc.v[h][j][1] += v.y;
        acc.v[h][j][2] += v.z;
        acc.v[h][j][3] += v.w;
      }
    __syncwarp();  // read before strip_store overwrites it
  }
  return true;
}
template <int NT>
__device__ __forceinline__ void strip_free(const Place<NT>& at) {
  if (halves_of(NT) == 2 && at.half == 0)
    bar_arrive(kBarPair + Place<NT>::kOwners + at.owner, 64);
}

// Y of the warp's columns (from n0 on): sums plus addend, through the warp's shared memory, so that
// a lane reads and writes 16 bytes of a row. An element's addend is read by the lane that writes
// it, before it does: the two may be the same array.
template <int NT>
__device__ __forceinline__ void strip_store(const LoraArgs& a, const Strip<NT>& acc, float* strip,
                                            int n0, int lane) {
  constexpr int kTimes = (NT * 16 + 31) / 32;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < halves_of(NT); ++h) {
    const int n = n0 + h * 16 + (lane & 1) * 8;
    uint4 extra[kTimes];
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int m = i * 16 + (lane >> 1);
      extra[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.addend != nullptr && m < a.M && n < a.N)
        extra[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.addend) +
                                                   static_cast<int64_t>(m) * a.N + n);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j < a.M) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          strip[(8 * j + 2 * t + (c & 1)) * kStripPitch + g + 8 * (c >> 1)] = acc.v[h][j][c];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int m = i * 16 + (lane >> 1);
      if (m < a.M && n < a.N) {
        const float2* v =
            reinterpret_cast<const float2*>(strip + m * kStripPitch + (lane & 1) * 8);
        const uint32_t e[4] = {extra[i].x, extra[i].y, extra[i].z, extra[i].w};
        uint32_t y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          y[q] = pack_bf16x2(v[q].x + bf16_bits_to_float(e[q] & 0xFFFFu),
                             v[q].y + bf16_bits_to_float(e[q] >> 16));
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) +
                                  static_cast<int64_t>(m) * a.N + n) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    __syncwarp();  // the strip is read before the next sums overwrite it
  }
}

// The warp's sums of a tile that blocks first..last share: its share to L2; the last of them to
// arrive adds all shares up in block order and writes Y.
template <int NT>
__device__ __forceinline__ void strip_share(const LoraArgs& a, Strip<NT>& acc,
                                            const Place<NT>& at, float* strip, int n0, int lane,
                                            bool is_first, int first, int last) {
  constexpr int H = halves_of(NT), kPerRow = 32 * Place<NT>::kOwners;
  auto share = [&](int b, bool head) {
    return reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(b) * 2 + (head ? 1 : 0)) *
                                                  a.part_floats) + at.owner * 32 + lane;
  };
  float4* mine = share(static_cast<int>(blockIdx.x), is_first);
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (8 * j < a.M)
        mine[(j * H + h) * kPerRow] = make_float4(acc.v[h][j][0], acc.v[h][j][1], acc.v[h][j][2],
                                                  acc.v[h][j][3]);
  if (!last_warp_to_arrive(a.counters + first * LoraTeam::kWarps + at.owner, last - first + 1,
                           lane))
    return;
  constexpr int kAtOnce = NT <= 2 ? 4 : 2;  // blocks whose shares are on their way at once
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc.v[h][j][c] = 0.0f;
    for (int b0 = first; b0 <= last; b0 += kAtOnce) {
      float4 w[kAtOnce][NT];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          w[u][j] = b0 + u <= last && 8 * j < a.M
                        ? __ldcg(share(b0 + u, b0 + u == first) + (j * H + h) * kPerRow)
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc.v[h][j][0] += w[u][j].x;
          acc.v[h][j][1] += w[u][j].y;
          acc.v[h][j][2] += w[u][j].z;
          acc.v[h][j][3] += w[u][j].w;
        }
    }
  }
  strip_store<NT>(a, acc, strip, n0, lane);
}

template <int WK, int NT>
__global__ void __launch_bounds__(kThreads, 1)
lora_few_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ LoraArgs a) {
  using S = Shape<WK>;
  constexpr bool kIsF32 = WK == kF32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + lora_ring_bytes(a.M, a.rank, kIsF32));
  uint8_t* S_mem = reinterpret_cast<uint8_t*>(red) + sum_bytes(a.M, kIsF32);  // S, scaled
  LoraTables& tb = *reinterpret_cast<LoraTables*>(S_mem + s_bytes(a.M, a.rank));
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int G = static_cast<int>(gridDim.x);
  const int me = static_cast<int>(blockIdx.x);

  Ring ring;
  ring.stages = lora_stages(a.M, a.rank, kIsF32);
  ring.row_bytes = lora_row_bytes(a.M, kIsF32);
  ring.weights = smem;
  ring.rows = smem + static_cast<size_t>(ring.stages) * kStageBytes;
  ring.full = tb.full;
  ring.rows_full = tb.rows_full;
  ring.empty = tb.empty;
  if (tid == kConsumers) {
    prefetch_tensormap(&mw);
    prefetch_tensormap(&mb);
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&tb.full[i], 1);
      mbar_init(&tb.rows_full[i], 32);  // the row producer's lanes
      mbar_init(&tb.empty[i], LoraTeam::kWarps);
    }
    mbar_init(&tb.s_ready, kSideThreads);
    fence_barrier_init();
    // This block's counter, and word that it is zero: blocks wait for that before they share a
    // tile, by which time all have long started.
    for (int i = 0; i < LoraTeam::kWarps; ++i) a.counters[me * LoraTeam::kWarps + i] = 0;
    arrive_global(&a.bar[0]);
  }
  {  // The rows' adapters, and the batch's different ones by first appearance.
    const int m = tid - kConsumers;
    int ad = -1;
    if (m >= 0 && m < a.M) {
      ad = a.adapter[m];
      if (ad < -1 || ad >= a.L) {
        record_error(a.err, MOE_DEVERR_BAD_INDEX);
        ad = -1;
      }
    }
    if (m >= 0 && m < kMaxRows) {
      tb.adapter[m] = ad;
      tb.scale[m] = ad >= 0 && a.scale != nullptr ? a.scale[ad] : 1.0f;
    }
    __syncthreads();
    uint64_t rows = 0;
    if (ad >= 0)
      for (int i = 0; i < a.M; ++i) rows |= static_cast<uint64_t>(tb.adapter[i] == ad) << i;
    const bool first = ad >= 0 && (rows & ((1ull << m) - 1ull)) == 0;
    const uint32_t f = __ballot_sync(0xFFFFFFFFu, first);
    if (m >= 0 && m < kMaxRows && lane == 0) tb.firsts[m >> 5] = f;
    __syncthreads();
    if (first) {
      const int at = __popc(f & ((1u << lane) - 1u)) + (m >= 32 ? __popc(tb.firsts[0]) : 0);
      tb.slot[at] = ad;
      tb.slot_rows[at] = rows;
    }
    // S is written where a row has an adapter; the rest of it stays zero.
    for (int i = tid; i < static_cast<int>(s_bytes(a.M, a.rank) / 4); i += kThreads)
      reinterpret_cast<uint32_t*>(S_mem)[i] = 0u;
  }
  __syncthreads();

  const int per_slot = pieces_of(a.rank);
  const int n_pieces = (__popc(tb.firsts[0]) + __popc(tb.firsts[1])) * per_slot;
  const int k_steps = (a.K + 2 * kBoxRows - 1) / (2 * kBoxRows);
  const int steps = k_steps + (n_pieces + kStagePieces - 1) / kStagePieces;
  const int tiles = (a.N + S::kCols - 1) / S::kCols;
  const SplitK sp(tiles, steps, G);
  const long long s0 = me < sp.grid ? sp.start(me) : 0, s1 = me < sp.grid ? sp.start(me + 1) : 0;

  // The block's segments (a tile and its stages [k0, k1)) in order, the first one last: it is a
  // tile's end, whose adapters' stages need S, and S takes a while. f returns false to stop.
  // (Divisions per segment only: a 64-bit one per stage cost more than the stage's HBM time.)
  auto segments = [&](auto f) {
    if (s0 >= s1) return;
    const long long head = min(s1, (s0 / steps + 1) * steps);  // end of the first segment
    long long s = head;
    while (true) {
      const bool last = s >= s1;
      const long long from = last ? s0 : s, tile = from / steps;
      const long long to = last ? head : min(s1, (tile + 1) * steps);
      if (!f(static_cast<int>(tile), static_cast<int>(from - tile * steps),
             static_cast<int>(to - tile * steps)) || last)
        return;
      s = to;
    }
  };
  auto walk = [&](auto f) {
    segments([&](int tile, int k0, int k1) {
      for (int k = k0; k < k1; ++k)
        if (!f(tile, k)) return false;
      return true;
    });
  };

  if (warp >= LoraTeam::kWarps) {
    give_registers<LoraTeam::kProducerRegs>();
    if (warp == LoraTeam::kWeightWarp) {
      if (lane == 0) {
        const uint64_t policy = l2_policy(-1);
        Cursor c;
        bool good = true;
        long long issued = 0;
        walk([&](int tile, int k) {
          if (!(good = acquire_weights(ring, c, issued, a.timeout_ns))) return false;
          const int col = tile * S::kCols, row = k * 2 * kBoxRows;
          uint8_t* dst = smem + static_cast<size_t>(c.stage) * kStageBytes;
          uint64_t* bar = &tb.full[c.stage];
          if (k >= k_steps) {
            // 16 rows of each box per piece; the last stage's unused ones repeat the last piece,
            // so that every stage has the same bytes.
            const int piece = (k - k_steps) * kStagePieces;
            int slot = piece / per_slot, part = piece - slot * per_slot;
            for (int j = 0; j < kStagePieces; ++j) {
              uint8_t* d = dst + (j >> 2) * 2 * kBoxBytes + (j & 3) * kPieceRanks * 128;
              const int r0 = part * kPieceRanks, ad = tb.slot[slot];
              tma_load_3d_hint(d, &mb, bar, col, r0, ad, policy);
              tma_load_3d_hint(d + kBoxBytes, &mb, bar, col + S::kBoxCols, r0, ad, policy);
              if (piece + j + 1 < n_pieces && ++part == per_slot) {
                part = 0;
                ++slot;
              }
            }
            c.next(ring.stages);
            ++issued;
            return true;
          }
          tma_load_3d_hint(dst, &mw, bar, col, row, 0, policy);
          tma_load_3d_hint(dst + kBoxBytes, &mw, bar, col + S::kBoxCols, row, 0, policy);
          tma_load_3d_hint(dst + 2 * kBoxBytes, &mw, bar, col, row + kBoxRows, 0, policy);
          tma_load_3d_hint(dst + 3 * kBoxBytes, &mw, bar, col + S::kBoxCols, row + kBoxRows, 0,
                           policy);
          c.next(ring.stages);
          ++issued;
          return true;
        });
        if (!good) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
        drain(tb.full, ring.stages, c, issued, a.timeout_ns);
      }
      __syncwarp();
    } else if (warp == LoraTeam::kRowWarp) {
      constexpr int kEl = kIsF32 ? 4 : 2;
      constexpr int kPieces = 2 * kBoxRows * kEl / 16;  // 16-byte pieces of a row
      constexpr int kPitch = kIsF32 ? kRowPitch128F32 : kRowPitch128;
      Cursor c;
      bool good = true;
      long long issued = 0;
      walk([&](int, int k_stage) {
        good = mbar_wait(&tb.empty[c.stage], c.phase ^ 1u, a.timeout_ns);
        good = __all_sync(0xFFFFFFFFu, good);
        if (!good) return false;
        const int k = k_stage * 2 * kBoxRows + lane % kPieces * (16 / kEl);
        if (k_stage < k_steps && k < a.K) {  // (an adapters' stage has no rows to copy)
          uint8_t* dst = ring.rows + c.stage * ring.row_bytes + lane % kPieces * 16;
          const uint8_t* src = static_cast<const uint8_t*>(a.X) + static_cast<int64_t>(k) * kEl;
#pragma unroll 4
          for (int m = lane / kPieces; m < a.M; m += 32 / kPieces)
            cp_async16(dst + m * kPitch, src + static_cast<int64_t>(m) * a.K * kEl);
        }
        cp_async_arrive(&tb.rows_full[c.stage]);
        c.next(ring.stages);
        ++issued;
        return true;
      });
      if (!good && lane == 0) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
      drain(tb.rows_full, ring.stages, c, issued, a.timeout_ns);
      __syncwarp();
    } else {
      // The side warps: S.
      const int sid = tid - (kConsumers + 64);
      for (int item = me; item < a.M * a.slices; item += G) {  // one, where there are SMs enough
        shrink<kIsF32>(a, tb, sid, item);
        bar_sync(kBarSide, kSideThreads);
      }
      if (sid == 0) {
        arrive_global(&a.bar[1]);
        (void)spin_until(&a.bar[1], G, a.timeout_ns, a.err);
      }
      __syncwarp();
      bar_sync(kBarSide, kSideThreads);
      gather_s<kIsF32>(a, tb, S_mem, sid);
      mbar_arrive(&tb.s_ready);
    }
  } else {
    take_registers<LoraTeam::kConsumerRegs>();
    bool ok = true, have_s = false, all_started = false;
    // Before the first adapters' stage: S.
    auto take_s = [&] {
      if (have_s) return;
      have_s = true;
      if (ok && !mbar_wait(&tb.s_ready, 0, a.timeout_ns)) {
        ok = false;
        record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
      }
      __syncwarp();
    };
    Cursor cur;
    auto wait_stage = [&] {
      if (ok && (!mbar_wait(&tb.full[cur.stage], cur.phase, a.timeout_ns) ||
                 !mbar_wait(&tb.rows_full[cur.stage], cur.phase, a.timeout_ns))) {
        ok = false;
        record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
      }
      __syncwarp();  // the lanes leave the wait one by one; what follows is for whole warps
    };
    auto release = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&tb.empty[cur.stage]);
    };
    // Before a thread counts its arrival at a shared tile: every block's counters are at zero.
    auto wait_started = [&](bool counts) {
      if (!all_started && counts) (void)spin_until(&a.bar[0], G, a.timeout_ns, a.err);
      __syncwarp();
      all_started = true;
    };
    if constexpr (!kIsF32) {
      const Place<NT> place(warp);
      // (A pair's strip is two warps' long.)
      float* strip = red + place.owner * (halves_of(NT) * NT * 8 * kStripPitch);
      strip_free<NT>(place);
      segments([&](int cb, int k0, int k1) {
        Strip<NT> acc;
        acc.zero();
        for (int k = k0; k < k1; ++k) {
          if (k >= k_steps) take_s();
          wait_stage();
          const uint32_t stage =
              smem_u32(ring.weights) + static_cast<uint32_t>(cur.stage) * kStageBytes;
          if (k < k_steps) {
            strip_stage<NT>(acc, place, stage, ring.rows + cur.stage * ring.row_bytes, lane,
                            k * 2 * kBoxRows, a.K, release);
          } else {
            strip_expand<NT>(acc, place, stage, lane, tb, S_mem, a.M,
                             (k - k_steps) * kStagePieces, n_pieces, per_slot);
            release();
          }
          cur.next(ring.stages);
        }
        if (!strip_meet<NT>(acc, place, strip, lane)) return true;
        const int n0 = cb * S::kCols + place.owner * 16 * halves_of(NT);
        if (k0 == 0 && k1 == steps) {
          strip_store<NT>(a, acc, strip, n0, lane);
        } else {
          const long long at = static_cast<long long>(cb) * steps;
          wait_started(lane == 0);
          strip_share<NT>(a, acc, place, strip, n0, lane, k0 == 0, sp.owner(at),
                          sp.owner(at + steps - 1));
        }
        strip_free<NT>(place);
        return true;
      });
      // (The last arrival there: no barrier is left half way.)
      if (halves_of(NT) == 2 && place.half == 1)
        bar_sync(kBarPair + Place<NT>::kOwners + place.owner, 64);
    } else {
      const int tile = warp % NT, part = warp / NT;
      int turn = 0;  // of two buffers: a write there is past the barrier after the last read
      segments([&](int cb, int k0, int k1) {
        RowsF32<NT> acc;
        acc.zero();
        for (int k = k0; k < k1; ++k) {
          if (k >= k_steps) take_s();
          wait_stage();
          const uint32_t stage =
              smem_u32(ring.weights) + static_cast<uint32_t>(cur.stage) * kStageBytes;
          if (8 * tile < a.M) {
            if (k >= k_steps)
              expand_f32<NT>(acc, stage, tile, part, lane, tb, S_mem,
                             (k - k_steps) * kStagePieces, n_pieces, per_slot);
            else
              stage_f32<NT>(acc, stage,
                            smem_u32(ring.rows) + static_cast<uint32_t>(
                                cur.stage * ring.row_bytes + 8 * tile * kRowPitch128F32),
                            part, lane, k * 2 * kBoxRows, a.K);
          }
          release();
          cur.next(ring.stages);
        }
        const bool whole = k0 == 0 && k1 == steps;
        const long long at = static_cast<long long>(cb) * steps;
        if (!whole) wait_started(lane == 0);
        turn ^= 1;
        finish_f32<NT>(a, acc, red + turn * (LoraTeam::kWarps * 16 * 32), cb * S::kCols, tid, whole,
                       k0 == 0, whole ? 0 : sp.owner(at), whole ? 0 : sp.owner(at + steps - 1));
        return true;
      });
    }
  }

  // The last block out returns the barrier counters to zero for the next launch.
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&a.bar[2], 1) == G - 1) {
      atomicExch(&a.bar[0], 0);
      atomicExch(&a.bar[1], 0);
      atomicExch(&a.bar[2], 0);
    }
  }
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t lora_part_floats(int64_t M) { return (M + 7) / 8 * 8 * Shape<kBF16>::kCols; }

// Slices of K per row: as many blocks as there are, at least 32 k each; at most 32, since every
// block adds them all up.
int lora_slices(int64_t M, int64_t K) {
  return static_cast<int>(
      std::max<int64_t>(1, std::min({kMaxGrid / M, (K + 31) / 32, static_cast<int64_t>(32)})));
}

template <int WK, int NT>
cudaError_t launch_few(const moe_lora_problem& p, const LoraArgs& a, const void* W, const void* B,
                       cudaStream_t stream) {
  CUtensorMap mw, mb;
  if (!make_stream_map(&mw, W, WK, p.N, p.K, 1) ||
      !make_stream_map(&mb, B, WK, p.N, p.rank, p.adapters, kPieceRanks))
    return cudaErrorInvalidValue;
  auto kernel = lora_few_kernel<WK, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(num_sms(), kMaxGrid)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, mw, mb, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_few_workspace_bytes(const moe_lora_problem& p) {
  const int64_t M = std::min<int64_t>(p.M, kMaxRows);
  return up256(sizeof(float) * kMaxGrid * p.rank) +  // slices x rows
         up256(sizeof(int) * kMaxGrid * LoraTeam::kWarps) +
         up256(sizeof(float) * 2 * kMaxGrid * lora_part_floats(M));
}

cudaError_t launch_lora_few(const moe_lora_problem& p, const LoraTensors& t, void* scratch,
                            int* err, int* bar, uint64_t timeout_ns, cudaStream_t stream) {
  LoraArgs a{};
  a.X = t.X;
  a.A = t.A;
  a.scale = t.scale;
  a.adapter = t.adapter;
  a.addend = t.addend;
  a.Y = t.Y;
  a.slices = lora_slices(p.M, p.K);
  uint8_t* w = static_cast<uint8_t*>(scratch);
  a.part_s = reinterpret_cast<float*>(w);
  w += up256(sizeof(float) * kMaxGrid * p.rank);
  a.counters = reinterpret_cast<int*>(w);
  w += up256(sizeof(int) * kMaxGrid * LoraTeam::kWarps);
  a.part = reinterpret_cast<float*>(w);
  a.part_floats = lora_part_floats(p.M);
  a.bar = bar;
  a.err = err;
  a.timeout_ns = timeout_ns;
  a.M = static_cast<int>(p.M);
  a.K = static_cast<int>(p.K);
  a.N = static_cast<int>(p.N);
  a.L = p.adapters;
  a.rank = p.rank;
  const int nt = (a.M + 7) / 8;
  if (p.dtype == MOE_DTYPE_F32) {
    if (nt == 1) return launch_few<kF32, 1>(p, a, t.W, t.B, stream);
    if (nt == 2) return launch_few<kF32, 2>(p, a, t.W, t.B, stream);
    if (nt <= 4) return launch_few<kF32, 4>(p, a, t.W, t.B, stream);
    return launch_few<kF32, 8>(p, a, t.W, t.B, stream);
  }
  if (nt == 1) return launch_few<kBF16, 1>(p, a, t.W, t.B, stream);
  if (nt == 2) return launch_few<kBF16, 2>(p, a, t.W, t.B, stream);
  if (nt == 3) return launch_few<kBF16, 3>(p, a, t.W, t.B, stream);
  if (nt == 4) return launch_few<kBF16, 4>(p, a, t.W, t.B, stream);
  if (nt <= 6) return launch_few<kBF16, 6>(p, a, t.W, t.B, stream);
  return launch_few<kBF16, 8>(p, a, t.W, t.B, stream);
}

}  // namespace moe
