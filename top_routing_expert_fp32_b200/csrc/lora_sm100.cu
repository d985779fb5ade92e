// The shared projection with per-row adapters (see lora.cu) for more than 64 rows, bf16:
//   Y = X W + addend + E,   E[m] = scale[a] (X[m] A[a]) B[a],  a = adapter[m]
// as one tcgen05 product over a longer reduction. For a tile of rows whose different adapters are
// a_0 .. a_{q-1} (its slots), after the k-steps of X W the accumulator takes S B[a_j] for every
// slot, S[m] = scale X[m] A[a], with the tensor-memory lanes (rows) of other adapters disabled in
// the instruction: a row meets only its own adapter's values, whatever the others hold. Rows of
// one adapter next to one another (prompts) make few slots, so the extra k-steps are a few per
// cent of K; a tile of all-different rows costs one step of 16 per rank-16 adapter.
//   1. shrink_kernel: S = X A. A group of 8 or 32 rows per cluster of blocks, K cut over the
//      blocks and their warps; each warp streams (adapter of the group, piece of K) steps
//      through its own TMA ring into mma.m16n8k16 (ranks x rows), the fp32 sums meet through
//      distributed shared memory. S, scaled, becomes two bf16 terms (16 bits of mantissa), both
//      operands of the product with B, as for few rows: a row's result has the same accuracy
//      whatever the batch. (In one term the error against 64 bits was 1.3 times the output
//      rounding's own where the adapter's part is as large as the rest.)
//   2. lora_gemm: the product, launched as a programmatic dependent of 1: it waits for S only when
//      its first tile comes to the extra k-steps, so the shrink hides behind the main loop.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "stream.cuh"

namespace moe {

namespace {

constexpr int kUnit = 16;          // k of one MMA
constexpr int kStageUnits = 4;     // MMAs per 64-wide k-block
// Pieces of B of an adapter, 16 ranks each, and how many a k-block takes. A k-block's A tile holds
// both terms of S for its pieces, so B is loaded once for the two: up to rank 32 all of a row's S
// (a k-block then takes the pieces of several adapters), above that 32 ranks (two pieces).
__host__ __device__ constexpr int pieces_of_rank(int rank) {
  const int u = (rank + kUnit - 1) / kUnit;
  return u <= 2 ? u : (u + 1) / 2 * 2;
}
__host__ __device__ constexpr int block_pieces(int rank) { return rank <= 32 ? kStageUnits : 2; }
// Ranks of a group: 64 columns of a row of S hold a group's first terms, then its second ones.
__host__ __device__ constexpr int group_ranks(int rank) {
  return rank <= 32 ? pieces_of_rank(rank) * kUnit : 32;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// ------------------------------------------------------------------ shrink

constexpr int kShrinkWarps = 4;
constexpr int kShrinkThreads = kShrinkWarps * 32;

struct ShrinkArgs {
  const int32_t* adapter;
  const float* scale;
  __nv_bfloat16* S;   // [M][ld]
  int32_t* n_slots;   // [tiles]
  int32_t* slots;     // [tiles][tile_rows] adapter of each slot
  uint32_t* masks;    // [tiles][tile_rows][tile_rows / 32] rows that do NOT have it
  int* err;
  int64_t M;
  int K, L, rank;
  int ld;             // columns of S, a multiple of 64
  int group;          // ranks of every 64 of them
  int tile_rows;      // 128 or 256
  int cluster;        // blocks per row group
  uint64_t timeout_ns;
};

// RT: 16-rank tiles (power of two), NT: tiles of 8 rows of a group. A step is 64 k: one or two
// boxes of A's ranks (up to 64 of them wide, swizzled over that width) and one of the rows.
template <int RT, int NT>
struct ShrinkShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRanks = 16 * RT;
  static constexpr int kCK = 64;
  static constexpr int kBoxRanks = kRanks < 64 ? kRanks : 64;
  static constexpr int kABoxBytes = kCK * kBoxRanks * 2;
  static constexpr int kABoxes = kRanks / kBoxRanks;
  static constexpr int kStageBytes = kABoxes * kABoxBytes + kRows * kCK * 2;
  static constexpr int kStages = RT >= 8 ? 2 : RT >= 4 ? 3 : 6;
  static constexpr size_t kSumBytes = sizeof(float) * kShrinkWarps * kRows * kRanks;
  static constexpr size_t kSmem =
      1024 + kSumBytes + static_cast<size_t>(kShrinkWarps) * kStages * kStageBytes;
  static_assert(kSmem <= 227 * 1024 - 4096, "shared memory of a block");
  static_assert(kStageBytes % 1024 == 0 && kSumBytes % 1024 == 0, "swizzle alignment");
  // Shared address of the 16 bytes of ranks [8 chunk, 8 chunk + 8) of a k-row of A (the box's
  // swizzle: 16-byte pieces exchanged by address bits 7 and up over 32, 64 or 128 bytes).
  __device__ static uint32_t a_piece(uint32_t stage, int row, int chunk) {
    constexpr int kPieces = kBoxRanks / 8;
    const int box = chunk / kPieces, c = chunk % kPieces;
    const int x = RT == 1 ? (row >> 2) & 1 : RT == 2 ? (row >> 1) & 3 : row & 7;
    return stage + box * kABoxBytes + row * (kBoxRanks * 2) + ((c ^ x) << 4);
  }
};

template <int RT, int NT>
__global__ void __launch_bounds__(kShrinkThreads)
shrink_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mx,
              const __grid_constant__ ShrinkArgs a) {
  using S = ShrinkShape<RT, NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t s_full[kShrinkWarps][S::kStages];
  __shared__ __align__(16) int s_tile[256];  // adapters of the tile's rows
  __shared__ int s_slot[256];   // the tile's slots
  __shared__ uint32_t s_first[8];
  __shared__ int s_item[S::kRows];
  __shared__ uint32_t s_mask[S::kRows];
  __shared__ int s_items;
  pdl_trigger();
  float* sums = reinterpret_cast<float*>(smem);  // [warp][row][rank]
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int rank_in_cluster = static_cast<int>(blockIdx.x) % a.cluster;
  const int64_t group = blockIdx.x / a.cluster;
  const int64_t row0 = group * S::kRows;
  const int64_t tile = row0 / a.tile_rows;
  const int64_t tile0 = tile * a.tile_rows;

  auto adapter_of = [&](int64_t m) {
    if (m >= a.M) return -1;
    const int ad = a.adapter[m];
    if (ad < -1 || ad >= a.L) {
      record_error(a.err, MOE_DEVERR_BAD_INDEX);
      return -1;
    }
    return ad;
  };
  for (int i = tid; i < a.tile_rows; i += kShrinkThreads) s_tile[i] = adapter_of(tile0 + i);
  for (int i = tid; i < static_cast<int>(S::kSumBytes / 4); i += kShrinkThreads) sums[i] = 0.0f;
  if (tid == 0) {
    for (int w = 0; w < kShrinkWarps; ++w)
      for (int i = 0; i < S::kStages; ++i) mbar_init(&s_full[w][i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  // The group's items: its different adapters and the rows that have them.
  if (warp == 0) {
    const int mine = lane < S::kRows ? s_tile[row0 - tile0 + lane] : -1;
    uint32_t left = __ballot_sync(0xFFFFFFFFu, mine >= 0);
    int n = 0;
    while (left != 0) {
      const int ad = __shfl_sync(0xFFFFFFFFu, mine, __ffs(left) - 1);
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine == ad);
      if (lane == 0) {
        s_item[n] = ad;
        s_mask[n] = m;
      }
      left &= ~m;
      ++n;
    }
    if (lane == 0) s_items = n;
  }
  __syncthreads();

  // Steps of this warp: for every item its pieces of K.
  const int pieces = (a.K + S::kCK - 1) / S::kCK;
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * rank_in_cluster / a.cluster);
  const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (rank_in_cluster + 1) / a.cluster);
  const int per_item = p1 - p0 > warp ? (p1 - p0 - warp + kShrinkWarps - 1) / kShrinkWarps : 0;
  const int total = per_item * s_items;
  uint8_t* ring = smem + S::kSumBytes + warp * S::kStages * S::kStageBytes;
  auto load = [&](int q) {
    if (q >= total || lane != 0) return;
    const int item = q / per_item;
    const int k0 = (p0 + warp + (q - item * per_item) * kShrinkWarps) * S::kCK;
    uint8_t* dst = ring + (q % S::kStages) * S::kStageBytes;
    uint64_t* bar = &s_full[warp][q % S::kStages];
    mbar_arrive_expect_tx(bar, S::kStageBytes);
#pragma unroll
    for (int i = 0; i < S::kABoxes; ++i)
      tma_load_3d(dst + i * S::kABoxBytes, &ma, bar, i * S::kBoxRanks, k0, s_item[item]);
    tma_load_2d(dst + S::kABoxes * S::kABoxBytes, &mx, bar, k0, static_cast<int>(row0));
  };
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][j][c] = 0.0f;
  for (int q = 0; q < S::kStages - 1; ++q) load(q);
  const int b = lane >> 3, i8 = lane & 7, t = lane & 3, g = lane >> 2;
  bool ok = true;
  for (int q = 0; q < total; ++q) {
    load(q + S::kStages - 1);
    if (ok && !mbar_wait(&s_full[warp][q % S::kStages], (q / S::kStages) & 1, a.timeout_ns)) {
      ok = false;
      record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
    }
    __syncwarp();  // the lanes leave the wait one by one; what follows is for whole warps
    const int item = q / per_item;
    const uint32_t mask = s_mask[item];
    const uint8_t* at = ring + (q % S::kStages) * S::kStageBytes;
    const uint8_t* xs = at + S::kABoxes * S::kABoxBytes;
    // Row tiles without a row of this adapter are left out; the usual case, all tiles, is a
    // branch of its own, since a test per instruction keeps the loads and MMAs from overlapping.
    uint32_t tiles = 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) tiles |= ((mask >> (8 * j)) & 0xFFu) != 0 ? 1u << j : 0u;
    auto step = [&](auto all) {
      constexpr bool kAll = decltype(all)::value;
#pragma unroll
      for (int kg = 0; kg < S::kCK / 32; ++kg) {
        uint32_t x[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (!kAll && ((tiles >> j) & 1u) == 0) continue;
          stream::ldsm_x4(smem_u32(xs) + (8 * j + i8) * 128 + (((kg * 4 + b) ^ i8) << 4), x[j]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int row = kg * 32 + 16 * s + (b >> 1) * 8 + i8;
          uint32_t w[RT][4];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            stream::ldsm_x4_trans(S::a_piece(smem_u32(at), row, r * 2 + (b & 1)), w[r]);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              if (kAll || ((tiles >> j) & 1u) != 0)
                stream::mma_bf16(acc[r][j], w[r], x[j][2 * s], x[j][2 * s + 1]);
        }
      }
    };
    if (tiles == (1u << NT) - 1u) step(std::true_type{});
    else step(std::false_type{});
    if (q - item * per_item == per_item - 1) {  // the item's last step: its rows' sums
      float* mine = sums + static_cast<size_t>(warp) * S::kRows * S::kRanks;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int row = 8 * j + 2 * t + (c & 1), rk = 16 * r + g + 8 * (c >> 1);
            if ((mask >> row) & 1u) mine[row * S::kRanks + rk] = acc[r][j][c];
            acc[r][j][c] = 0.0f;
          }
        }
      }
    }
    __syncwarp();  // the stage is read before the next load overwrites it
  }
  // (Every step issued was waited for; after a timeout the copies get another bounded wait.)
  if (!ok)
    for (int q = total - 1; q >= 0 && q >= total - S::kStages; --q)
      (void)mbar_wait(&s_full[warp][q % S::kStages], (q / S::kStages) & 1, a.timeout_ns);
  __syncwarp();

  // The tile's slots: its different adapters by first appearance.
  for (int i0 = 0; i0 < a.tile_rows; i0 += kShrinkThreads) {
    const int i = i0 + tid;
    const int mine = i < a.tile_rows ? s_tile[i] : -1;
    bool first = mine >= 0;
    const int4* all = reinterpret_cast<const int4*>(s_tile);
#pragma unroll 8
    for (int j = 0; j < (i0 + kShrinkThreads) / 4; ++j) {  // (every earlier row, four at a time)
      const int4 v = all[j];
      first = first && !((v.x == mine && 4 * j < i) || (v.y == mine && 4 * j + 1 < i) ||
                         (v.z == mine && 4 * j + 2 < i) || (v.w == mine && 4 * j + 3 < i));
    }
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, first);
    if (lane == 0) s_first[(i0 >> 5) + warp] = m;
  }
  __syncthreads();
  const int words = a.tile_rows / 32;
  int n_slots = 0;
  for (int w = 0; w < words; ++w) n_slots += __popc(s_first[w]);
  for (int i = tid; i < a.tile_rows; i += kShrinkThreads) {
    if ((s_first[i >> 5] >> (i & 31)) & 1u) {
      int at = __popc(s_first[i >> 5] & ((1u << (i & 31)) - 1u));
      for (int w = 0; w < (i >> 5); ++w) at += __popc(s_first[w]);
      s_slot[at] = s_tile[i];
    }
  }
  __syncthreads();
  if (row0 == tile0 && rank_in_cluster == 0) {
    if (tid == 0) a.n_slots[tile] = n_slots;
    for (int i = warp; i < n_slots; i += kShrinkWarps) {
      if (lane == 0) a.slots[tile * a.tile_rows + i] = s_slot[i];
      for (int w = 0; w < words; ++w) {
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, s_tile[w * 32 + lane] != s_slot[i]);
        if (lane == 0) a.masks[(tile * a.tile_rows + i) * words + w] = m;
      }
    }
  }

  // Every block finishes its share of the group's rows: the sum over blocks and warps, scaled.
  cluster_sync_all();
  for (int l = rank_in_cluster + a.cluster * warp; l < S::kRows; l += a.cluster * kShrinkWarps) {
    if (row0 + l >= a.M) break;
    const int ad = s_tile[row0 - tile0 + l];
    const float sc = ad >= 0 && a.scale != nullptr ? a.scale[ad] : 1.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.S + (row0 + l) * a.ld);
    for (int c = lane; c < a.ld / 64 * a.group / 2; c += 32) {
      uint32_t hi = 0u, lo = 0u;
      if (2 * c < a.rank && ad >= 0) {
        // All blocks' values are on their way before the first is added.
        const uint32_t here =
            smem_u32(sums + static_cast<size_t>(l) * S::kRanks + 2 * c);
        float2 part[8][kShrinkWarps];
#pragma unroll
        for (int blk = 0; blk < 8; ++blk) {
          if (blk < a.cluster) {
            const uint32_t at = mapa_shared(here, static_cast<uint32_t>(blk));
#pragma unroll
            for (int w = 0; w < kShrinkWarps; ++w)
              asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                           : "=f"(part[blk][w].x), "=f"(part[blk][w].y)
                           : "r"(at + w * S::kRows * S::kRanks * 4)
                           : "memory");
          }
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int blk = 0; blk < 8; ++blk) {
          if (blk < a.cluster) {
#pragma unroll
            for (int w = 0; w < kShrinkWarps; ++w) {
              s0 += part[blk][w].x;
              s1 += part[blk][w].y;
            }
          }
        }
        s0 *= sc;
        s1 *= sc;
        hi = pack_bf16x2(s0, s1);
        // A value that is infinite, or becomes so in bf16, has no remainder.
        const float r0 = s0 - bf16_bits_to_float(hi & 0xFFFFu);
        const float r1 = s1 - bf16_bits_to_float(hi >> 16);
        lo = pack_bf16x2(fabsf(r0) < INFINITY ? r0 : 0.0f, fabsf(r1) < INFINITY ? r1 : 0.0f);
      }
      const int at = 2 * c / a.group * 32 + c % (a.group / 2);
      out[at] = hi;
      out[at + a.group / 2] = lo;
    }
  }
  cluster_sync_all();  // no block leaves while another reads its sums
}

// ------------------------------------------------------------------ the product

constexpr int kRows = 128;               // rows of A (and accumulator lanes) per CTA
constexpr int BK = 64;                   // k-block: one 128-byte swizzle row of bf16
constexpr int kABytes = kRows * BK * 2;  // 16 KB
constexpr int kBoxBytes = 64 * BK * 2;   // 8 KB: 64 columns x 64 k-rows
constexpr int kUnitBytes = kBoxBytes / kStageUnits;  // 16 k-rows of a box
constexpr int kEpiWarps = 8;             // two per TMEM lane quarter
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStoreStage = 32 * 64;     // per epilogue warp: 32 rows x 32 bf16
constexpr int kTmemCols = 512;

// NB: 64-column boxes of B per CTA and stage. A single CTA computes 128 x 64 NB tiles with two
// accumulators; a pair of CTAs 256 x 512 (NB = 4): each holds its 128 rows of A and half of B's
// columns, two N = 256 MMAs per k-step fill all of tensor memory, and for those a CTA loads
// 48 KB where two 128 x 256 tiles would load 96.
template <bool PAIR, int NB>
struct GemmShape {
  static_assert(!PAIR || NB == 4, "pairs are wide");
  static constexpr int kTileRows = PAIR ? 256 : 128;
  static constexpr int kTileCols = PAIR ? 512 : 64 * NB;
  static constexpr int kMmaN = PAIR ? 256 : 64 * NB;
  static constexpr int kMmas = PAIR ? 2 : 1;
  static constexpr int kAccBufs = PAIR ? 1 : 2;
  static constexpr int kBBytes = NB * kBoxBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = NB == 4 ? 4 : NB == 2 ? 6 : 8;
  // Lane masks of a stage's slots (at most kStageUnits).
  static constexpr int kMaskWords = kTileRows / 32;
  static constexpr int kMaskBytes = kStageUnits * kMaskWords * 4;
  static constexpr int kIdBytes = kTileRows * 4;  // adapters of a tile's slots
  static constexpr int kSmemBytes = kStages * (kStageBytes + kMaskBytes) +
                                    kEpiWarps * kStoreStage + kIdBytes + 1024 /*align*/ +
                                    512 /*barriers*/;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  // kind::f16: D fp32, A bf16 K-major, B bf16 MN-major.
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                     (static_cast<uint32_t>(kMmaN >> 3) << 17) |
                                     (static_cast<uint32_t>(kTileRows >> 4) << 24);
};

// D[tmem] += A[smem] * B[smem] on the tensor-memory lanes whose bit in `off` is clear.
__device__ __forceinline__ void umma_bf16_ss_masked(uint32_t d, uint64_t ad, uint64_t bd,
                                                    uint32_t idesc, const uint32_t* off) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}
__device__ __forceinline__ void umma_bf16_ss_pair_masked(uint32_t d, uint64_t ad, uint64_t bd,
                                                         uint32_t idesc, const uint32_t* off) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, "
      "{%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]),
      "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}

struct GemmArgs {
  const int32_t* n_slots;
  const int32_t* slots;
  const uint32_t* masks;
  const __nv_bfloat16* addend;
  __nv_bfloat16* Y;
  int* err;
  uint64_t timeout_ns;
  int64_t M;
  int K, N;
  int units;        // pieces of B of an adapter
  int per_block;    // pieces of a k-block
  int second_step;  // bytes from a piece's first terms to its second ones in a row of the A tile
};

template <bool PAIR, int NB>
__global__ void __launch_bounds__(kThreads, 1)
lora_gemm(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
          const __grid_constant__ CUtensorMap ms, const __grid_constant__ CUtensorMap mb,
          const __grid_constant__ GemmArgs p) {
  using S = GemmShape<PAIR, NB>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = smem + S::kStages * kABytes;
  uint8_t* sM = sB + S::kStages * S::kBBytes;  // lane masks
  uint8_t* sT = sM + S::kStages * S::kMaskBytes;
  int* s_ids = reinterpret_cast<int*>(sT + kEpiWarps * kStoreStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(sT + kEpiWarps * kStoreStage + S::kIdBytes);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint64_t* ids_full = drained + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(ids_full + 1);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;  // 0: the CTA that issues the MMAs
  const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int n_units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

  // Tiles, row tiles innermost: tiles in flight share W's columns through L2. A last round of
  // pairs that would keep at most half of them busy runs as half tiles (one MMA per k-step).
  const int64_t m_tiles = (p.M + S::kTileRows - 1) / S::kTileRows;
  const int64_t n_tiles = (p.N + S::kTileCols - 1) / S::kTileCols;
  const int64_t tiles = m_tiles * n_tiles;
  const int64_t rest = tiles % n_units;
  const int64_t split = PAIR && 2 * rest <= n_units ? rest : 0;
  const int64_t first_half = tiles - split, work = tiles + split;
  auto decode = [&](int64_t id, int64_t& m_tile, int& n0, int& mmas) {
    int64_t base = id;
    int half = -1;
    if (id >= first_half && split > 0) {
      base = first_half + (id - first_half) / 2;
      half = static_cast<int>((id - first_half) & 1);
    }
    m_tile = base % m_tiles;
    n0 = static_cast<int>(base / m_tiles) * S::kTileCols + (half > 0 ? S::kTileCols / 2 : 0);
    mmas = half >= 0 ? 1 : S::kMmas;
  };
  const int num_kb = (p.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(drained, 1);
    mbar_init(ids_full, 1);
    fence_barrier_init();
    prefetch_tensormap(&mx);
    prefetch_tensormap(&mw);
    prefetch_tensormap(&ms);
    prefetch_tensormap(&mb);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(s_tmem, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(s_tmem, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncwarp();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------------------- TMA producer
      stream::Cursor c;
      long long issued = 0;
      bool ok = true, s_ready = false;
      const uint64_t keep = l2_policy(1), plain = l2_policy(0);
      uint32_t ids_phase = 0;
      for (int64_t id = unit; id < work && ok; id += n_units) {
        int64_t m_tile;
        int n0, mmas;
        decode(id, m_tile, n0, mmas);
        const int row0 =
            static_cast<int>(m_tile * S::kTileRows) + static_cast<int>(rank) * kRows;
        int slots = 0, kbs = num_kb;
        for (int kb = 0; kb < kbs; ++kb) {
          if (kb == num_kb - 1) {
            // The adapters' k-blocks follow: from here on S is needed.
            if (!s_ready) pdl_wait();
            s_ready = true;
            slots = p.n_slots[m_tile];
            kbs = num_kb + (slots * p.units + p.per_block - 1) / p.per_block;
            if (slots > 0) {  // their adapters, in whole 16-byte pieces
              const uint32_t n = static_cast<uint32_t>(slots + 3) / 4 * 16;
              mbar_arrive_expect_tx(ids_full, n);
              bulk_g2s(s_ids, p.slots + m_tile * S::kTileRows, n, ids_full);
            }
          }
          if (!mbar_wait(&empty[c.stage], c.phase ^ 1u, p.timeout_ns)) {
            record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          uint8_t* a_dst = sA + c.stage * kABytes;
          uint8_t* b_dst = sB + c.stage * S::kBBytes;
          const int boxes = PAIR ? 2 * mmas : NB;
          // Column of box i: pairs hold 128 columns of each MMA's 256 per CTA.
          auto box_col = [&](int i) {
            return PAIR ? n0 + 256 * (i >> 1) + static_cast<int>(rank) * 128 + 64 * (i & 1)
                        : n0 + 64 * i;
          };
          const uint32_t bar = PAIR ? mapa_shared(smem_u32(&full[c.stage]), 0) : 0u;
          if (kb < num_kb) {
            const uint32_t bytes = kABytes + boxes * kBoxBytes;
            if (rank == 0) mbar_arrive_expect_tx(&full[c.stage], (PAIR ? 2 : 1) * bytes);
            const int k0 = kb * BK;
            if (PAIR) tma_load_2d_pair_hint(a_dst, &mx, bar, k0, row0, keep);
            else tma_load_2d_hint(a_dst, &mx, &full[c.stage], k0, row0, keep);
            for (int i = 0; i < boxes; ++i) {
              if (PAIR)
                tma_load_3d_pair_hint(b_dst + i * kBoxBytes, &mw, bar, box_col(i), k0, 0, plain);
              else
                tma_load_3d_hint(b_dst + i * kBoxBytes, &mw, &full[c.stage], box_col(i), k0, 0,
                                 plain);
            }
          } else {
            // k-block of up to four units u = slot * units + v (a piece of 16 ranks of the slot's
            // adapter): S's columns for all of them, B's rows and the slots' lane masks.
            const int u0 = (kb - num_kb) * p.per_block;
            const int n = min(p.per_block, slots * p.units - u0);
            const int slot0 = u0 / p.units, slot1 = (u0 + n - 1) / p.units;
            const int64_t list = m_tile * S::kTileRows;
            const uint32_t mask_bytes = (slot1 - slot0 + 1) * S::kMaskWords * 4;
            const uint32_t bytes = kABytes + boxes * n * kUnitBytes;
            if (rank == 0) {
              mbar_arrive_expect_tx(&full[c.stage], (PAIR ? 2 : 1) * bytes + mask_bytes);
              bulk_g2s(sM + c.stage * S::kMaskBytes, p.masks + (list + slot0) * S::kMaskWords,
                       mask_bytes, &full[c.stage]);
            }
            const int s_col = p.units > 2 ? (u0 % p.units) / 2 * 64 : 0;
            if (PAIR) tma_load_2d_pair_hint(a_dst, &ms, bar, s_col, row0, keep);
            else tma_load_2d_hint(a_dst, &ms, &full[c.stage], s_col, row0, keep);
            if (kb == num_kb) {
              if (!mbar_wait(ids_full, ids_phase, p.timeout_ns)) {
                record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
                ok = false;
              }
              ids_phase ^= 1u;
            }
            int slot = slot0, v = u0 % p.units;
            for (int j = 0; j < n; ++j) {
              const int ad = ok ? s_ids[slot] : 0;
              for (int i = 0; i < boxes; ++i) {
                uint8_t* dst = b_dst + i * kBoxBytes + j * kUnitBytes;
                if (PAIR) tma_load_3d_pair_hint(dst, &mb, bar, box_col(i), v * kUnit, ad, plain);
                else tma_load_3d_hint(dst, &mb, &full[c.stage], box_col(i), v * kUnit, ad, plain);
              }
              if (++v == p.units) {
                v = 0;
                ++slot;
              }
            }
          }
          c.next(S::kStages);
          ++issued;
        }
      }
      // Every copy has landed before the CTA ends (pairs: both CTAs' are counted on the first's
      // barriers).
      if (rank == 0) stream::drain(full, S::kStages, c, issued, p.timeout_ns);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // -------------------------------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, s_ready = false;
      int it = 0;
      for (int64_t id = unit; id < work && ok; id += n_units, ++it) {
        int64_t m_tile;
        int n0, mmas;
        decode(id, m_tile, n0, mmas);
        const int acc = it % S::kAccBufs;
        const uint32_t acc_phase = static_cast<uint32_t>(it / S::kAccBufs) & 1u;
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, p.timeout_ns) ||
            (PAIR && !mbar_wait(&tempty[1], acc_phase ^ 1u, p.timeout_ns))) {
          record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * S::kMmaN);
        int units = 0, kbs = num_kb;
        for (int kb = 0; kb < kbs; ++kb) {
          if (kb == num_kb - 1) {
            if (!s_ready) pdl_wait();
            s_ready = true;
            units = p.n_slots[m_tile] * p.units;
            kbs = num_kb + (units + p.per_block - 1) / p.per_block;
          }
          if (!mbar_wait(&full[stage], phase, p.timeout_ns)) {
            record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_addr = smem_u32(sA + stage * kABytes);
          const uint32_t b_addr = smem_u32(sB + stage * S::kBBytes);
          // A: K-major SW128, 16 elements = 32 bytes on inside the swizzle row. B: MN-major SW128,
          // 64-column boxes kBoxBytes apart, 16 k-rows = 2048 bytes on.
          if (kb < num_kb) {
#pragma unroll
            for (int kk = 0; kk < kStageUnits; ++kk) {
              const uint64_t ad = smem_desc_sw128(a_addr + kk * 32, 16, 1024);
              for (int h = 0; h < mmas; ++h) {
                const uint64_t bd =
                    smem_desc_sw128(b_addr + 2 * h * kBoxBytes + kk * kUnitBytes, kBoxBytes, 1024);
                const uint32_t dh = d + static_cast<uint32_t>(256 * h);
                if (PAIR) umma_bf16_ss_pair(dh, ad, bd, S::kIdesc, (kb | kk) != 0 ? 1u : 0u);
                else umma_bf16_ss(dh, ad, bd, S::kIdesc, (kb | kk) != 0 ? 1u : 0u);
              }
            }
          } else {
            const int u0 = (kb - num_kb) * p.per_block, n = min(p.per_block, units - u0);
            const int slot0 = u0 / p.units;
            const uint32_t* masks = reinterpret_cast<const uint32_t*>(sM + stage * S::kMaskBytes);
            for (int j = 0; j < n; ++j) {
              const int slot = (u0 + j) / p.units, v = (u0 + j) % p.units;
              uint32_t off[S::kMaskWords];
#pragma unroll
              for (int w = 0; w < S::kMaskWords; ++w)
                off[w] = masks[(slot - slot0) * S::kMaskWords + w];
              const uint32_t s_addr = a_addr + (v % p.per_block) * 32;
              for (int h = 0; h < mmas; ++h) {
                const uint64_t bd =
                    smem_desc_sw128(b_addr + 2 * h * kBoxBytes + j * kUnitBytes, kBoxBytes, 1024);
                const uint32_t dh = d + static_cast<uint32_t>(256 * h);
                auto term = [&](uint32_t at) {
                  const uint64_t ad = smem_desc_sw128(at, 16, 1024);
                  if (PAIR) umma_bf16_ss_pair_masked(dh, ad, bd, S::kIdesc, off);
                  else umma_bf16_ss_masked(dh, ad, bd, S::kIdesc, off);
                };
                term(s_addr);
                term(s_addr + p.second_step);
              }
            }
          }
          if (PAIR) umma_commit_pair(&empty[stage], 0x3);
          else umma_commit(&empty[stage]);
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) {
          if (PAIR) umma_commit_pair(&tfull[acc], 0x3);
          else umma_commit(&tfull[acc]);
        }
      }
      if (PAIR) umma_commit_pair(drained, 0x1);
      else umma_commit(drained);
      if (!mbar_wait(drained, 0, p.timeout_ns)) record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
    }
  } else {  // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp may access TMEM lanes [32q, 32q + 32)
    const int c_first = (warp - 2) / 4;  // of its quarter's two warps: alternate 32-column chunks
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : 0u;
    int it = 0;
    for (int64_t id = unit; id < work; id += n_units, ++it) {
      int64_t m_tile;
      int n0, mmas;
      decode(id, m_tile, n0, mmas);
      const int acc = it % S::kAccBufs;
      const bool ok = mbar_wait_suspend(&tfull[acc], static_cast<uint32_t>(it / S::kAccBufs) & 1u,
                                        p.timeout_ns);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        if (lane == 0) record_error(p.err, MOE_DEVERR_WAIT_TIMEOUT);
        break;
      }
      __syncwarp();
      tc_fence_after_sync();
      const int64_t row0 = m_tile * S::kTileRows + static_cast<int64_t>(rank) * kRows + q * 32;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * S::kMmaN);
      uint8_t* buf = sT + (warp - 2) * kStoreStage;
      const int chunks = mmas * S::kMmaN / 32;
      auto release = [&](int part) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(part * 8));
          else mbar_arrive(&tempty[acc]);
        }
      };
      // 32 columns at a time, the next load under way during this one's stores.
      uint32_t ra[32];
      if (c_first < chunks) tmem_ld_32cols(t_row + c_first * 32, ra);
      bool gave_lower = false;
      for (int c = c_first; c < chunks; c += 2) {
        tmem_ld_wait();
        uint32_t w[16];
        const int64_t m = row0 + lane;
        const int col0 = n0 + c * 32;
        if (p.addend != nullptr && m < p.M) {
          const __nv_bfloat16* src = p.addend + m * p.N + col0;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (col0 + 8 * v < p.N) {
              const uint4 e = *reinterpret_cast<const uint4*>(src + 8 * v);
              const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int at = 8 * v + 2 * x;
                const float e0 = bf16_bits_to_float(ew[x] & 0xFFFFu);
                const float e1 = bf16_bits_to_float(ew[x] >> 16);
                ra[at] = __float_as_uint(__uint_as_float(ra[at]) + e0);
                ra[at + 1] = __float_as_uint(__uint_as_float(ra[at + 1]) + e1);
              }
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
          w[x] = pack_bf16x2(__uint_as_float(ra[2 * x]), __uint_as_float(ra[2 * x + 1]));
        if (c + 2 < chunks) tmem_ld_32cols(t_row + (c + 2) * 32, ra);
        if (PAIR && !gave_lower && c + 2 >= 8) {  // columns below 256 are read
          // (the load just issued, if any, reads the upper half)
          release(0);
          gave_lower = true;
        }
        if (c + 2 >= chunks) release(PAIR ? 1 : 0);
        // Through shared memory: each store instruction writes 8 whole 64-byte row segments.
        uint4* mine = reinterpret_cast<uint4*>(buf + lane * 64);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          mine[v ^ ((lane >> 1) & 3)] =
              make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        __syncwarp();
        const int sg = lane & 3, col = col0 + sg * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int l = 8 * i + (lane >> 2);
          const uint4 val = reinterpret_cast<const uint4*>(buf + l * 64)[sg ^ ((l >> 1) & 3)];
          if (row0 + l < p.M && col < p.N)
            *reinterpret_cast<uint4*>(p.Y + (row0 + l) * p.N + col) = val;
        }
        __syncwarp();
      }
      if (c_first >= chunks) release(PAIR ? 1 : 0);
    }
  }

  __syncwarp();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if (PAIR) tmem_dealloc_pair(tmem_base, kTmemCols);
    else tmem_dealloc(tmem_base, kTmemCols);
  }
  pdl_wait();  // this grid ends after the one it depends on, also where it had no tile
}

// ------------------------------------------------------------------ host side

constexpr int kSms = 148;

// 256-row pairs once they fill the device, single CTAs otherwise.
bool use_pairs(const moe_lora_problem& p) {
  return (p.M + 255) / 256 * ((p.N + 511) / 512) >= kSms / 2;
}
int tile_rows_of(const moe_lora_problem& p) { return use_pairs(p) ? 256 : 128; }
int64_t tiles_of(const moe_lora_problem& p) {
  return (p.M + tile_rows_of(p) - 1) / tile_rows_of(p);
}
int s_cols_of(const moe_lora_problem& p) {
  return (pieces_of_rank(p.rank) * kUnit + group_ranks(p.rank) - 1) / group_ranks(p.rank) * 64;
}

template <int RT, int NT>
cudaError_t launch_shrink(const ShrinkArgs& a, const LoraTensors& t, cudaStream_t stream) {
  using S = ShrinkShape<RT, NT>;
  CUtensorMap ma, mx;
  if (!make_box_map_3d_bf16(&ma, t.A, a.rank, a.K, a.L, S::kBoxRanks, S::kCK) ||
      !make_tensor_map_2d_bf16(&mx, t.X, a.K, a.M, S::kCK, S::kRows))
    return cudaErrorInvalidValue;
  auto kernel = shrink_kernel<RT, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t groups = (a.M + S::kRows - 1) / S::kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * a.cluster));
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, ma, mx, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_shrink_rank(const ShrinkArgs& a, const LoraTensors& t, cudaStream_t stream) {
  if (a.rank <= 16) return launch_shrink<1, NT>(a, t, stream);
  if (a.rank <= 32) return launch_shrink<2, NT>(a, t, stream);
  if (a.rank <= 64) return launch_shrink<4, NT>(a, t, stream);
  return launch_shrink<8, (NT > 2 ? 2 : NT)>(a, t, stream);  // (smaller groups: shared memory)
}

template <bool PAIR, int NB>
cudaError_t launch_gemm(const moe_lora_problem& p, const CUtensorMap& mx, const CUtensorMap& mw,
                        const CUtensorMap& ms, const CUtensorMap& mb,
                        const GemmArgs& g, cudaStream_t stream) {
  using S = GemmShape<PAIR, NB>;
  auto kernel = lora_gemm<PAIR, NB>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.M + S::kTileRows - 1) / S::kTileRows *
                        ((p.N + S::kTileCols - 1) / S::kTileCols);
  const int units = PAIR ? num_sms() / 2 : num_sms();
  const int64_t used = PAIR ? units : std::min<int64_t>(units, tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * used : used));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, mx, mw, ms, mb, g);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_sm100_workspace_bytes(const moe_lora_problem& p) {
  return up256(sizeof(int32_t) * tiles_of(p)) +
         up256(sizeof(int32_t) * tiles_of(p) * tile_rows_of(p)) +
         up256(sizeof(uint32_t) * tiles_of(p) * tile_rows_of(p) * (tile_rows_of(p) / 32)) +
         up256(2 * static_cast<size_t>(p.M) * s_cols_of(p));
}

cudaError_t launch_lora_sm100(const moe_lora_problem& p, const LoraTensors& t, void* scratch,
                              int* err, uint64_t timeout_ns, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(scratch);
  int32_t* n_slots = reinterpret_cast<int32_t*>(w);
  w += up256(sizeof(int32_t) * tiles_of(p));
  int32_t* slots = reinterpret_cast<int32_t*>(w);
  w += up256(sizeof(int32_t) * tiles_of(p) * tile_rows_of(p));
  uint32_t* masks = reinterpret_cast<uint32_t*>(w);
  w += up256(sizeof(uint32_t) * tiles_of(p) * tile_rows_of(p) * (tile_rows_of(p) / 32));

  ShrinkArgs a{};
  a.timeout_ns = timeout_ns;
  a.adapter = t.adapter;
  a.scale = t.scale;
  a.S = reinterpret_cast<__nv_bfloat16*>(w);
  a.n_slots = n_slots;
  a.slots = slots;
  a.masks = masks;
  a.err = err;
  a.ld = s_cols_of(p);
  a.group = group_ranks(p.rank);
  a.M = p.M;
  a.K = static_cast<int>(p.K);
  a.L = p.adapters;
  a.rank = p.rank;
  a.tile_rows = tile_rows_of(p);
  // Single CTAs: the tile width whose rounds cost least. A k-block of a 128 x 64 NB tile loads
  // 16 + 8 NB KB, which takes longer than its MMAs (64 bytes per clock and SM from L2).
  const bool pairs = use_pairs(p);
  const int64_t m_tiles = (p.M + 127) / 128;
  auto tiles_with = [&](int nb) { return m_tiles * ((p.N + 64 * nb - 1) / (64 * nb)); };
  auto cost = [&](int nb) { return (tiles_with(nb) + kSms - 1) / kSms * (2 + nb); };
  int nb = cost(2) <= cost(1) ? 2 : 1;
  if (cost(4) <= cost(nb)) nb = 4;
  const int64_t ctas = pairs ? kSms : std::min<int64_t>(kSms, tiles_with(nb));

  // Groups of 32 rows share an adapter's reads; few rows take groups of 8, whose different
  // adapters then spread over more blocks. A group's K goes over as many blocks (at most 8) as
  // the device has left (one round of the large groups' blocks, which take an SM each: 4096 rows
  // 358 us against 369 in two), but where the product leaves SMs free the shrink keeps to those:
  // a CTA of the product that waits for its SM starts late by the whole shrink (200 rows by 5000
  // columns: 29 us with 100 blocks beside 80 CTAs, 22 us with 50).
  const bool small = p.M <= 512;
  const int64_t groups = small ? (p.M + 7) / 8 : (p.M + 31) / 32;
  const int64_t room = kSms - ctas >= groups ? kSms - ctas : small ? 2 * kSms : kSms;
  a.cluster = 1;
  while (a.cluster < 8 && groups * a.cluster * 2 <= room && a.K >= 256 * a.cluster * 2)
    a.cluster *= 2;
  cudaError_t e =
      small ? launch_shrink_rank<1>(a, t, stream) : launch_shrink_rank<4>(a, t, stream);
  if (e != cudaSuccess) return e;

  CUtensorMap mx, mw, ms, mb;
  if (!make_tensor_map_2d_bf16(&mx, t.X, p.K, p.M, 64, kRows) ||
      !make_tensor_map_2d_bf16(&ms, a.S, a.ld, p.M, 64, kRows) ||
      !make_box_map_3d_bf16(&mw, t.W, p.N, p.K, 1, 64, BK) ||
      !make_box_map_3d_bf16(&mb, t.B, p.N, p.rank, p.adapters, 64, kUnit))
    return cudaErrorInvalidValue;
  GemmArgs g{};
  g.n_slots = n_slots;
  g.slots = slots;
  g.masks = masks;
  g.addend = static_cast<const __nv_bfloat16*>(t.addend);
  g.Y = static_cast<__nv_bfloat16*>(t.Y);
  g.err = err;
  g.timeout_ns = timeout_ns;
  g.M = p.M;
  g.K = static_cast<int>(p.K);
  g.N = static_cast<int>(p.N);
  g.units = pieces_of_rank(p.rank);
  g.per_block = block_pieces(p.rank);
  g.second_step = 2 * group_ranks(p.rank);
  if (pairs) return launch_gemm<true, 4>(p, mx, mw, ms, mb, g, stream);
  if (nb == 4) return launch_gemm<false, 4>(p, mx, mw, ms, mb, g, stream);
  if (nb == 2) return launch_gemm<false, 2>(p, mx, mw, ms, mb, g, stream);
  return launch_gemm<false, 1>(p, mx, mw, ms, mb, g, stream);
}

}  // namespace moe
