// A projection shared by all rows beside the low-rank adapter of each row's own request:
//   Y[m] = addend[m] + X[m] W + scale[a] (X[m] A[a]) B[a],   a = adapter[m] (-1: none)
// for at most 64 rows, in one cooperative kernel (more rows: lora_sm100.cu, lora_f32.cu).
//
// What bounds it: one pass over W (and over the used adapters). W runs through the ring of
// stream.cuh in equal shares per block, as the few-token layer's down projection does. The
// adapters' part hides behind it:
//   1. Shrink. While the ring fills, the consumers compute S = X A: block (row, slice of K), a
//      16-byte piece of an A row per thread, fp32 partial sums to L2. The block arrives at the
//      grid barrier and goes on with W.
//   2. Expand, scale S B[a] for the rows of a tile, in fp32 on the CUDA cores, cut into units
//      (4 rows x 128 columns x 16 ranks) and spread over the tile's stages: a unit's loads of B
//      are issued in one stage and used in the next, so their latency passes under the stream.
//      (All at the end of the tile, 48 rows of 48 adapters took 81 us where W takes 21.) A block
//      that has a share of a tile takes the same share of its units. The barrier is waited for
//      at the first unit.
// S stays fp32 throughout, so the only rounding is that of Y.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "stream.cuh"

namespace moe {

namespace {

using namespace stream;

constexpr int kMaxRank = 128;
// 128 values of a row: bf16 with 16 bytes against bank conflicts, fp32 (read as broadcasts) plain.
constexpr int kRowPitch128 = 272, kRowPitch128F32 = 512;

struct LoraArgs {
  const void* X;
  const void* A;
  const void* B;
  const float* scale;
  const int32_t* adapter;
  const void* addend;
  void* Y;
  float* part_s;   // [slices][M][rank]
  float* part;     // [grid][2][part_floats]: sums of shared tiles
  float* delta;    // [grid][part_floats]: adapters' part of the block's current tile
  int* counters;   // [kMaxGrid]: arrivals at shared tiles
  int* bar;        // [2] workspace header ints, zero at rest
  int* err;
  int64_t part_floats;
  uint64_t timeout_ns;
  int M, K, N, L, rank, slices;
};

struct LoraTables {
  uint64_t full[kMaxStages];
  uint64_t rows_full[kMaxStages];
  uint64_t empty[kMaxStages];
  int adapter[kMaxRows];  // -1: none
  int flag;
};

constexpr size_t kMaxSmem = 232448;
constexpr size_t s_bytes(int M, int rank) {
  return (sizeof(float) * static_cast<size_t>(M) * rank + 15) & ~size_t(15);
}
__host__ __device__ constexpr size_t lora_ring_bytes(int M, int rank) {
  return (kMaxSmem - 1024 - sizeof(float) * kRedFloats - s_bytes(M, rank) - sizeof(LoraTables)) &
         ~size_t(1023);
}
// A stage's rows, whole tiles of 8.
__host__ __device__ constexpr int lora_row_bytes(int M, bool f32) {
  return (M + 7) / 8 * 8 * (f32 ? kRowPitch128F32 : kRowPitch128);
}
__host__ __device__ constexpr int lora_stages(int M, int rank, bool f32) {
  const int s = static_cast<int>(lora_ring_bytes(M, rank) /
                                 (kStageBytes + static_cast<size_t>(lora_row_bytes(M, f32))));
  return s < kMaxStages ? s : kMaxStages;
}
static_assert(lora_stages(kMaxRows, kMaxRank, false) >= kInFlight, "ring");
static_assert(lora_stages(kMaxRows, kMaxRank, true) >= 2, "ring");

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint4 a =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
      v[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
    }
  }
}

// This block's partial S: row blockIdx.x % M over one slice of K. kVec values of a row of A per
// thread (16 bytes).
template <bool F32>
__device__ void shrink(const LoraArgs& a, const LoraTables& tb, float* red, int tid) {
  constexpr int kVec = F32 ? 4 : 8;
  const int m = static_cast<int>(blockIdx.x) % a.M, slice = static_cast<int>(blockIdx.x) / a.M;
  if (slice >= a.slices) return;
  const int ad = tb.adapter[m];
  if (ad < 0) return;  // nobody reads this row's sums
  const int per_row = a.rank / kVec, subs = kConsumers / per_row;
  const int chunk = (a.K + a.slices - 1) / a.slices;
  const int k0 = min(a.K, slice * chunk), k1 = min(a.K, k0 + chunk);
  const int v = tid % per_row, sub = tid / per_row;
  float acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
  if (sub < subs) {
#pragma unroll 4
    for (int k = k0 + sub; k < k1; k += subs) {
      const int64_t at = static_cast<int64_t>(m) * a.K + k;
      const float x = F32 ? __ldg(static_cast<const float*>(a.X) + at)
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(a.X)[at]);
      float w[8];
      load8<F32>(a.A, (static_cast<int64_t>(ad) * a.K + k) * a.rank + v * kVec, w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = fmaf(x, w[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) red[sub * a.rank + v * kVec + i] = acc[i];
  }
  named_bar_sync(kBarConsumers, kConsumers);
  if (tid < a.rank) {
    float s = 0.0f;
    for (int q = 0; q < subs; ++q) s += red[q * a.rank + tid];
    a.part_s[(static_cast<int64_t>(slice) * a.M + m) * a.rank + tid] = s;
  }
}

// Adds the addend to two columns of a row and stores them.
template <bool F32>
__device__ __forceinline__ void finish(const LoraArgs& a, int m, int n, float2 v) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = static_cast<int64_t>(m) * a.N + n;
  if constexpr (F32) {
    if (a.addend != nullptr) {
      const float2 b = *reinterpret_cast<const float2*>(static_cast<const float*>(a.addend) + at);
      v.x += b.x;
      v.y += b.y;
    }
    *reinterpret_cast<float2*>(static_cast<float*>(a.Y) + at) = v;
  } else {
    if (a.addend != nullptr) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(a.addend) + at);
      v.x += bf16_bits_to_float(w & 0xFFFFu);
      v.y += bf16_bits_to_float(w >> 16);
    }
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.Y) + at) = pack_bf16x2(v.x, v.y);
  }
}

// The adapters' part of a tile in units: thread tid holds place i = tid + kConsumers * it of the
// epilogue's order (row i / kPairs, two columns) for iteration it, kUnitRanks ranks at a time.
constexpr int kUnitRanks = 16;

template <int WK>
struct Expand {
  static constexpr bool kIsF32 = WK == kF32;
  using P = Places<WK>;
  using Word = typename std::conditional<kIsF32, float2, uint32_t>::type;
  Word b[kUnitRanks];
  float2 sum = make_float2(0.0f, 0.0f);
  int unit = -1;  // whose words are loaded; -1: none

  __device__ __forceinline__ static int chunks(int rank) {
    return (rank + kUnitRanks - 1) / kUnitRanks;
  }
  __device__ __forceinline__ static int iterations(int M) {
    return (M * P::kPairs + kConsumers - 1) / kConsumers;
  }
  // Loads unit u (iteration u / chunks, ranks from (u % chunks) * kUnitRanks).
  __device__ __forceinline__ void issue(const LoraArgs& a, const LoraTables& tb, int u, int col0,
                                        int tid) {
    unit = u;
    const int n_chunks = chunks(a.rank);
    const int i = tid + kConsumers * (u / n_chunks), r0 = (u % n_chunks) * kUnitRanks;
    const int m = P::row(i), n = col0 + P::col(i);
    const int ad = m < a.M && n < a.N ? tb.adapter[m] : -1;
    const int64_t base = (static_cast<int64_t>(ad) * a.rank + r0) * a.N + n;
#pragma unroll
    for (int r = 0; r < kUnitRanks; ++r) {
      if constexpr (kIsF32) {
        b[r] = make_float2(0.0f, 0.0f);
        if (ad >= 0 && r0 + r < a.rank)
          b[r] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.B) + base +
                                                       static_cast<int64_t>(r) * a.N));
      } else {
        b[r] = 0u;
        if (ad >= 0 && r0 + r < a.rank)
          b[r] = __ldg(reinterpret_cast<const uint32_t*>(
              static_cast<const __nv_bfloat16*>(a.B) + base + static_cast<int64_t>(r) * a.N));
      }
    }
  }
  // Multiplies the loaded unit by S (rows past the rank and rows without an adapter: no terms);
  // after a place's last ranks its sum goes to `delta`.
  __device__ __forceinline__ void complete(const LoraArgs& a, const LoraTables& tb, const float* S,
                                           float2* delta, int tid) {
    if (unit < 0) return;
    const int n_chunks = chunks(a.rank), it = unit / n_chunks, r0 = (unit % n_chunks) * kUnitRanks;
    const int i = tid + kConsumers * it, m = P::row(i);
    if (r0 == 0) sum = make_float2(0.0f, 0.0f);
    if (m < a.M && tb.adapter[m] >= 0) {
      const float* s = S + m * a.rank + r0;
#pragma unroll
      for (int r = 0; r < kUnitRanks; ++r) {
        if (r0 + r < a.rank) {
          float2 v;
          if constexpr (kIsF32) v = b[r];
          else v = make_float2(bf16_bits_to_float(b[r] & 0xFFFFu), bf16_bits_to_float(b[r] >> 16));
          sum.x = fmaf(s[r], v.x, sum.x);
          sum.y = fmaf(s[r], v.y, sum.y);
        }
      }
    }
    if (r0 + kUnitRanks >= a.rank) delta[i] = sum;
    unit = -1;
  }
};

template <int WK, int NT>
__global__ void __launch_bounds__(kThreads, 1)
lora_few_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ LoraArgs a) {
  using S = Shape<WK>;
  using P = Places<WK>;
  constexpr bool kIsF32 = WK == kF32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + lora_ring_bytes(a.M, a.rank));
  float* sums = red + kRedFloats;  // S [M][rank], scaled
  LoraTables& tb = *reinterpret_cast<LoraTables*>(reinterpret_cast<uint8_t*>(sums) +
                                                  s_bytes(a.M, a.rank));
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
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&tb.full[i], 1);
      mbar_init(&tb.rows_full[i], 1);
      mbar_init(&tb.empty[i], kConsumerWarps);
    }
    fence_barrier_init();
    a.counters[me] = 0;  // seen by the others after the grid barrier
  }
  if (tid >= kConsumers && tid < kConsumers + a.M) {
    const int m = tid - kConsumers, ad = a.adapter[m];
    if (ad < -1 || ad >= a.L) record_error(a.err, MOE_DEVERR_BAD_INDEX);
    tb.adapter[m] = ad >= 0 && ad < a.L ? ad : -1;
  }
  __syncthreads();

  const int steps = (a.K + 2 * kBoxRows - 1) / (2 * kBoxRows);
  const int tiles = (a.N + S::kCols - 1) / S::kCols;
  SplitK sp{static_cast<long long>(tiles) * steps, 0};
  sp.grid = static_cast<int>(min(static_cast<long long>(G), sp.total));
  const long long s0 = me < sp.grid ? sp.start(me) : 0, s1 = me < sp.grid ? sp.start(me + 1) : 0;

  if (warp >= kConsumerWarps) {
    give_registers<kProducerRegs>();
    if (warp == kWeightWarp) {
      if (lane == 0) {
        const uint64_t policy = l2_policy(-1);
        Cursor c;
        bool good = true;
        long long issued = 0;
        for (long long s = s0; s < s1; ++s) {
          if (!(good = acquire_weights(ring, c, issued, a.timeout_ns))) break;
          const int col = static_cast<int>(s / steps) * S::kCols;
          const int row = static_cast<int>(s % steps) * 2 * kBoxRows;
          uint8_t* dst = smem + static_cast<size_t>(c.stage) * kStageBytes;
          uint64_t* bar = &tb.full[c.stage];
          tma_load_3d_hint(dst, &mw, bar, col, row, 0, policy);
          tma_load_3d_hint(dst + kBoxBytes, &mw, bar, col + S::kBoxCols, row, 0, policy);
          tma_load_3d_hint(dst + 2 * kBoxBytes, &mw, bar, col, row + kBoxRows, 0, policy);
          tma_load_3d_hint(dst + 3 * kBoxBytes, &mw, bar, col + S::kBoxCols, row + kBoxRows, 0,
                           policy);
          c.next(ring.stages);
          ++issued;
        }
        if (!good) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
        drain(tb.full, ring.stages, c, issued, a.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kRowWarp) {
      constexpr int kEl = kIsF32 ? 4 : 2;
      Cursor c;
      bool good = true;
      long long issued = 0;
      for (long long s = s0; s < s1; ++s) {
        const int k = static_cast<int>(s % steps) * 2 * kBoxRows;
        const uint32_t bytes = static_cast<uint32_t>(min(2 * kBoxRows, a.K - k) * kEl);
        good = mbar_wait(&tb.empty[c.stage], c.phase ^ 1u, a.timeout_ns);
        good = __all_sync(0xFFFFFFFFu, good);
        if (!good) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&tb.rows_full[c.stage], bytes * static_cast<uint32_t>(a.M));
        __syncwarp();
        for (int m = lane; m < a.M; m += 32)
          bulk_g2s(ring.rows + c.stage * ring.row_bytes +
                       m * (kIsF32 ? kRowPitch128F32 : kRowPitch128),
                   static_cast<const uint8_t*>(a.X) + (static_cast<int64_t>(m) * a.K + k) * kEl,
                   bytes, &tb.rows_full[c.stage]);
        c.next(ring.stages);
        ++issued;
      }
      if (!good && lane == 0) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
      drain(tb.rows_full, ring.stages, c, issued, a.timeout_ns);
      __syncwarp();
    } else if (warp >= kConsumerWarps + 2) {
      // The remaining warps bring the adapters' columns of this block's tiles to L2 ahead of the
      // epilogues that read them.
      constexpr int kEl = kIsF32 ? 4 : 2;
      for (long long s = s0; s < s1; s += steps - s % steps) {
        const int col = static_cast<int>(s / steps) * S::kCols;
        for (int i = tid - (kConsumers + 64); i < a.M * a.rank; i += 64) {
          const int ad = tb.adapter[i / a.rank];
          if (ad < 0) continue;
          const uint8_t* p = static_cast<const uint8_t*>(a.B) +
                             ((static_cast<int64_t>(ad) * a.rank + i % a.rank) * a.N + col) * kEl;
          for (int q = 0; q < S::kCols * kEl; q += 128)
            if (col * kEl + q < a.N * kEl)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(p + q) : "memory");
        }
      }
    }
  } else {
    take_registers<kConsumerRegs>();
    shrink<kIsF32>(a, tb, red, tid);
    grid_arrive(a.bar, tid);
    bool ok = true, have_s = false;
    // Before the first epilogue: every block's share of S, and the counters.
    auto take_s = [&] {
      if (have_s) return;
      have_s = true;
      if (!grid_wait(a.bar, G, tid, &tb.flag, a.timeout_ns, a.err)) ok = false;
      const int n = a.M * a.rank;
      int per = 1;  // threads per value, over the slices
      while (per * 2 <= a.slices && per * 2 * n <= kConsumers) per *= 2;
      const int part = per > 1 ? tid / n : 0;
      for (int i = per > 1 ? tid % n : tid; i < n && part < per; i += kConsumers) {
        float s = 0.0f;
        if (tb.adapter[i / a.rank] >= 0) {
#pragma unroll 8
          for (int q = part; q < a.slices; q += per)
            s += __ldcg(a.part_s + static_cast<int64_t>(q) * n + i);
        }
        if (per > 1) red[part * n + i] = s;
        else sums[i] = s;
      }
      named_bar_sync(kBarConsumers, kConsumers);
      for (int i = tid; i < n; i += kConsumers) {
        float s = per > 1 ? 0.0f : sums[i];
        if (per > 1)
          for (int q = 0; q < per; ++q) s += red[q * n + i];
        const int ad = tb.adapter[i / a.rank];
        sums[i] = ad >= 0 && a.scale != nullptr ? s * __ldg(a.scale + ad) : s;
      }
      named_bar_sync(kBarConsumers, kConsumers);
    };
    Cursor cur;
    const int first_row = (warp >> 2) * kBoxRows + warp_row<WK>(warp);
    for (long long s = s0; s < s1;) {
      const long long tile = s / steps;
      const int k0 = static_cast<int>(s - tile * steps);
      const int k1 = static_cast<int>(min(static_cast<long long>(steps), k0 + (s1 - s)));
      const int cb = static_cast<int>(tile);
      Acc<WK, NT> acc;
      acc.zero();
      // Units [u_begin, u_end) of the tile are this block's, due evenly over its stages.
      Expand<WK> ex;
      float2* delta = reinterpret_cast<float2*>(a.delta + static_cast<int64_t>(me) * a.part_floats);
      const int iters = Expand<WK>::iterations(a.M), chunks = Expand<WK>::chunks(a.rank);
      auto units_before = [&](int k) {  // whole iterations, so that a place has one block
        return static_cast<int>(static_cast<long long>(iters) * k / steps) * chunks;
      };
      const int u_begin = units_before(k0), u_end = units_before(k1);
      int u_next = u_begin;
      for (int k = k0; k < k1; ++k) {
        const int due = u_begin + static_cast<int>(static_cast<long long>(u_end - u_begin) *
                                                   (k + 1 - k0) / (k1 - k0));
        if (ex.unit >= 0 || due - u_next > 1) take_s();
        ex.complete(a, tb, sums, delta, tid);
        for (; u_next < due; ++u_next) {
          ex.complete(a, tb, sums, delta, tid);  // more than one unit a stage: one at a time
          ex.issue(a, tb, u_next, cb * S::kCols, tid);
        }
        if (ok && (!mbar_wait(&tb.full[cur.stage], cur.phase, a.timeout_ns) ||
                   !mbar_wait(&tb.rows_full[cur.stage], cur.phase, a.timeout_ns))) {
          ok = false;
          record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
        }
        const uint32_t box = smem_u32(ring.weights) +
                             static_cast<uint32_t>(cur.stage) * kStageBytes +
                             static_cast<uint32_t>(warp >> 1) * kBoxBytes;
        const uint8_t* rows = ring.rows + cur.stage * ring.row_bytes;
        const int at = k * 2 * kBoxRows + first_row;
        if constexpr (kIsF32) {
          multiply_f32<NT>(acc, box, warp, lane, rows + first_row * 4, kRowPitch128F32, a.M, at,
                           a.K);
          __syncwarp();
          if (lane == 0) mbar_arrive(&tb.empty[cur.stage]);
        } else {
          Weights<WK> w;
          Frag<WK, NT, false> f;
          w.load(box, warp, lane);
          f.load_rows(rows, kRowPitch128, first_row / 32, at, a.K, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&tb.empty[cur.stage]);
          multiply<WK, NT, false>(acc, w, f);
        }
        cur.next(ring.stages);
      }
      take_s();
      ex.complete(a, tb, sums, delta, tid);
      const bool whole = k0 == 0 && k1 == steps;
      float2* mine = reinterpret_cast<float2*>(
          a.part + (static_cast<int64_t>(me) * 2 + (k0 > 0 ? 0 : 1)) * a.part_floats);
      for (int j = 0; j < NT && 8 * j < a.M; ++j) {
        put_tile<WK, NT>(red, acc, j, warp, lane);
        named_bar_sync(kBarConsumers, kConsumers);
        for (int i = tid; i < P::kCount; i += kConsumers) {
          float2 v = take_pair<WK>(red, -1, P::row(i), P::col(i));
          const int place = j * P::kCount + i;  // written by this thread, where it is a unit's
          const int unit = place / kConsumers * chunks;
          if (unit >= u_begin && unit < u_end) {
            const float2 d = delta[place];
            v.x += d.x;
            v.y += d.y;
          }
          if (whole) finish<kIsF32>(a, 8 * j + P::row(i), cb * S::kCols + P::col(i), v);
          else mine[place] = v;
        }
        named_bar_sync(kBarConsumers, kConsumers);
      }
      if (!whole) {
        const int first = sp.owner(tile * steps), last = sp.owner(tile * steps + steps - 1);
        if (last_to_finish(a.counters + first, last - first + 1, tid, &tb.flag)) {
          for (int i = tid; i < (a.M + 7) / 8 * P::kCount; i += kConsumers) {
            float2 v = make_float2(0.0f, 0.0f);
            for (int b = first; b <= last; ++b) {
              const float2 p = __ldcg(reinterpret_cast<const float2*>(
                                          a.part + (static_cast<int64_t>(b) * 2 +
                                                    (b == first ? 1 : 0)) * a.part_floats) + i);
              v.x += p.x;
              v.y += p.y;
            }
            finish<kIsF32>(a, P::row(i), cb * S::kCols + P::col(i), v);
          }
        }
      }
      s += k1 - k0;
    }
    take_s();  // every block waits for the barrier, so that the counters may return to zero
  }

  // The last block out returns the barrier counters to zero for the next launch.
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&a.bar[1], 1) == G - 1) {
      atomicExch(&a.bar[0], 0);
      atomicExch(&a.bar[1], 0);
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
cudaError_t launch_few(const moe_lora_problem& p, const LoraArgs& a, const void* W,
                       cudaStream_t stream) {
  CUtensorMap mw;
  if (!make_stream_map(&mw, W, WK, p.N, p.K, 1)) return cudaErrorInvalidValue;
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
  e = cudaLaunchKernelEx(&cfg, kernel, mw, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_few_workspace_bytes(const moe_lora_problem& p) {
  return up256(sizeof(float) * lora_slices(p.M, p.K) * p.M * p.rank) +
         up256(sizeof(int) * kMaxGrid) +
         up256(sizeof(float) * 3 * kMaxGrid * lora_part_floats(p.M));
}

cudaError_t launch_lora_few(const moe_lora_problem& p, const LoraTensors& t, void* scratch,
                            int* err, int* bar, uint64_t timeout_ns, cudaStream_t stream) {
  LoraArgs a{};
  a.X = t.X;
  a.A = t.A;
  a.B = t.B;
  a.scale = t.scale;
  a.adapter = t.adapter;
  a.addend = t.addend;
  a.Y = t.Y;
  const int max_slices = lora_slices(p.M, p.K);  // what the workspace holds
  a.slices = std::max(1, std::min<int>(max_slices, std::min(num_sms(), kMaxGrid) / p.M));
  uint8_t* w = static_cast<uint8_t*>(scratch);
  a.part_s = reinterpret_cast<float*>(w);
  w += up256(sizeof(float) * max_slices * p.M * p.rank);
  a.counters = reinterpret_cast<int*>(w);
  w += up256(sizeof(int) * kMaxGrid);
  a.part = reinterpret_cast<float*>(w);
  a.part_floats = lora_part_floats(p.M);
  a.delta = a.part + 2 * kMaxGrid * a.part_floats;
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
    if (nt == 1) return launch_few<kF32, 1>(p, a, t.W, stream);
    if (nt == 2) return launch_few<kF32, 2>(p, a, t.W, stream);
    if (nt <= 4) return launch_few<kF32, 4>(p, a, t.W, stream);
    return launch_few<kF32, 8>(p, a, t.W, stream);
  }
  if (nt == 1) return launch_few<kBF16, 1>(p, a, t.W, stream);
  if (nt == 2) return launch_few<kBF16, 2>(p, a, t.W, stream);
  if (nt == 3) return launch_few<kBF16, 3>(p, a, t.W, stream);
  if (nt == 4) return launch_few<kBF16, 4>(p, a, t.W, stream);
  if (nt <= 6) return launch_few<kBF16, 6>(p, a, t.W, stream);
  return launch_few<kBF16, 8>(p, a, t.W, stream);
}

}  // namespace moe
