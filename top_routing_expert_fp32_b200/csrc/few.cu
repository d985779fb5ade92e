// The whole layer for a few tokens (at most 64) in one cooperative kernel:
//   z = x W_r + b,  softmax, top-k, capacity,  H = g act(x W1_e) (.) (x W2_e),
//   out[t] = sum over t's kept experts of H W3_e
// (Grok-1 book ch.5, 5.2 and 5.3.5; LLMs-from-scratch ch.12, 12.1; walkthrough 1.1-3.2).
//
// What bounds it: one pass over the matrices of the experts that keep a token. Everything else
// is latency, so there is one launch and two grid barriers:
//   1. Router. The D reduction is cut over the blocks (fp32 partial logits to L2), barrier, then
//      every block adds the partials and takes all decisions itself (one warp per token; ballots
//      for the capacity positions), which is cheaper than a second exchange.
//   2. Up. The (expert, 128 columns of F, 64 rows of D) stages of W1 and W2 run through the
//      ring (stream.cuh) in equal shares per block. The gate is folded into H here, so that the
//      combine below is a plain sum. H is kept as two bf16 terms (16 bits of mantissa): the
//      second term costs one more instruction per stage on tensor cores that are idle anyway, and
//      leaves the output's own rounding as the only one that shows.
//   3. Barrier, while the ring already fills with W3, which does not depend on H.
//   4. Down. Stages ordered (128 columns of D, expert, 128 rows of F): a column block's sum runs
//      over all experts in shared memory per token, which is the combine.
// (64 columns for fp32 weights, 256 for 8-bit ones: 256 bytes either way.)
// Rows of an expert are its kept tokens in capacity order, read from X by index: no
// permutation is written. More than 32 rows of an expert (8-bit weights: 16) are several pieces,
// each reading the expert's weights: the sums of so many rows are about what the registers hold. A
// tile shared by several blocks is summed by the last to finish, in block order, so equal inputs
// give equal bits.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "stream.cuh"

namespace moe {

namespace {

using namespace stream;

constexpr int kMaxRecords = kMaxRows * 8;
constexpr int kMaxE = 64;
// Products: an expert's kept rows in pieces of at most Shape::kPieceRows (16 or 32).
constexpr int kMaxParts = kMaxE + kMaxRecords / 16;
constexpr int kMaxWarps = 16;
constexpr int kCounters = kMaxGrid * (kMaxWarps + 1);
constexpr int kMaxSlices = 64;  // pieces of D of the router's partial logits

struct FewArgs {
  const void* X;
  const float* W_r;
  const float* bias;
  const float* S1;
  const float* S2;
  const float* S3;
  void* out;
  float* logits;
  int32_t* idx;
  float* gate;
  int32_t* load;
  int32_t* offsets;
  int32_t* pos;
  uint8_t* dropped;
  float* colsum;
  float* part_logits;  // [slices][N][E]
  float* part;         // [grid][2][part_floats]: sums of shared tiles
  int* counters;       // [kMaxGrid][kMaxWarps]: the warps' arrivals at shared up tiles, then
                       // [kMaxGrid]: the blocks' at shared down tiles
  void* H;             // see h_groups
  int* bar;            // [2] workspace header ints, zero at rest
  int* err;
  int64_t part_floats;
  int64_t capacity;
  uint64_t timeout_ns;
  int N, D, F, E, k;
  int tokens_per_group, slices;  // router split
  bool renorm, token_major, renorm_kept;
  int act;
};

struct Part {
  int16_t expert;
  int16_t row0;  // first row of the piece among all kept rows
  int16_t n;     // rows, at least 1
  int16_t tile;  // its first tile of 8 rows in H
};

struct Tables {
  uint64_t full[kMaxStages];
  uint64_t rows_full[kMaxStages];
  uint64_t empty[kMaxStages];
  float gate[kMaxRecords];
  float row_gate[kMaxRecords];
  float zmax[kMaxRows];
  float sum[kMaxRows];
  int load[kMaxE];
  int off[kMaxE + 1];
  Part part[kMaxParts];
  int n_parts;
  int max_rows;  // of any piece
  int flag;
  int16_t row_tok[kMaxRecords];
  int16_t pos[kMaxRecords];
  int16_t pos_order[kMaxRecords];
  uint8_t idx[kMaxRecords];    // of record (t, j) at t * k + j
  uint8_t order[kMaxRecords];  // the same in capacity order
};

// Shared memory: the ring, the warps' sums, the column block's sums per token (first the
// logits), the tables. The ring takes what the batch leaves; how many stages that makes depends
// on the rows of the largest piece, which the kernel learns from the routing.
template <int WK>
constexpr size_t out_bytes(int N, int E) {
  return (sizeof(float) * static_cast<size_t>(N) *
              static_cast<size_t>(E > Shape<WK>::kCols ? E : Shape<WK>::kCols) + 15) & ~size_t(15);
}
constexpr size_t kMaxSmem = 232448;
template <int WK>
__host__ __device__ constexpr size_t ring_bytes(int N, int E) {
  return (kMaxSmem - 1024 - kRedBytes - out_bytes<WK>(N, E) - sizeof(Tables)) &
         ~size_t(1023);
}
__host__ __device__ constexpr int ring_stages(size_t bytes, int row_tiles) {
  const int s =
      static_cast<int>(bytes / (kStageBytes + static_cast<size_t>(row_tiles) * kTileBytes));
  return s < kMaxStages ? s : kMaxStages;
}
static_assert(ring_stages(ring_bytes<kW8>(kMaxRows, kMaxE), 2) >= 2, "ring");
static_assert(ring_stages(ring_bytes<kBF16>(kMaxRows, kMaxE), 4) >= kInFlight, "ring");
static_assert(ring_stages(ring_bytes<kF32>(kMaxRows, kMaxE), 4) >= kInFlight, "ring");

// H. 16-bit kinds: per tile of 8 rows and 32 values of F two planes (the first and the second
// bf16 term) of 32 threads x 16 bytes, each thread's four pairs (stream.cuh's Frag):
// one coalesced load per plane. fp32: plain rows.
__host__ __device__ inline int64_t h_groups(int64_t F) { return (F + 255) / 256 * 8; }
constexpr int kHGroupBytes = 1024;
__host__ __device__ inline int64_t h_row_f32(int64_t F) { return (F + 63) / 64 * 64; }

__device__ __forceinline__ float act_value(int act, float a) {
  if (act == MOE_ACT_SILU) return activation<MOE_ACT_SILU>(a);
  if (act == MOE_ACT_GELU_ERF) return activation<MOE_ACT_GELU_ERF>(a);
  return activation<MOE_ACT_GELU_TANH>(a);
}

// Order-preserving integer image of a float (+0 and -0 alike), for selection by maximum; never 0,
// whatever the float.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t u = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return u != 0u ? u : 1u;
}

// ------------------------------------------------------------------ router

// This block's partial logits: tokens [t0, t1) over rows [d0, d1) of D.
template <int WK>
__device__ void partial_logits(const FewArgs& a, float* red, int tid) {
  constexpr int kConsumers = Team<WK>::kConsumers;
  const int groups = (a.N + a.tokens_per_group - 1) / a.tokens_per_group;
  const int group = static_cast<int>(blockIdx.x) % groups;
  const int slice = static_cast<int>(blockIdx.x) / groups;
  if (slice >= a.slices) return;
  const int t0 = group * a.tokens_per_group;
  const int nt = min(a.tokens_per_group, a.N - t0);
  const int rows = (a.D + a.slices - 1) / a.slices;
  const int d0 = min(a.D, slice * rows), d1 = min(a.D, d0 + rows);
  int ep = 1;
  while (ep < a.E) ep <<= 1;
  const int e = tid & (ep - 1), sl = tid / ep, subs = kConsumers / ep;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  if (e < a.E) {
    constexpr int kAtOnce = WK == kW8 ? 2 : 4;  // rows of W_r whose loads are on their way at once
    for (int d = d0 + sl; d < d1; d += kAtOnce * subs) {
      float w[kAtOnce], x[kAtOnce][8];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int du = d + u * subs;
        const bool in = du < d1;
        w[u] = in ? __ldg(a.W_r + static_cast<int64_t>(du) * a.E + e) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[u][i] = 0.0f;
          if (in && i < nt) {
            const int64_t at = static_cast<int64_t>(t0 + i) * a.D + du;
            x[u][i] = WK == kF32 ? __ldg(static_cast<const float*>(a.X) + at)
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(a.X)[at]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(x[u][i], w[u], acc[i]);
    }
  }
  for (int i = 0; i < nt; ++i) {  // sum the row interleave in order
    float v = acc[0];
#pragma unroll
    for (int q = 1; q < 8; ++q)
      if (q == i) v = acc[q];
    red[(i * subs + sl) * ep + e] = v;
  }
  bar_sync(kBarConsumers, kConsumers);
  for (int o = tid; o < nt * ep; o += kConsumers) {
    const int i = o / ep, ee = o & (ep - 1);
    if (ee < a.E) {
      float s = 0.0f;
#pragma unroll 8
      for (int q = 0; q < subs; ++q) s += red[(i * subs + q) * ep + ee];
      a.part_logits[(static_cast<int64_t>(slice) * a.N + t0 + i) * a.E + ee] = s;
    }
  }
}

// All logits in shared memory, z[t * E + e].
template <int kConsumers>
__device__ void sum_logits(const FewArgs& a, float* z, float* red, int tid) {
  const int n = a.N * a.E;
  int parts = 1;  // threads per logit
  while (parts < a.slices && parts * 2 * n <= kConsumers) parts *= 2;
  if (parts > 1) {
    const int l = tid % n, part = tid / n;
    if (part < parts)
      red[part * n + l] = sum_partials<8>(a.part_logits + l, n, part, parts, a.slices);
    bar_sync(kBarConsumers, kConsumers);
    if (tid < n) {
      float s = a.bias != nullptr ? a.bias[tid % a.E] : 0.0f;
      float sum = 0.0f;
#pragma unroll 8
      for (int q = 0; q < parts; ++q) sum += red[q * n + tid];
      z[tid] = sum + s;
    }
  } else {
    for (int l = tid; l < n; l += kConsumers) {
      const float s = sum_partials<16>(a.part_logits + l, n, 0, 1, a.slices);
      z[l] = s + (a.bias != nullptr ? a.bias[l % a.E] : 0.0f);
    }
  }
  bar_sync(kBarConsumers, kConsumers);
}

// Top-k and gates, one warp per token (the rules of select.cuh's plain top-k: descending fp32
// logits, the lower index first among equals, gates from exp(z - max)). The selection always
// yields k distinct experts, whatever the logits hold; a NaN, which that scan neither replaces nor
// takes for another value, ranks by its bits here (a positive one first).
template <int kWarps>
__device__ void select_all(const FewArgs& a, Tables& tb, const float* z, int warp, int lane) {
  for (int t = warp; t < a.N; t += kWarps) {
    const float* zt = z + t * a.E;
    const bool in0 = lane < a.E, in1 = lane + 32 < a.E;
    const float z0 = in0 ? zt[lane] : 0.0f, z1 = in1 ? zt[lane + 32] : 0.0f;
    // Images of the values, 0 for none: the largest by a warp reduction, its lowest lane by a
    // ballot (experts below 32 first).
    uint32_t k0 = in0 ? ordered(z0) : 0u, k1 = in1 ? ordered(z1) : 0u;
    float zmax = 0.0f, zsel = 0.0f;
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, k0 > k1 ? k0 : k1);
      const uint32_t b0 = __ballot_sync(0xFFFFFFFFu, k0 == best),
                     b1 = __ballot_sync(0xFFFFFFFFu, k1 == best);
      const int e = b0 != 0 ? __ffs(b0) - 1 : __ffs(b1) + 31;
      if (e == lane) k0 = 0u;
      if (e == lane + 32) k1 = 0u;
      const float v = zt[e];
      if (j == 0) zmax = v;
      if (lane == j) {
        mine = e;
        zsel = v;
      }
    }
    float all = (in0 ? expf(z0 - zmax) : 0.0f) + (in1 ? expf(z1 - zmax) : 0.0f);
    float sel = lane < a.k ? expf(zsel - zmax) : 0.0f;
    const float num = sel;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      sel += __shfl_xor_sync(0xFFFFFFFFu, sel, o);
    }
    if (lane < a.k) {
      tb.idx[t * a.k + lane] = static_cast<uint8_t>(mine);
      tb.order[a.token_major ? t * a.k + lane : lane * a.N + t] = static_cast<uint8_t>(mine);
      tb.gate[t * a.k + lane] = num / (a.renorm ? sel : all);
    }
    if (lane == 0) {
      tb.zmax[t] = zmax;
      tb.sum[t] = all;
    }
  }
}

// Loads, capacity positions, segment offsets, the experts with rows, and the rows' tokens and
// gates (walkthrough 1.3, 3.1, 3.2; MoE series 2.2).
template <int kConsumers, int kPieceRows>
__device__ void assign_rows(const FewArgs& a, Tables& tb, int tid, int warp, int lane) {
  const int R = a.N * a.k;
  const uint32_t below = (1u << lane) - 1u;
  for (int e = warp; e < a.E; e += kConsumers / 32) {
    int base = 0;
    for (int r0 = 0; r0 < R; r0 += 32) {
      const int r = r0 + lane;  // record in capacity order
      const bool hit = r < R && tb.order[r] == e;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, hit);
      if (hit) tb.pos_order[r] = static_cast<int16_t>(base + __popc(m & below));
      base += __popc(m);
    }
    if (lane == 0) tb.load[e] = base;
  }
  bar_sync(kBarConsumers, kConsumers);
  for (int r = tid; r < R; r += kConsumers) {
    const int t = r / a.k;
    tb.pos[r] = tb.pos_order[a.token_major ? r : (r - t * a.k) * a.N + t];
  }
  if (warp == 0) {
    int before = 0, parts = 0, tiles = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? static_cast<int>(min(static_cast<int64_t>(tb.load[e]), a.capacity))
                            : 0;
      // Inclusive prefix sums over the lanes: rows, pieces and row tiles (n <= 64 a lane).
      int sum = n | ((n + kPieceRows - 1) / kPieceRows) << 12 | ((n + 7) / 8) << 20;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int total = __shfl_sync(0xFFFFFFFFu, sum, 31);
      const int np = (n + kPieceRows - 1) / kPieceRows, nt = (n + 7) / 8;
      const int row = before + (sum & 0xFFF) - n;
      const int part = parts + ((sum >> 12) & 0xFF) - np;
      const int tile = tiles + (sum >> 20) - nt;
      if (e < a.E) tb.off[e] = row;
      for (int q = 0; q < np; ++q)
        tb.part[part + q] = {static_cast<int16_t>(e), static_cast<int16_t>(row + q * kPieceRows),
                             static_cast<int16_t>(min(kPieceRows, n - q * kPieceRows)),
                             static_cast<int16_t>(tile + q * (kPieceRows / 8))};
      const int most = __reduce_max_sync(0xFFFFFFFFu, n);
      if (lane == 0) tb.max_rows = e0 == 0 ? most : max(tb.max_rows, most);
      before += total & 0xFFF;
      parts += (total >> 12) & 0xFF;
      tiles += total >> 20;
    }
    if (lane == 0) {
      tb.off[a.E] = before;
      tb.n_parts = parts;
    }
  }
  bar_sync(kBarConsumers, kConsumers);
  for (int r = tid; r < R; r += kConsumers) {
    const int t = r / a.k;
    const int p = tb.pos[r];
    if (p < a.capacity) {
      float g = tb.gate[r];
      if (a.renorm_kept) {
        float kept = 0.0f;
        int slots = 0;
        for (int j = 0; j < a.k; ++j) {
          if (tb.pos[t * a.k + j] < a.capacity) {
            kept += tb.gate[t * a.k + j];
            ++slots;
          }
        }
        // (As the combine: kept gates that are all 0 share equally.)
        if (slots < a.k) g = kept == 0.0f ? 1.0f / static_cast<float>(slots) : g / kept;
      }
      const int row = tb.off[tb.idx[r]] + p;
      tb.row_tok[row] = static_cast<int16_t>(t);
      tb.row_gate[row] = g;
    }
  }
}

template <int kConsumers>
__device__ void export_routing(const FewArgs& a, const Tables& tb, const float* z, int tid) {
  const int R = a.N * a.k;
  for (int r = tid; r < R; r += kConsumers) {
    const int p = tb.pos[r];
    if (a.idx) a.idx[r] = tb.idx[r];
    if (a.gate) a.gate[r] = tb.gate[r];
    if (a.pos) a.pos[r] = p;
    if (a.dropped) a.dropped[r] = p >= a.capacity;
  }
  if (a.logits)
    for (int l = tid; l < a.N * a.E; l += kConsumers) a.logits[l] = z[l];
  if (tid < a.E) {
    if (a.load) a.load[tid] = tb.load[tid];
    if (a.colsum) {
      float s = 0.0f;
      for (int t = 0; t < a.N; ++t) s += expf(z[t * a.E + tid] - tb.zmax[t]) / tb.sum[t];
      a.colsum[tid] = s;
    }
  }
  if (a.offsets && tid <= a.E) a.offsets[tid] = tb.off[tid];
}

// ------------------------------------------------------------------ consumers

template <int WK>
struct Consumer {
  Ring ring;
  Cursor cur;
  RedTurn<WK> red;
  int tid, warp, lane;
  bool ok;
  uint64_t timeout_ns;
  int* err;

  __device__ void wait_full() {
    if (ok && (!mbar_wait(&ring.full[cur.stage], cur.phase, timeout_ns) ||
               !mbar_wait(&ring.rows_full[cur.stage], cur.phase, timeout_ns))) {
      ok = false;
      record_error(err, MOE_DEVERR_WAIT_TIMEOUT);
    }
    __syncwarp();  // the lanes leave the wait one by one; what follows is for whole warps
  }
  __device__ uint32_t my_box() const {
    return smem_u32(ring.weights) + static_cast<uint32_t>(cur.stage) * kStageBytes +
           static_cast<uint32_t>(box_of<WK>(warp)) * kBoxBytes;
  }
  __device__ const uint8_t* rows() const { return ring.rows + cur.stage * ring.row_bytes; }
  __device__ void release() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[cur.stage]);
    cur.next(ring.stages);
  }
};

// ---- up: stages [k0, k1) of one column tile of one piece

// Two H values of row r of a piece: columns f, f + 1 (f even).
template <int WK>
__device__ __forceinline__ void store_h(const FewArgs& a, const Part& pt, int r, int f, float h0,
                                        float h1) {
  if constexpr (WK == kF32) {
    if (f < a.F)
      *reinterpret_cast<float2*>(static_cast<float*>(a.H) + (pt.row0 + r) * h_row_f32(a.F) + f) =
          make_float2(h0, h1);
  } else {
    const int pair = (f & 31) >> 1, t = pair & 3, block = pair >> 2;
    uint32_t* w = reinterpret_cast<uint32_t*>(
                      static_cast<uint8_t*>(a.H) +
                      ((pt.tile + (r >> 3)) * h_groups(a.F) + (f >> 5)) * kHGroupBytes) +
                  ((r & 7) * 4 + t) * 4 + block;
    const uint32_t hi = pack_bf16x2(h0, h1);
    const float r0 = h0 - bf16_bits_to_float(hi & 0xFFFFu);
    const float r1 = h1 - bf16_bits_to_float(hi >> 16);
    // A value that is infinite, or becomes so in bf16, has no remainder.
    w[0] = hi;
    w[128] = pack_bf16x2(fabsf(r0) < INFINITY ? r0 : 0.0f, fabsf(r1) < INFINITY ? r1 : 0.0f);
  }
}

template <int WK>
__device__ __forceinline__ void finish_h(const FewArgs& a, const Tables& tb, const Part& pt, int r,
                                         int f, float2 h1, float2 h2) {
  if (r >= pt.n) return;
  float v0 = 0.0f, v1 = 0.0f;  // columns past F: zeros, which the down projection reads
  if (f < a.F) {
    if constexpr (WK == kW8) {
      const int64_t at = static_cast<int64_t>(pt.expert) * a.F + f;
      const float2 s1 = __ldg(reinterpret_cast<const float2*>(a.S1 + at));
      const float2 s2 = __ldg(reinterpret_cast<const float2*>(a.S2 + at));
      h1.x *= s1.x;
      h1.y *= s1.y;
      h2.x *= s2.x;
      h2.y *= s2.y;
    }
    const float g = tb.row_gate[pt.row0 + r];
    v0 = act_value(a.act, h1.x) * h2.x * g;
    v1 = act_value(a.act, h1.y) * h2.y * g;
  }
  store_h<WK>(a, pt, r, f, v0, v1);
}

// 16- and 8-bit weights: a warp owns 16 columns of the tile, both matrices and all of k, so its
// sums are final in its registers: it makes H, or writes its share, without the other warps, and
// goes on with the next tile while they still multiply. (With the matrices and k cut over the
// warps, whose sums met in shared memory eight rows at a time, the 8-bit Mixtral-shaped layer took
// 231 us for 8 tokens and 332 for 32, against 224 and 315; bf16 the same.)
//   v[matrix][j][c]: row 8 j + 2 t + (c & 1), lane = 4 g + t; column g + 8 (c >> 1) of the 16
//   (bf16) or 2 g + (c >> 1) (8-bit).
template <int NT>
struct UpSums {
  float v[2][NT][4];
};

// acc += a stage (64 k) of both matrices.
template <int WK, int NT>
__device__ __forceinline__ void up_stage(UpSums<NT>& acc, Consumer<WK>& c, int k0, int D) {
  const uint32_t stage =
      smem_u32(c.ring.weights) + static_cast<uint32_t>(c.cur.stage) * kStageBytes;
  constexpr int kSideWarps = Team<WK>::kWarps / 2;
  const uint32_t side = static_cast<uint32_t>(c.warp / kSideWarps);
  const int at = c.warp % kSideWarps;  // which 16 columns of the box
  Frag<NT, false> f[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    f[q].load_rows(c.rows(), kRowPitch, q, k0 + q * 32, D, c.lane);
  constexpr int kLoads = WK == kBF16 ? 4 : 2;  // of a matrix: 16 or 32 k each
  uint32_t w[2][kLoads][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t r = static_cast<uint32_t>(
          WK == kBF16 ? 16 * i + (c.lane >> 4) * 8 + (c.lane & 7) : 32 * i + c.lane);
      const uint32_t chunk =
          static_cast<uint32_t>(WK == kBF16 ? at * 2 + ((c.lane >> 3) & 1) : at);
      ldsm_x4_trans(stage + (static_cast<uint32_t>(m) * 2 + side) * kBoxBytes + r * 128 +
                        ((chunk ^ (r & 7u)) << 4),
                    w[m][i]);
    }
  c.release();
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int b = 0; b < 2; ++b)  // 16 k each
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t x[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (WK == kBF16) {
            x[2 * h] = w[m][2 * q + b][2 * h];
            x[2 * h + 1] = w[m][2 * q + b][2 * h + 1];
          } else {
            i8x4_to_bf16(w[m][q][2 * b + h], x[2 * h], x[2 * h + 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mma_bf16(acc.v[m][j], x, f[q].r[j][0][2 * b], f[q].r[j][0][2 * b + 1]);
      }
}

// H of the warp's columns (from f0 on) of the piece's rows.
template <int WK, int NT>
__device__ __forceinline__ void finish_strip(const FewArgs& a, const Tables& tb, const Part& pt,
                                             const UpSums<NT>& s, int f0, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (8 * j >= pt.n) break;
    if constexpr (WK == kW8) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        finish_h<WK>(a, tb, pt, 8 * j + 2 * t + r, f0 + 2 * g,
                     make_float2(s.v[0][j][r], s.v[0][j][2 + r]),
                     make_float2(s.v[1][j][r], s.v[1][j][2 + r]));
    } else {
      // Two columns of a row to one lane: of lanes g and g + 1 (g even) the first takes row 2 t,
      // the second row 2 t + 1.
      const bool odd = (g & 1) != 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 v[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float mine = odd ? s.v[m][j][2 * h + 1] : s.v[m][j][2 * h];
          const float other = __shfl_xor_sync(
              0xFFFFFFFFu, odd ? s.v[m][j][2 * h] : s.v[m][j][2 * h + 1], 4);
          v[m] = odd ? make_float2(other, mine) : make_float2(mine, other);
        }
        finish_h<WK>(a, tb, pt, 8 * j + 2 * t + (odd ? 1 : 0), f0 + 8 * h + (g & ~1), v[0], v[1]);
      }
    }
  }
}

template <int WK, int NT>
__device__ __forceinline__ void up_strip(const FewArgs& a, Tables& tb, Consumer<WK>& c,
                                         const SplitK& sp, long long tile, int steps, int k0,
                                         int k1, const Part pt, int fb) {
  constexpr int kConsumers = Team<WK>::kConsumers;
  UpSums<NT> acc;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc.v[m][j][q] = 0.0f;
  for (int s = k0; s < k1; ++s) {
    c.wait_full();
    up_stage<WK, NT>(acc, c, s * kBoxRows, a.D);
  }
  const int f0 = fb * Shape<WK>::kCols + c.warp * 16;
  if (k0 > 0 || k1 < steps) {
    const int first = sp.owner(tile * steps), last = sp.owner(tile * steps + steps - 1);
    auto share = [&](int b, bool head) {
      return reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(b) * 2 + (head ? 1 : 0)) *
                                                    a.part_floats) + c.tid;
    };
    float4* mine = share(static_cast<int>(blockIdx.x), k0 == 0);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        mine[(2 * j + m) * kConsumers] =
            make_float4(acc.v[m][j][0], acc.v[m][j][1], acc.v[m][j][2], acc.v[m][j][3]);
    if (!last_warp_to_arrive(a.counters + first * kMaxWarps + c.warp, last - first + 1, c.lane))
      return;
    // The last to arrive adds the shares up in block order, two blocks' loads at a time.
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float4 sum[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      for (int b0 = first; b0 <= last; b0 += 2) {
        float4 w[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            w[u][m] = b0 + u <= last
                          ? __ldcg(share(b0 + u, b0 + u == first) + (2 * j + m) * kConsumers)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sum[m].x += w[u][m].x;
            sum[m].y += w[u][m].y;
            sum[m].z += w[u][m].z;
            sum[m].w += w[u][m].w;
          }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        acc.v[m][j][0] = sum[m].x;
        acc.v[m][j][1] = sum[m].y;
        acc.v[m][j][2] = sum[m].z;
        acc.v[m][j][3] = sum[m].w;
      }
    }
  }
  finish_strip<WK, NT>(a, tb, pt, acc, f0, c.lane);
}

// fp32 weights: the warps' sums meet in shared memory.
template <int WK, int NT>
__device__ __forceinline__ void up_tile(const FewArgs& a, Tables& tb, Consumer<WK>& c,
                                        const SplitK& sp, long long tile, int steps, int k0,
                                        int k1, const Part pt, int fb) {
  using S = Shape<WK>;
  using P = Places<WK>;
  constexpr int kConsumers = Team<WK>::kConsumers;
  Acc<WK, NT> acc;
  acc.zero();
  const int first_row = warp_row<WK>(c.warp);
  for (int s = k0; s < k1; ++s) {
    c.wait_full();
    const int d0 = s * kBoxRows + first_row;
    multiply_f32<NT>(acc, c.my_box(), c.warp, c.lane, smem_u32(c.rows()) + first_row * 4,
                     kRowPitchF32, pt.n, d0, a.D);
    c.release();
  }

  // Both branches' sums over the block's stages; the whole tile's, or a share of it.
  const bool whole = k0 == 0 && k1 == steps;
  float2* mine = reinterpret_cast<float2*>(
      a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (k0 > 0 ? 0 : 1)) * a.part_floats);
  for (int j = 0; j < NT && 8 * j < pt.n; ++j) {
    float* red = c.red.next();
    put_tile<WK, NT>(red, acc, j, c.warp, c.lane);
    bar_sync(kBarConsumers, kConsumers);
    for (int i = c.tid; i < P::kCount; i += kConsumers) {
      const float2 h1 = take_pair<WK>(red, 0, P::row(i), P::col(i));
      const float2 h2 = take_pair<WK>(red, 1, P::row(i), P::col(i));
      if (whole) {
        finish_h<WK>(a, tb, pt, 8 * j + P::row(i), fb * S::kCols + P::col(i), h1, h2);
      } else {
        mine[(2 * j) * P::kCount + i] = h1;
        mine[(2 * j + 1) * P::kCount + i] = h2;
      }
    }
    c.red.done();
  }
  if (whole) return;
  const int first = sp.owner(tile * steps), last = sp.owner(tile * steps + steps - 1);
  if (!last_to_finish<kConsumers>(a.counters + first * kMaxWarps, last - first + 1, c.tid,
                                  &tb.flag))
    return;
  for (int j = 0; j < NT && 8 * j < pt.n; ++j) {
    float2 h[2][P::kMine];
#pragma unroll
    for (int branch = 0; branch < 2; ++branch) {
#pragma unroll
      for (int q = 0; q < P::kMine; ++q) h[branch][q] = make_float2(0.0f, 0.0f);
      const int at = (2 * j + branch) * P::kCount;
      add_shares<kConsumers>(h[branch], a.part, a.part_floats, first, last, at + c.tid,
                             at + P::kCount);
    }
#pragma unroll
    for (int q = 0; q < P::kMine; ++q) {
      const int i = c.tid + q * kConsumers;
      if (i < P::kCount)
        finish_h<WK>(a, tb, pt, 8 * j + P::row(i), fb * S::kCols + P::col(i), h[0][q], h[1][q]);
    }
  }
}

// ---- down: stages [s0, s1) of one piece's part of one column block, added into outacc

template <int WK, int NT>
__device__ __forceinline__ void down_run(const FewArgs& a, Tables& tb, Consumer<WK>& c, int s0,
                                         int s1, const Part pt, int cb, float* outacc) {
  using S = Shape<WK>;
  using P = Places<WK>;
  constexpr int kConsumers = Team<WK>::kConsumers;
  Acc<WK, NT> acc;
  acc.zero();
  // The first two boxes hold the stage's first 64 k-rows, the others the next.
  const int first_row = (box_of<WK>(c.warp) >> 1) * kBoxRows + warp_row<WK>(c.warp);
  for (int s = s0; s < s1; ++s) {
    c.wait_full();
    if constexpr (WK == kF32) {
      multiply_f32<NT>(acc, c.my_box(), c.warp, c.lane, smem_u32(c.rows()) + first_row * 4,
                       2 * kBoxRows * 4, pt.n, s * 2 * kBoxRows + first_row, a.F);
      c.release();
    } else {
      Weights<WK> w;
      Frag<NT, true> f;
      w.load(c.my_box(), c.warp, c.lane);
      f.load_ordered(c.rows(), first_row / 32, c.lane);
      c.release();
      multiply<WK, NT, true>(acc, w, f);
    }
  }
  for (int j = 0; j < NT && 8 * j < pt.n; ++j) {
    float* red = c.red.next();
    put_tile<WK, NT>(red, acc, j, c.warp, c.lane);
    bar_sync(kBarConsumers, kConsumers);
    for (int i = c.tid; i < P::kCount; i += kConsumers) {
      const int r = 8 * j + P::row(i);
      if (r >= pt.n) continue;
      float2 v = take_pair<WK>(red, -1, P::row(i), P::col(i));
      if constexpr (WK == kW8) {
        const int d = cb * S::kCols + P::col(i);
        if (d < a.D) {
          const float2 s = __ldg(reinterpret_cast<const float2*>(
              a.S3 + static_cast<int64_t>(pt.expert) * a.D + d));
          v.x *= s.x;
          v.y *= s.y;
        }
      }
      float2* o = reinterpret_cast<float2*>(
          outacc + static_cast<int>(tb.row_tok[pt.row0 + r]) * S::kCols + P::col(i));
      o->x += v.x;
      o->y += v.y;
    }
    c.red.done();
  }
}

template <int WK>
__device__ __forceinline__ void store_out(const FewArgs& a, int t, int d, float2 v) {
  if (d >= a.D) return;
  const int64_t at = static_cast<int64_t>(t) * a.D + d;
  if constexpr (WK == kF32)
    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = v;
  else
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at) = pack_bf16x2(v.x, v.y);
}

// CALL(row tiles) for n rows, where a piece has at most MAXNT row tiles.
#define MOE_FEW_ROWS(n, CALL)                             \
  do {                                                    \
    if (MAXNT == 1 || (n) <= 8) { CALL(1); }              \
    else if (MAXNT == 2 || (n) <= 16) { CALL((MAXNT < 2 ? 1 : 2)); }  \
    else if ((n) <= 24) { CALL((MAXNT < 4 ? 1 : 3)); }    \
    else { CALL((MAXNT < 4 ? 1 : 4)); }                   \
  } while (0)

// ------------------------------------------------------------------ the kernel

// MAXNT: row tiles of the largest possible piece (the tokens of a batch bound an expert's rows).
// A kernel that holds only what its batch can need keeps its loops out of local memory (8-bit, two
// row tiles: 40 bytes of a thread spilled, 208 loaded back over the kernel's code): a spill costs
// an L2 access here, since the ring leaves the L1 cache almost nothing.
template <int WK, int MAXNT>
__global__ void __launch_bounds__(Team<WK>::kThreads, 1)
few_kernel(const __grid_constant__ CUtensorMap m1, const __grid_constant__ CUtensorMap m2,
           const __grid_constant__ CUtensorMap m3, const __grid_constant__ FewArgs a) {
  using S = Shape<WK>;
  using P = Places<WK>;
  constexpr int kConsumers = Team<WK>::kConsumers;
  using T = Team<WK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const size_t ring_size = ring_bytes<WK>(a.N, a.E);
  float* red = reinterpret_cast<float*>(smem + ring_size);
  float* outacc = red + kRedBytes / sizeof(float);  // first logits, then the column block's sums
  Tables& tb = *reinterpret_cast<Tables*>(reinterpret_cast<uint8_t*>(outacc) +
                                          out_bytes<WK>(a.N, a.E));
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int G = static_cast<int>(gridDim.x);

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&tb.full[i], 1);
      mbar_init(&tb.rows_full[i], 32);  // the row producer's lanes
      mbar_init(&tb.empty[i], T::kWarps);
    }
    fence_barrier_init();
    // Arrivals at this block's shared tiles; seen by the others after the first grid barrier.
    for (int i = 0; i < kMaxWarps; ++i) a.counters[blockIdx.x * kMaxWarps + i] = 0;
    a.counters[kMaxGrid * kMaxWarps + blockIdx.x] = 0;
  }
  __syncthreads();

  bool ok = true;
  if (warp < T::kWarps) {
    partial_logits<WK>(a, red, tid);
    ok = grid_barrier<kConsumers>(a.bar, G, tid, &tb.flag, a.timeout_ns, a.err);
    sum_logits<kConsumers>(a, outacc, red, tid);
    select_all<T::kWarps>(a, tb, outacc, warp, lane);
    bar_sync(kBarConsumers, kConsumers);
    assign_rows<kConsumers, S::kPieceRows>(a, tb, tid, warp, lane);
  }
  bar_sync(kBarAll, T::kThreads);

  const int up_steps = (a.D + kBoxRows - 1) / kBoxRows;
  const int up_cols = (a.F + S::kCols - 1) / S::kCols;
  const int run_steps = (a.F + 2 * kBoxRows - 1) / (2 * kBoxRows);
  const int down_cols = (a.D + S::kCols - 1) / S::kCols;
  const int parts = tb.n_parts;
  const int down_steps = parts * run_steps;
  const SplitK up(static_cast<long long>(parts) * up_cols, up_steps, G);
  const SplitK down(parts > 0 ? down_cols : 0, down_steps, G);
  const int me = static_cast<int>(blockIdx.x);
  const long long u0 = me < up.grid ? up.start(me) : 0, u1 = me < up.grid ? up.start(me + 1) : 0;
  const long long d0 = me < down.grid ? down.start(me) : 0,
                  d1 = me < down.grid ? down.start(me + 1) : 0;

  const int row_tiles = max(1, min(S::kPieceRows, tb.max_rows) + 7) / 8;
  Ring ring;
  ring.stages = ring_stages(ring_size, row_tiles);
  ring.row_bytes = row_tiles * kTileBytes;
  ring.weights = smem;
  ring.rows = smem + static_cast<size_t>(ring.stages) * kStageBytes;
  ring.full = tb.full;
  ring.rows_full = tb.rows_full;
  ring.empty = tb.empty;

  // Stages in order: f_up(piece, column tile, k-stage), then f_down(piece, column block, k-stage);
  // a callback that returns false ends the walk.
  auto walk = [&](auto f_up, auto between, auto f_down) {
    for (long long s = u0; s < u1;) {
      const long long tile = s / up_steps;
      int k = static_cast<int>(s - tile * up_steps);
      const int k_end = static_cast<int>(min(static_cast<long long>(up_steps), k + (u1 - s)));
      const Part pt = tb.part[tile / up_cols];
      const int fb = static_cast<int>(tile % up_cols);
      s += k_end - k;
      for (; k < k_end; ++k)
        if (!f_up(pt, fb, k)) return;
    }
    between();
    for (long long s = d0; s < d1;) {
      const long long tile = s / down_steps;
      const int in = static_cast<int>(s - tile * down_steps);
      const int pi = in / run_steps;
      int k = in - pi * run_steps;
      const int k_end = static_cast<int>(min(static_cast<long long>(run_steps), k + (d1 - s)));
      const Part pt = tb.part[pi];
      s += k_end - k;
      for (; k < k_end; ++k)
        if (!f_down(pt, static_cast<int>(tile), k)) return;
    }
  };

  if (warp >= T::kWarps) {
    give_registers<T::kProducerRegs>();
    if (warp == T::kWeightWarp) {
      // Weight producer: one thread issues this block's stages of both products in order.
      if (lane == 0) {
        // Weights are read once; evict_first read 6.4 TB/s where the default read 6.0.
        const uint64_t policy = l2_policy(-1);
        Cursor c;
        bool good = true;
        long long issued = 0;
        auto up_stage = [&](const Part& pt, int fb, int k) {
          if (!(good = acquire_weights(ring, c, issued, a.timeout_ns))) return false;
          uint8_t* dst = smem + static_cast<size_t>(c.stage) * kStageBytes;
          uint64_t* bar = &tb.full[c.stage];
          const int col = fb * S::kCols, row = k * kBoxRows, e = pt.expert;
          tma_load_3d_hint(dst, &m1, bar, col, row, e, policy);
          tma_load_3d_hint(dst + kBoxBytes, &m1, bar, col + S::kBoxCols, row, e, policy);
          tma_load_3d_hint(dst + 2 * kBoxBytes, &m2, bar, col, row, e, policy);
          tma_load_3d_hint(dst + 3 * kBoxBytes, &m2, bar, col + S::kBoxCols, row, e, policy);
          c.next(ring.stages);
          ++issued;
          return true;
        };
        auto down_stage = [&](const Part& pt, int cb, int k) {
          if (!(good = acquire_weights(ring, c, issued, a.timeout_ns))) return false;
          uint8_t* dst = smem + static_cast<size_t>(c.stage) * kStageBytes;
          uint64_t* bar = &tb.full[c.stage];
          const int col = cb * S::kCols, row = 2 * k * kBoxRows, e = pt.expert;
          tma_load_3d_hint(dst, &m3, bar, col, row, e, policy);
          tma_load_3d_hint(dst + kBoxBytes, &m3, bar, col + S::kBoxCols, row, e, policy);
          tma_load_3d_hint(dst + 2 * kBoxBytes, &m3, bar, col, row + kBoxRows, e, policy);
          tma_load_3d_hint(dst + 3 * kBoxBytes, &m3, bar, col + S::kBoxCols, row + kBoxRows, e,
                           policy);
          c.next(ring.stages);
          ++issued;
          return true;
        };
        walk(up_stage, [] {}, down_stage);
        if (!good) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
        drain(tb.full, ring.stages, c, issued, a.timeout_ns);
      }
      __syncwarp();
    } else if (warp == T::kRowWarp) {
      // Row producer: the kept tokens' rows of X, 16 bytes per lane and copy; then tiles of H,
      // one bulk copy each, after the barrier that completes H.
      Cursor c;
      bool good = true;
      long long issued = 0;
      auto acquire = [&] {  // all lanes: the stage is free
        good = mbar_wait(&tb.empty[c.stage], c.phase ^ 1u, a.timeout_ns);
        good = __all_sync(0xFFFFFFFFu, good);
        return good;
      };
      auto up_rows = [&](const Part& pt, int, int k) {
        constexpr int kEl = WK == kF32 ? 4 : 2;
        constexpr int kPieces = kBoxRows * kEl / 16;  // of a row
        constexpr int kPitch = WK == kF32 ? kRowPitchF32 : kRowPitch;
        if (!acquire()) return false;
        const int d = k * kBoxRows + lane % kPieces * (16 / kEl);
        if (d < a.D) {
          uint8_t* dst = ring.rows + c.stage * ring.row_bytes + lane % kPieces * 16;
          for (int r = lane / kPieces; r < pt.n; r += 32 / kPieces)
            cp_async16(dst + r * kPitch,
                       static_cast<const uint8_t*>(a.X) +
                           (static_cast<int64_t>(tb.row_tok[pt.row0 + r]) * a.D + d) * kEl);
        }
        cp_async_arrive(&tb.rows_full[c.stage]);
        c.next(ring.stages);
        ++issued;
        return true;
      };
      auto h_ready = [&] {
        bar_sync(kBarRows, kConsumers + 32);
        fence_proxy_async_all();
      };
      auto down_rows = [&](const Part& pt, int, int k) {
        if (!acquire()) return false;
        uint8_t* dst = ring.rows + c.stage * ring.row_bytes;
        uint64_t* bar = &tb.rows_full[c.stage];
        if constexpr (WK == kF32) {
          constexpr int kPieces = 2 * kBoxRows * 4 / 16;  // 32: a row per copy
          const int f = k * 2 * kBoxRows + lane * 4;
          if (f < a.F)
            for (int r = 0; r < pt.n; ++r)
              cp_async16(dst + r * (kPieces * 16) + lane * 16,
                         static_cast<const float*>(a.H) + (pt.row0 + r) * h_row_f32(a.F) + f);
          cp_async_arrive(bar);
        } else {
          const int tiles = (pt.n + 7) / 8;
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(tiles) * kTileBytes);
          else mbar_arrive(bar);
          __syncwarp();
          if (lane < tiles)
            bulk_g2s(dst + lane * kTileBytes,
                     static_cast<const uint8_t*>(a.H) +
                         ((pt.tile + lane) * h_groups(a.F) + k * 4) * kHGroupBytes,
                     kTileBytes, bar);
        }
        c.next(ring.stages);
        ++issued;
        return true;
      };
      bool waited = false;
      walk(up_rows, [&] { h_ready(); waited = true; }, down_rows);
      if (!waited) h_ready();  // the consumers arrive there in any case
      if (!good && lane == 0) record_error(a.err, MOE_DEVERR_WAIT_TIMEOUT);
      drain(tb.rows_full, ring.stages, c, issued, a.timeout_ns);
      __syncwarp();
    }
  } else {
    take_registers<T::kConsumerRegs>();
    if (me == 0) export_routing<kConsumers>(a, tb, outacc, tid);
    if (parts == 0) {  // a capacity of zero keeps nothing: zeros
      for (int cb = me; cb < down_cols; cb += G)
        for (int i = tid; i < a.N * P::kPairs; i += kConsumers)
          store_out<WK>(a, P::row(i), cb * S::kCols + P::col(i), make_float2(0.0f, 0.0f));
    }
    Consumer<WK> c{ring, Cursor{}, RedTurn<WK>{red}, tid, warp, lane, ok, a.timeout_ns, a.err};
    for (long long s = u0; s < u1;) {
      const long long tile = s / up_steps;
      const int k0 = static_cast<int>(s - tile * up_steps);
      const int k1 = static_cast<int>(min(static_cast<long long>(up_steps), k0 + (u1 - s)));
      const Part pt = tb.part[tile / up_cols];
      const int fb = static_cast<int>(tile % up_cols);
#define MOE_UP(NT)                                                        \
  if constexpr (WK == kF32)                                               \
    up_tile<WK, NT>(a, tb, c, up, tile, up_steps, k0, k1, pt, fb);        \
  else                                                                    \
    up_strip<WK, NT>(a, tb, c, up, tile, up_steps, k0, k1, pt, fb)
      MOE_FEW_ROWS(pt.n, MOE_UP);
#undef MOE_UP
      s += k1 - k0;
    }
    fence_proxy_async_all();  // H is read by bulk copies
    if (!grid_barrier<kConsumers>(a.bar, 2 * G, tid, &tb.flag, a.timeout_ns, a.err)) c.ok = false;
    bar_arrive(kBarRows, kConsumers + 32);

    for (long long s = d0; s < d1;) {
      const long long tile = s / down_steps;
      const int k0 = static_cast<int>(s - tile * down_steps);
      const int k1 = static_cast<int>(min(static_cast<long long>(down_steps), k0 + (d1 - s)));
      const int cb = static_cast<int>(tile);
      for (int i = tid; i < a.N * S::kCols; i += kConsumers) outacc[i] = 0.0f;
      bar_sync(kBarConsumers, kConsumers);
      for (int k = k0; k < k1;) {
        const int pi = k / run_steps;
        const int s0 = k - pi * run_steps;
        const int s1 = min(run_steps, s0 + (k1 - k));
        const Part pt = tb.part[pi];
#define MOE_DOWN(NT) down_run<WK, NT>(a, tb, c, s0, s1, pt, cb, outacc)
        MOE_FEW_ROWS(pt.n, MOE_DOWN);
#undef MOE_DOWN
        k += s1 - s0;
      }
      bar_sync(kBarConsumers, kConsumers);  // the last sums are in
      const bool whole = k0 == 0 && k1 == down_steps;
      float2* mine = reinterpret_cast<float2*>(
          a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (k0 > 0 ? 0 : 1)) * a.part_floats);
      for (int i = tid; i < a.N * P::kPairs; i += kConsumers) {
        const float2 v = *reinterpret_cast<const float2*>(outacc + 2 * i);
        if (whole) store_out<WK>(a, P::row(i), cb * S::kCols + P::col(i), v);
        else mine[i] = v;
      }
      if (!whole) {
        const int first = down.owner(tile * down_steps),
                  last = down.owner(tile * down_steps + down_steps - 1);
        if (last_to_finish<kConsumers>(a.counters + kMaxGrid * kMaxWarps + first, last - first + 1,
                                       tid, &tb.flag)) {
          constexpr int kChunk = WK == kW8 ? 4 : 8;
          for (int i0 = tid; i0 < a.N * P::kPairs; i0 += kChunk * kConsumers) {
            float2 v[kChunk];
#pragma unroll
            for (int q = 0; q < kChunk; ++q) v[q] = make_float2(0.0f, 0.0f);
            add_shares<kConsumers>(v, a.part, a.part_floats, first, last, i0, a.N * P::kPairs);
#pragma unroll
            for (int q = 0; q < kChunk; ++q) {
              const int i = i0 + q * kConsumers;
              if (i < a.N * P::kPairs)
                store_out<WK>(a, P::row(i), cb * S::kCols + P::col(i), v[q]);
            }
          }
        }
      }
      bar_sync(kBarConsumers, kConsumers);
      s += k1 - k0;
    }
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

// Floats of a block's share of one tile: two matrices of up to four row tiles, or all tokens.
int64_t part_floats_of(int kind, int64_t N) {
  const int64_t cols = kind == kF32 ? Shape<kF32>::kCols
                       : kind == kBF16 ? Shape<kBF16>::kCols : Shape<kW8>::kCols;
  return cols * std::max<int64_t>(N, 16 * std::min<int64_t>(4, (N + 7) / 8));
}

template <int WK, int MAXNT>
cudaError_t launch(const moe_problem& p, const FewArgs& a, const void* W1, const void* W2,
                   const void* W3, cudaStream_t stream) {
  CUtensorMap m1, m2, m3;
  if (!make_stream_map(&m1, W1, WK, p.F, p.D, p.E) ||
      !make_stream_map(&m2, W2, WK, p.F, p.D, p.E) ||
      !make_stream_map(&m3, W3, WK, p.D, p.F, p.E))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(
      few_kernel<WK, MAXNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(num_sms(), kMaxGrid)));
  cfg.blockDim = dim3(Team<WK>::kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, few_kernel<WK, MAXNT>, m1, m2, m3, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int WK>
cudaError_t launch_kind(const moe_problem& p, const FewArgs& a, const FewTensors& t,
                        cudaStream_t stream) {
  if (p.N <= 8) return launch<WK, 1>(p, a, t.W1, t.W2, t.W3, stream);
  if (p.N <= 16 || Shape<WK>::kPieceRows == 16)
    return launch<WK, 2>(p, a, t.W1, t.W2, t.W3, stream);
  return launch<WK, Shape<WK>::kPieceRows / 8>(p, a, t.W1, t.W2, t.W3, stream);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

}  // namespace

bool make_stream_map(CUtensorMap* m, const void* ptr, int kind, uint64_t cols, uint64_t rows,
                     uint64_t count, uint32_t box_rows) {
  if (encode_fn() == nullptr) return false;
  const uint64_t el = kind == kF32 ? 4 : kind == kBF16 ? 2 : 1;
  const cuuint64_t dims[3] = {cols, rows, count};
  const cuuint64_t strides[2] = {cols * el, cols * rows * el};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / el), box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = kind == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : kind == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return encode_fn()(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_box_map_3d_bf16(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows,
                          uint64_t count, uint32_t box_cols, uint32_t box_rows) {
  if (encode_fn() == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, count};
  const cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_cols == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                     : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                      : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace of moe_forward_few: partial logits, counters, shared-tile sums, H.
size_t few_workspace_bytes(const moe_problem& p) {
  if (p.N < 1) return 0;
  const int64_t N = std::min<int64_t>(p.N, kMaxRows);
  auto up256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const int64_t R = N * p.k;
  // bf16 problems may come with either weight kind: the larger of the two.
  const int kind = p.dtype == MOE_DTYPE_F32 ? kF32 : kW8;
  return up256(sizeof(float) * kMaxSlices * N * p.E) + up256(sizeof(int) * kCounters) +
         up256(sizeof(float) * 2 * kMaxGrid * part_floats_of(kind, N)) +
         up256(kind == kF32 ? sizeof(float) * R * h_row_f32(p.F)
                            : static_cast<size_t>((std::min<int64_t>(p.E, R) + R / 8) *
                                                  h_groups(p.F) * kHGroupBytes));
}

cudaError_t launch_few(const moe_problem& p, int64_t capacity, const FewTensors& t, void* scratch,
                       int* err, int* bar, uint64_t timeout_ns, cudaStream_t stream) {
  FewArgs a{};
  a.X = t.X;
  a.W_r = t.W_r;
  a.bias = t.bias;
  a.S1 = t.S1;
  a.S2 = t.S2;
  a.S3 = t.S3;
  a.out = t.out;
  a.logits = t.logits;
  a.idx = t.idx;
  a.gate = t.gate;
  a.load = t.load;
  a.offsets = t.offsets;
  a.pos = t.pos;
  a.dropped = t.dropped;
  a.colsum = t.colsum;
  auto up256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  uint8_t* w = static_cast<uint8_t*>(scratch);
  a.part_logits = reinterpret_cast<float*>(w);
  w += up256(sizeof(float) * kMaxSlices * p.N * p.E);
  a.counters = reinterpret_cast<int*>(w);
  w += up256(sizeof(int) * kCounters);
  a.part = reinterpret_cast<float*>(w);
  a.part_floats = part_floats_of(p.dtype == MOE_DTYPE_F32 ? kF32 : kW8, p.N);
  w += up256(sizeof(float) * 2 * kMaxGrid * a.part_floats);
  a.H = w;
  a.bar = bar;
  a.err = err;
  a.capacity = capacity;
  a.timeout_ns = timeout_ns;
  a.N = static_cast<int>(p.N);
  a.D = static_cast<int>(p.D);
  a.F = static_cast<int>(p.F);
  a.E = p.E;
  a.k = p.k;
  // Router split: few tokens share nothing but W_r, so each token's D goes over many blocks;
  // with more tokens a block takes up to 8 of them, which bounds the partial logits that every
  // block reads back.
  a.tokens_per_group = p.N <= 8 ? 1 : p.N <= 32 ? 4 : 8;
  const int groups = (a.N + a.tokens_per_group - 1) / a.tokens_per_group;
  const int grid = std::min(num_sms(), kMaxGrid);
  a.slices = std::max(1, std::min({grid / groups, kMaxSlices, (a.D + 31) / 32}));
  a.renorm = p.renormalize != 0;
  a.token_major = p.capacity_order == MOE_ORDER_TOKEN_MAJOR;
  a.renorm_kept = p.drop_policy == MOE_DROP_RENORM_KEPT;
  a.act = p.activation;
  if (t.S1 != nullptr) return launch_kind<kW8>(p, a, t, stream);
  if (p.dtype == MOE_DTYPE_F32) return launch_kind<kF32>(p, a, t, stream);
  return launch_kind<kBF16>(p, a, t, stream);
}

}  // namespace moe
