// Attention of many new tokens over a paged KV cache on the tcgen05 tensor cores: prompts, chunks of
// prompts, and batches that mix them with decode steps.
//
//   o = softmax(q K^T / sqrt(d)) V over slots 0 .. L - n + i of the query's row,  lse = ln sum e^s.
//
// Query rows. The g query heads of a key/value head are rows of one tile: row i g + j is new token i
// under head j, floor(128 / g) tokens fill a 128-row tile, and K and V are read once for the group. A
// work item is (row of the batch, key/value head, one or two tiles, a range of the cached tokens).
//
// One launch, persistent, one CTA an SM. Each CTA works out the list of items from the rows' lengths (the longest
// first within a row, cut along the cached tokens where whole tiles would leave SMs idle) and takes items off it
// by an atomic counter (which item runs where does not change any sum). When the list is empty, the CTAs wait for
// the pieces of what was cut, and join them in their order.
//
// One CTA: two softmax warpgroups, two loader warps and an MMA warp.
//   * The loaders bring 128 cached tokens at a time by TMA into a ring of K and V tiles (128-byte
//     swizzle): boxes of the tokens of a page, at the slots that the page table gives, and around the
//     row's length rows gathered four a copy. Tokens past the length are rows outside the tensor map:
//     they arrive as zeros, so pages of any size may end anywhere and what lies behind the length is
//     never read.
//   * The MMA warp issues S = Q K^T (both operands in shared memory) and O += P V (P in tensor
//     memory, V as stored, along the head dimension), alternating between two units, so that one
//     unit's products run while the other's softmax does.
//   * A unit is a warpgroup with a 128-row S and O accumulator in tensor memory; a thread owns a query
//     row. P overwrites S in place. The running maximum is only raised when a score exceeds it by more
//     than 2^8, so that the output in tensor memory is rarely rescaled; p then stays below 2^8 (fp16, whose
//     weights are lifted: 2^15), and the sum and the output share the same factor.
//   With two tiles the units are the tiles, over the same K and V; with one, the units take the cached
//   tiles in turn (even, odd) and are joined through shared memory at the end.
//
// Sums, maxima, S and O are fp32; the weights p are rounded to the cache's type, as the product takes
// them; l is the sum of the unrounded p.
//
// Bound: the round of a unit, S to weights to its products, of which two in turn keep the tensor cores 61% busy at
// 1.9 GHz (exponentials 36%, issue 42%); in long calls the clock falls besides, with the power limit.
// Measured on a GB300 with states in turn, 32 / 8 heads of 128, bf16: 2048 new tokens at 65536 1500 to 1530 us (1410 to
// 1440 TFLOP/s); a chunk of 512 among 15 sequences that decode, at 16384, 209 us; up to five drafted tokens of eight
// ragged sequences up to 16384 82 us, 4800 GB/s. Four prompts of 4096, 32 / 32 heads, fp16: 440 us (1250). Where one
// state's calls follow each other in a graph, the first take 1470 us (1470 TFLOP/s) and the last 399 (1380). At d = 64 the
// products halve and the softmax does not: 1024 new tokens of two sequences at 16384 319 us, 835 TFLOP/s.
//
// Every wait is bounded; one that gives up records PALU_ERR_TIMEOUT, and all roles wait for their own
// copies and products in flight before tensor memory is freed.
#include "kv.h"
#include "internal.h"
#include "kv_tc_ptx.cuh"

namespace palu {
namespace {

constexpr int kTile = 128;               // query rows of a tile, cached tokens of a step
constexpr int kThreads = 384;            // two softmax warpgroups; two loader warps, MMA and an idle warp
constexpr int kWhole = kKvTcWhole;       // tiles of so few steps are not cut: the join would cost more
// Registers: launched with 168 a thread (65536 / 384, in eights); 2 * 128 * 200 + 128 * 104 = 384 * 168.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
// log2 by which a score may exceed the running maximum before that is raised, and by which fp16 weights are lifted
// (softmax_base): together 15, the range of the type. An fp16 weight's rounding is then at most 2^-32 of the row's
// largest. Raised from 4 on, with a lift of 11, four prompts of 4096 took 481 us against 441; from 6 on, 453.
constexpr float kRaise = 8.f, kLift = 7.f;

template <int DH> struct Lay {
  // All tiles: 64 elements (128 bytes) of all rows, then the next 64. (Groups of eight tokens with both blocks
  // side by side, which one TMA box can bring, were 3 to 5% slower.)
  static constexpr int kHalf = kTile * 128;             // 64 elements of 128 rows
  static constexpr int kTileB = kHalf * (DH / 64);
  static constexpr int kStages = DH == 128 ? 5 : 10;
  static constexpr int kOffKv = 2 * kTileB;             // behind two query tiles
  static constexpr int kOffBar = kOffKv + kStages * kTileB;
  static constexpr int kSmem = kOffBar + 2048 + 1024;   // barriers, items, the units' exchange; alignment
  static constexpr uint32_t kColO = 2 * kTile;          // tensor memory: S (and P) of the units, then O
};

struct Item {
  int q0, n, L, tok0, tiles, kv0, kv1, split, h, b;
};

struct Plan {
  int target;                             // longest piece, in steps of 128 cached tokens
  int items, joins, slots;                // of one head: items, cut tiles, pieces of cut tiles
};

struct Shared {
  uint64_t full[10], empty[10];
  uint64_t q_full, q_empty, x_full, x_empty, drained;
  uint64_t s_full[2], o_full[2], p_full[2][2];
  uint64_t item_full[2], item_empty[2];
  Item item[2];
  Plan plan;
  unsigned cut;                           // pieces of cut tiles that this CTA has taken
  uint32_t tmem;
  int abort_flag;
  float2 ml[kTile];
};
static_assert(sizeof(Shared) <= 2048, "shared block");

struct TcParams {
  KvAttendArgs a;
  KvTcPlan plan;
  int per_tile;        // tokens of a 128-row tile: floor(128 / g)
  int box;             // cached tokens a TMA box takes: 8 .. 128, a power of two; 0: rows are gathered
  int64_t oob_row;     // a row index outside the gather maps
  int out_sectors;     // the output is 32-byte aligned, and with it each 16 columns of a head; else 16-byte aligned
  uint64_t wait_ns;
};

// ------------------------------------------------------------------------------------------- plan
// The list of items, which every CTA works out for itself from the rows, 32 at a time, one a lane. A row of n new
// tokens makes `tiles` tiles (or pairs of tiles), the last tokens' first, as they see most; all of a row's tiles are
// cut along the cached tokens into the same number of pieces, so that none is longer than the target.
struct Rows32 {
  int q0, n, L;                           // this lane's row
  int tiles, pieces;
  int item0, slot0, join0;                // items (of one head), pieces of cut tiles and cut tiles before the row
  int items, slots, joins;                // the same behind the 32 rows, for the whole warp
  int row0;
};

__device__ __forceinline__ int steps_of(int tokens) { return (max(tokens, 0) + kTile - 1) / kTile; }

// loads the rows row0 .. row0 + 31; cuts them by the target and counts on from `items`, `slots` and `joins`
__device__ __forceinline__ unsigned rows_load(Rows32& x, const KvRows& R, int row0, int per) {
  const int b = row0 + (threadIdx.x & 31);
  unsigned bad = 0;
  x.row0 = row0;
  x.q0 = x.n = x.L = 0;
  if (b < R.batch) kv_row(R, b, x.q0, x.n, x.L, bad);
  x.tiles = ((x.n + per - 1) / per + 1) / 2;
  return bad;
}
__device__ __forceinline__ void rows_cut(Rows32& x, int target) {
  const int lane = threadIdx.x & 31;
  x.pieces = max(1, (steps_of(x.L) + target - 1) / target);
  // three running sums in one word: items (28 bits), pieces of cut tiles (18), cut tiles (18)
  const bool cut = x.pieces > 1;
  const uint64_t v = uint64_t(x.tiles * x.pieces) | uint64_t(cut ? x.tiles * x.pieces : 0) << 28 |
                     uint64_t(cut ? x.tiles : 0) << 46;
  uint64_t y = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  const uint64_t before = y - v, all = __shfl_sync(0xffffffffu, y, 31);
  x.item0 = x.items + int(before & 0xfffffff);
  x.slot0 = x.slots + int(before >> 28 & 0x3ffff);
  x.join0 = x.joins + int(before >> 46);
  x.items += int(all & 0xfffffff);
  x.slots += int(all >> 28 & 0x3ffff);
  x.joins += int(all >> 46);
}

// The plan: the same for every warp that asks. `first` gets the first 32 rows, cut.
__device__ __forceinline__ Plan plan_rows(const TcParams& P, Rows32& first, bool report) {
  const KvRows& R = P.a.rows;
  const int lane = threadIdx.x & 31, n_kv = P.a.n_kv, sms = P.plan.sm_count;
  // this lane's rows: the longest, and the steps of all their tiles (from the first tile's and the last's)
  auto load = [&](Rows32& x, int row0, int& top, float& sum) {
    const unsigned bad = rows_load(x, R, row0, P.per_tile);
    if (bad && report) record_error(P.a.err, kCodeDevice, bad, row0 + lane, row0 + lane);
    const int c1 = steps_of(x.L), c0 = steps_of(min(x.L, x.L - x.n + min(x.n, 2 * P.per_tile)));
    top = x.tiles ? c1 : 0;
    sum = 0.5f * float(c0 + c1) * x.tiles;
  };
  int top, tiles_all;
  float sum;
  load(first, 0, top, sum);
  tiles_all = first.tiles;
  int longest = top;
  float all = sum;
  for (int row0 = 32; row0 < R.batch; row0 += 32) {
    Rows32 x;
    int t;
    float s;
    load(x, row0, t, s);
    longest = max(longest, t);
    all += s;
    tiles_all += x.tiles;
  }
  longest = max(1, __reduce_max_sync(0xffffffffu, longest));
  tiles_all = __reduce_add_sync(0xffffffffu, tiles_all);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (report && lane == 0 && tiles_all > P.plan.tile_cap) record_error(P.a.err, kCodeDevice, kErrRows, tiles_all, 0);

  int target = longest;
  if (longest > kWhole) {
    if (R.batch <= 32) {
      // Each lane weighs one way to cut: the longest row into s pieces, the others into pieces as long. The time is
      // estimated as the waves of items times their mean length and start-up, at least the longest item, and the join
      // of what was cut (six steps: with four, two ragged rows of up to 1024 new tokens at 2048 took 58 us against 34;
      // with eight, 64 new tokens at 1024 20 against 16).
      const int s = lane < 16 ? lane + 1 : lane < 24 ? 16 + (lane - 15) * 4 : 48 + (lane - 23) * 13;
      const int mine = (longest + s - 1) / s;
      const float inv = 1.f / mine;
      int items = 0, cuts = 0;
      for (int b = 0; b < R.batch; ++b) {
        const int w = __shfl_sync(0xffffffffu, first.tiles, b);
        const int p = max(1, int(ceilf(__shfl_sync(0xffffffffu, top, b) * inv - 1e-4f)));
        items += w * p;
        if (p > 1) cuts += w * p;
      }
      const float waves = ceilf(float(items) * n_kv / sms);
      float est = fmaxf(waves * (all / max(items, 1) + 2.f), mine + 2.f) + (cuts ? 6.f : 0.f);
      if (float(cuts) * n_kv > float(P.plan.slots)) est = INFINITY;
      // the best way, the fewest pieces among equals; estimates are not negative, so their bits order them
      const unsigned e = __float_as_uint(est);
      const int best = __ffs(__ballot_sync(0xffffffffu, e == __reduce_min_sync(0xffffffffu, e))) - 1;
      target = __shfl_sync(0xffffffffu, mine, best);
    } else {
      // many rows: where one is longer than twice an SM's share, all are cut into shares (those longer than one have
      // pieces). Cut wherever one is longer than a share, 48 rows of up to 128 new tokens up to 2048 on one key/value head
      // took 54 us against 41; uncut, 33 of 16 up to 12000 90 against 54, and 40 decodes with a chunk of 512 at 8192 102
      // against 55; cut from two on, 100 rows of up to 16 up to 1500 (12 steps, a share of six) 41 against 27.
      const int share = max(kWhole, int(ceilf(all * n_kv / sms)));
      if (longest > 2 * share) target = share;
    }
  }
  for (;;) {
    first.items = first.slots = first.joins = 0;
    rows_cut(first, target);
    Rows32 x = first;
    for (int row0 = 32; row0 < R.batch; row0 += 32) {
      rows_load(x, R, row0, P.per_tile);
      rows_cut(x, target);
    }
    // A cut that the workspace does not hold is made coarser until it fits: the first branch weighs with rounded quotients,
    // the second not at all (a row of two shares whose first new tokens see little has as many pieces as one whose all see
    // much). Left whole instead, a decode at 57000 beside a prompt of 7400 and 31 short rows took 441 us against 129.
    if (x.slots == 0 || (int64_t)x.slots * n_kv <= P.plan.slots) return Plan{target, x.items, x.joins, x.slots};
    target = min(longest, target + (target + 3) / 4);
  }
}

// ------------------------------------------------------------------------------------------- join
// 32 bytes of output; `sector`: p is 32-byte aligned, as one store of that size needs
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], int sector) {
  if (!sector) {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The join, by the softmax warps of all CTAs once every piece is stored: o = sum_k 2^(m_k - M) o_k / L over a tile's
// pieces, in their order. A warp takes 32 query rows, a lane one, and 16 columns; four pieces' loads are in flight at a
// time (they come from L2: one piece after the other took a microsecond each; eight at a time took longer, with fewer
// registers left). Where such units are no more than the CTAs and have two pieces a warp or more, a CTA takes a unit
// and its warps share the pieces: 8 new tokens at 65536 (19 pieces) 63.8 against 70.6 us, of two sequences (9 pieces)
// 92.0 against 89.3, so not there. As a kernel of its own behind this one the join took 2 to 7 us more.
constexpr int kJoinRows = 32, kJoinWarps = 8, kJoinLoads = 4;
// waits, at most `limit_ns`, until `pieces` are stored
__device__ __forceinline__ bool pieces_wait(const unsigned* stored, unsigned pieces, uint64_t limit_ns) {
  const uint64_t t0 = tc::globaltimer();
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(stored) : "memory");
    if (v == pieces) return true;
    if (tc::globaltimer() - t0 > limit_ns) return false;
    __nanosleep(50);
  }
}

struct JoinShared {
  float4 acc[kJoinWarps][4][32];
  float2 ml[kJoinWarps][32];
};
static_assert(sizeof(JoinShared) <= 2 * Lay<64>::kTileB, "in the queries' space");

template <int DH, bool BF16>
__device__ __forceinline__ void join_pieces(const TcParams& P, const Plan& plan, Rows32& rows, JoinShared& X) {
  const KvAttendArgs& a = P.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  rows.items = rows.slots = rows.joins = 0;
  rows_cut(rows, plan.target);
  // unit: columns fastest, then heads, tiles, and last the row groups of which a tile may have none
  constexpr int kParts = DH / 16;
  const int inner = plan.joins * a.n_kv * kParts;
  const int live = (min(2 * P.per_tile, a.rows.max_new) * a.g + kJoinRows - 1) / kJoinRows;
  const bool share = plan.slots >= 2 * kJoinWarps * plan.joins && (int64_t)inner * live <= gridDim.x;
  const int first = share ? blockIdx.x : blockIdx.x + gridDim.x * warp, step = gridDim.x * (share ? 1 : kJoinWarps);
  for (int un = first; un < inner * 2 * (kTile / kJoinRows); un += step) {
    const int group = un / inner, in_group = un % inner, join = in_group / kParts / a.n_kv;
    Rows32 x = rows;                                               // the row of the cut tile
    unsigned at;
    while (!(at = __ballot_sync(0xffffffffu, x.pieces > 1 && join >= x.join0 && join < x.join0 + x.tiles))) {
      rows_load(x, a.rows, x.row0 + 32, P.per_tile);
      rows_cut(x, plan.target);
    }
    const int src = __ffs(at) - 1, in_row = join - __shfl_sync(0xffffffffu, x.join0, src);
    const int q0 = __shfl_sync(0xffffffffu, x.q0, src), n = __shfl_sync(0xffffffffu, x.n, src);
    const int pieces = __shfl_sync(0xffffffffu, x.pieces, src);
    const int slot = __shfl_sync(0xffffffffu, x.slot0, src) + in_row * pieces;
    const int tok0 = (__shfl_sync(0xffffffffu, x.tiles, src) - 1 - in_row) * 2 * P.per_tile;
    const int tiles = n - tok0 > P.per_tile ? 2 : 1;
    const int h = in_group / kParts % a.n_kv, tile = group % 2, r0 = group / 2 * kJoinRows, r = r0 + lane;
    const int c0 = in_group % kParts * 4;
    if (tile >= tiles || r0 >= P.per_tile * a.g || tok0 + tile * P.per_tile + r0 / a.g >= n) continue;
    const int i = tok0 + tile * P.per_tile + r / a.g;
    const bool live_row = r < P.per_tile * a.g && i < n;
    const int64_t s0 = ((int64_t)slot * a.n_kv + h) * 2 + tile;
    const int64_t pitch = (int64_t)2 * a.n_kv * kTile;             // rows between two pieces' partials
    const float2* ml = a.part_ml + s0 * kTile + r;
    const float4* po = reinterpret_cast<const float4*>(a.part_o) + (s0 * (DH / 4) + c0) * kTile + r;
    float M = -INFINITY, L = 0.f;
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 (&v)[4], float w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c].x = fmaf(v[c].x, w, acc[c].x);
        acc[c].y = fmaf(v[c].y, w, acc[c].y);
        acc[c].z = fmaf(v[c].z, w, acc[c].z);
        acc[c].w = fmaf(v[c].w, w, acc[c].w);
      }
    };
    if (live_row) {
      const int dk = share ? kJoinWarps : 1;
#pragma unroll 1
      for (int k0 = share ? warp : 0; k0 < pieces; k0 += kJoinLoads * dk) {
        float2 v[kJoinLoads];
        float4 y[kJoinLoads][4];
#pragma unroll
        for (int e = 0; e < kJoinLoads; ++e) {
          const int k = k0 + e * dk;
          v[e] = make_float2(-INFINITY, 0.f);
          if (k >= pieces) continue;
          v[e] = __ldcg(&ml[k * pitch]);
#pragma unroll
          for (int c = 0; c < 4; ++c) y[e][c] = __ldcg(&po[k * pitch * (DH / 4) + c * kTile]);
        }
        float top = M;
#pragma unroll
        for (int e = 0; e < kJoinLoads; ++e) top = fmaxf(top, v[e].x);
        const float base = top == -INFINITY ? 0.f : top, f = exp2f(M - base);
        M = top;
        L *= f;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
#pragma unroll
        for (int e = 0; e < kJoinLoads; ++e) {
          if (k0 + e * dk >= pieces) continue;
          const float w = exp2f(v[e].x - base);
          L = fmaf(v[e].y, w, L);
          add(y[e], w);
        }
      }
    }
    if (share) {
      X.ml[warp][lane] = make_float2(M, L);
#pragma unroll
      for (int c = 0; c < 4; ++c) X.acc[warp][c][lane] = acc[c];
      tc::named_bar(1, kJoinWarps * 32);
      if (warp == 0) {
        for (int k = 1; k < kJoinWarps; ++k) M = fmaxf(M, X.ml[k][lane].x);
        const float base = M == -INFINITY ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < kJoinWarps; ++k) {
          const float2 v = X.ml[k][lane];
          float4 y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] = X.acc[k][c][lane];
          const float w = exp2f(v.x - base);
          L = fmaf(v.y, w, L);
          add(y, w);
        }
      }
    }
    if (live_row && (!share || warp == 0)) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int64_t row = (int64_t)(q0 + i) * a.n_heads + h * a.g + r % a.g;
      if (c0 == 0 && a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
      uint32_t w8[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        w8[2 * c] = pack2<BF16>(acc[c].x * inv, acc[c].y * inv);
        w8[2 * c + 1] = pack2<BF16>(acc[c].z * inv, acc[c].w * inv);
      }
      store32(static_cast<uint16_t*>(a.out) + row * DH + c0 * 4, w8, P.out_sectors);
    }
    if (share) tc::named_bar(1, kJoinWarps * 32);
  }
}

// ------------------------------------------------------------------------------------------- attend
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// steps of unit u of an item (its cached tiles), and the tile of its step k
__device__ __forceinline__ int unit_steps(const Item& it, int u, int per) {
  if (it.tiles == 1) return (it.kv1 - it.kv0 + 1 - u) / 2;
  if (u == 1) return it.kv1 - it.kv0;
  const int seen = max(0, min(it.L, it.L - it.n + it.tok0 + per));   // the first tile sees less than the second
  return max(0, min(it.kv1, (seen + kTile - 1) / kTile) - it.kv0);
}
__device__ __forceinline__ int unit_tile(const Item& it, int u, int k) {
  return it.tiles == 1 ? it.kv0 + u + 2 * k : it.kv0 + k;
}

template <int DH, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kb,
                        const __grid_constant__ CUtensorMap tm_vb, const TcParams P) {
  using Y = Lay<DH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& S = *reinterpret_cast<Shared*>(smem + Y::kOffBar);
  volatile int* abort_flag = &S.abort_flag;
  const KvAttendArgs& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Y::kStages; ++i) {
      tc::mbar_init(&S.full[i], 1);
      tc::mbar_init(&S.empty[i], 1);
    }
    tc::mbar_init(&S.q_full, 1);
    tc::mbar_init(&S.q_empty, 1);              // the products that read the queries
    tc::mbar_init(&S.x_full, 4);
    tc::mbar_init(&S.x_empty, 4);
    tc::mbar_init(&S.drained, 1);
    for (int u = 0; u < 2; ++u) {
      tc::mbar_init(&S.s_full[u], 1);
      tc::mbar_init(&S.o_full[u], 1);
      for (int k = 0; k < 2; ++k) tc::mbar_init(&S.p_full[u][k], 4);
      tc::mbar_init(&S.item_full[u], 1);
      tc::mbar_init(&S.item_empty[u], 10);     // eight softmax warps, the MMA warp, the value loader
    }
    S.abort_flag = 0;
    S.cut = 0;
    tc::fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(&S.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = S.tmem;
  grid_wait();                                 // for the plan
  grid_release();

  if (warp >= 8) {
    tc::regs_shrink<kRegsOther>();
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------------ loaders
      // Warp 8 takes the items and loads Q and K, warp 10 V. Both count every stage of the ring, in the order
      // in which the products take them: K runs one tile ahead of V, two where the units alternate. Copies are
      // issued by one lane with uniform operands: 32 lanes issuing their own took 90 ns a copy.
      const bool keys = warp == 8;
      const CUtensorMap* rows_map = keys ? &tm_k : &tm_v;
      const CUtensorMap* box_map = keys ? &tm_kb : &tm_vb;
      Rows32 rows;
      Plan plan{};
      if (keys) {
        plan = plan_rows(P, rows, blockIdx.x == 0);
        if (lane == 0) S.plan = plan;        // the first item's arrival publishes it
      }
      const int total = plan.items * a.n_kv;
      const int oob = int(P.oob_row), box = P.box, n_box = box ? kTile / box : 0;
      const int ps = a.pages.page_size, tile_pages = kTile / ps, tile_rest = kTile % ps;
      const int table_pages = int(a.rows.table_pages), n_pages = int(a.pages.n_pages);
      const int oob_slot = n_pages * ps;
      int st = 0, loads_q = 0, seq = 0;    // the ring's next stage; stages counted
      int n_x = 0;                         // exchanges of the units, and whether the last is still to be waited for
      bool exchanged = false;
      uint32_t par = 1, mine = 0;          // what `empty` is waited for; which of the last stages this warp filled
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_short(bar, phase, abort_flag, P.wait_ns));
        return ok;
      };
      if (lane == 0) {
        if (keys) tc::tma_prefetch(&tm_q);
        tc::tma_prefetch(rows_map);
        tc::tma_prefetch(box_map);
      }
      for (int i = 0; ok; ++i) {
        Item it{};
        if (keys) {
          if (!wait(&S.item_empty[i & 1], ((i >> 1) & 1) ^ 1)) break;
          int idx = 0;
          if (lane == 0) idx = (int)atomicAdd(&P.plan.head->next, 1u);
          idx = __shfl_sync(0xffffffffu, idx, 0);
          if (idx < total) {
            const int e = idx / a.n_kv;    // never less than the one before
            while (e >= rows.items) {
              rows_load(rows, a.rows, rows.row0 + 32, P.per_tile);
              rows_cut(rows, plan.target);
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, e < rows.item0 + rows.tiles * rows.pieces)) - 1;
            const int in_row = e - __shfl_sync(0xffffffffu, rows.item0, src);
            const int pieces = __shfl_sync(0xffffffffu, rows.pieces, src), tile = in_row / pieces;
            it.b = rows.row0 + src;
            it.h = idx % a.n_kv;
            it.q0 = __shfl_sync(0xffffffffu, rows.q0, src);
            it.n = __shfl_sync(0xffffffffu, rows.n, src);
            it.L = __shfl_sync(0xffffffffu, rows.L, src);
            it.tok0 = (__shfl_sync(0xffffffffu, rows.tiles, src) - 1 - tile) * 2 * P.per_tile;
            it.tiles = it.n - it.tok0 > P.per_tile ? 2 : 1;
            const int last = min(it.n, it.tok0 + it.tiles * P.per_tile) - 1;
            const int steps = steps_of(min(it.L, it.L - it.n + last + 1)), len = (steps + pieces - 1) / pieces;
            it.kv0 = min(steps, in_row % pieces * len);
            it.kv1 = min(steps, it.kv0 + len);
            it.split = pieces > 1 ? __shfl_sync(0xffffffffu, rows.slot0, src) + in_row : -1;
          }
          if (lane == 0) {
            S.item[i & 1] = it;
            tc::mbar_arrive(&S.item_full[i & 1]);
          }
        } else {
          if (!wait(&S.item_full[i & 1], (i >> 1) & 1)) break;
          it = S.item[i & 1];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
        }
        const int b = __shfl_sync(0xffffffffu, it.b, 0), L = __shfl_sync(0xffffffffu, it.L, 0);
        const int h = __shfl_sync(0xffffffffu, it.h, 0), tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
        const int kv0 = __shfl_sync(0xffffffffu, it.kv0, 0), kv1 = __shfl_sync(0xffffffffu, it.kv1, 0);
        if (tiles == 0) break;
        if (kv1 == kv0) continue;
        const int32_t* table = a.rows.page_table ? a.rows.page_table + (int64_t)b * table_pages : nullptr;
        if (keys) {
          // the queries' space: read by the last item's products and, where its units met there, by warpgroup 0
          if (!wait(&S.q_empty, (loads_q & 1) ^ 1)) break;
          if (exchanged && !wait(&S.x_empty, n_x++ & 1)) break;
          exchanged = tiles == 1 && kv1 - kv0 > 1;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&S.q_full, uint32_t(tiles) * P.per_tile * a.g * DH * 2);
            for (int t = 0; t < tiles; ++t)
              for (int c = 0; c < DH / 64; ++c)
                tc::tma_load_3d(smem + t * Y::kTileB + c * Y::kHalf, &tm_q, &S.q_full, c * 64, h * a.g,
                                it.q0 + it.tok0 + t * P.per_tile);
          }
          ++loads_q;
          __syncwarp();
        }
        // One tile of 128 cached tokens: boxes of `box` tokens where they lie in one page below the length, and
        // rows gathered four at a time where not (the box that holds the length's end; pages of odd sizes).
        // A lane looks up the slot of its box one tile ahead: the next tile's is 128 tokens on.
        const int g0 = box ? L & -box : 0, g1 = box && g0 < L ? g0 + box : g0;   // the box with the length's end
        int tb = kv0 * kTile + lane * box;
        int pg = tb / ps, off = tb - pg * ps;   // without a table ps is not exceeded: pg is 0
        int next_page = -1, next_off = 0, next_t = 0;
        auto look = [&]() {
          next_page = table ? -1 : b;
          if (lane < n_box && tb < L && table && pg < table_pages) next_page = table[pg];
          next_off = off;
          next_t = tb;
          tb += kTile;
          pg += tile_pages;
          off += tile_rest;
          if (off >= ps) {
            off -= ps;
            ++pg;
          }
        };
        if (box) look();
        auto load = [&](int j) {
          const int t0 = j * kTile;
          int slot = oob_slot;                   // of this lane's box; outside the pool: zeros
          if (lane < n_box && next_t < L) {
            if (next_page >= 0 && next_page < n_pages) slot = next_page * ps + next_off;
            else record_error(a.err, kCodeDevice, kErrPage, next_t, b);
          }
          const int lo = box ? g0 : t0, hi = box ? g1 : t0 + kTile;   // the rows to gather
          const bool gather = lo < hi && lo < t0 + kTile && hi > t0;
          int r[4];
          if (gather) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = lo + lane * 4 + e;
              r[e] = oob;
              if (t < hi && t < L) {
                const int64_t s = kv_slot(a.rows, a.pages, b, t);
                if (s >= 0) r[e] = int(s) * a.n_kv + h;
                else record_error(a.err, kCodeDevice, kErrPage, t, b);
              }
            }
          }
          if (!wait(&S.empty[st], par)) return;
          uint8_t* dst = smem + Y::kOffKv + st * Y::kTileB;
          if (tc::elect_one()) tc::mbar_arrive_expect_tx(&S.full[st], Y::kTileB);
          __syncwarp();
          const int skip = gather && box ? (lo - t0) / box : -1;
          for (int x = 0; x < n_box; ++x) {
            const int sx = __shfl_sync(0xffffffffu, slot, x);
            if (x != skip && tc::elect_one()) {
#pragma unroll
              for (int c = 0; c < DH / 64; ++c)
                tc::tma_load_3d(dst + c * Y::kHalf + x * box * 128, box_map, &S.full[st], c * 64, h, sx);
            }
            __syncwarp();
          }
          if (gather) {
            uint8_t* gd = dst + (lo - t0) * 128;
            for (int x = 0; x < (hi - lo) / 4; ++x) {
              const int r0 = __shfl_sync(0xffffffffu, r[0], x), r1 = __shfl_sync(0xffffffffu, r[1], x);
              const int r2 = __shfl_sync(0xffffffffu, r[2], x), r3 = __shfl_sync(0xffffffffu, r[3], x);
              if (tc::elect_one()) {
#pragma unroll
                for (int c = 0; c < DH / 64; ++c)
                  tc::tma_gather4(gd + c * Y::kHalf + x * 512, rows_map, &S.full[st], c * 64, r0, r1, r2, r3);
              }
              __syncwarp();
            }
          }
          mine |= 1u;
          if (box) look();
        };
        auto step = [&](bool k_tile, int j) {
          mine <<= 1;
          ++seq;
          if (k_tile == keys && !(P.plan.test_stall && !keys)) load(j);
          if (++st == Y::kStages) {
            st = 0;
            par ^= 1;
          }
        };
        const int lead = min(tiles == 1 ? 2 : 1, kv1 - kv0);
        for (int j = kv0; ok && j < kv0 + lead; ++j) step(true, j);
        for (int j = kv0; ok && j < kv1; ++j) {
          step(false, j);
          if (ok && j + lead < kv1) step(true, j + lead);
        }
      }
      if (!ok) {   // copies still in flight must land before the CTA exits
        volatile int quiet = 0;
        for (int d = 0; d < Y::kStages && d < seq; ++d) {
          const int p = seq - 1 - d;
          if (mine >> d & 1u) tc::mbar_wait_bounded(&S.full[p % Y::kStages], (p / Y::kStages) & 1, &quiet, P.wait_ns / 10);
        }
        if (loads_q) tc::mbar_wait_bounded(&S.q_full, (loads_q - 1) & 1, &quiet, P.wait_ns / 10);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA
      // The whole warp walks the loop, so that stages and descriptors stay in uniform registers, and one lane
      // issues: from a branch of one thread each product took 80 cycles to issue, longer than it runs. One warp
      // issues for both units, in turn: with a warp each, the units fell into step and waited together.
      const uint32_t id_qk = tc::idesc_f16(kTile, kTile, BF16);
      const uint32_t id_pv = tc::idesc_f16(kTile, DH, BF16) | tc::kIdescBMajorMN;
      const uint32_t base = tc::smem_addr(smem);
      const uint64_t dq = tc::sdesc_sw128(base, 16, 1024), dk = tc::sdesc_sw128(base + Y::kOffKv, 16, 1024);
      const uint64_t dv = tc::sdesc_sw128(base + Y::kOffKv, Y::kHalf, 1024);
      int st = 0, loads_q = 0;           // the ring's stage that comes next
      uint32_t par = 0, np[2] = {0, 0};  // its phase; the weights' phases of the units
      // A wait that gives up only raises the abort flag, at which every later wait gives up at once; the loop
      // looks at the flag once a tile, so that a wait that need not wait costs little more than its test.
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (!tc::mbar_try_wait(bar, phase)) tc::mbar_wait_short(bar, phase, abort_flag, P.wait_ns);
      };
      auto stage = [&]() -> int {        // waits for the next stage of the ring and takes it
        const int s = st;
        wait(&S.full[s], par);
        if (++st == Y::kStages) {
          st = 0;
          par ^= 1;
        }
        return s;
      };
      // S_u = Q K^T of key stage s; `last`: the item's last product that reads the queries
      auto qk = [&](int u, uint64_t q, int s, bool free, bool last) {
        const uint64_t kd = dk + uint64_t(s) * (Y::kTileB >> 4);
        __syncwarp();
        tc::tc_fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t off = ((k / 4) * Y::kHalf + (k % 4) * 32) >> 4;
            tc::umma_f16(tmem + u * kTile, q + off, kd + off, id_qk, k != 0);
          }
          tc::umma_commit(&S.s_full[u]);
          if (free) tc::umma_commit(&S.empty[s]);
          if (last) tc::umma_commit(&S.q_empty);
        }
      };
      // O_u += P_u V of value stage s, the first half's weights first; `last`: the item's last for the unit
      auto pv = [&](int u, int s, bool first, bool free, bool last) {
        const uint64_t vd = dv + uint64_t(s) * (Y::kTileB >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(&S.p_full[u][half], np[u]);
          __syncwarp();
          tc::tc_fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int k = half * 4; k < half * 4 + 4; ++k)
              tc::umma_f16_ts(tmem + Y::kColO + u * DH, tmem + u * kTile + k * 8, vd + ((k * 2048) >> 4), id_pv,
                              !first || k != 0);
            if (half == 1 && free) tc::umma_commit(&S.empty[s]);
            if (half == 1 && last) tc::umma_commit(&S.o_full[u]);
          }
        }
        np[u] ^= 1;
      };
      auto dead = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };
      for (int i = 0;; ++i) {
        wait(&S.item_full[i & 1], (i >> 1) & 1);
        if (dead()) break;
        Item it = S.item[i & 1];
        it.L = __shfl_sync(0xffffffffu, it.L, 0);
        it.n = __shfl_sync(0xffffffffu, it.n, 0);
        it.tok0 = __shfl_sync(0xffffffffu, it.tok0, 0);
        it.tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
        it.kv0 = __shfl_sync(0xffffffffu, it.kv0, 0);
        it.kv1 = __shfl_sync(0xffffffffu, it.kv1, 0);
        if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
        if (it.tiles == 0) break;
        const int n = it.kv1 - it.kv0;
        if (n == 0) continue;
        wait(&S.q_full, loads_q & 1);
        ++loads_q;
        if (it.tiles == 2) {
          // both units over each tile; unit 0 may see fewer (it stops first)
          const int n0 = unit_steps(it, 0, P.per_tile);
          const uint64_t dq1 = dq + (Y::kTileB >> 4);
          int sk = stage();
          if (n0 > 0) qk(0, dq, sk, false, false);
          qk(1, dq1, sk, true, n == 1);
          for (int k = 0; k < n; ++k) {
            if (dead()) break;
            const int sv = stage();
            if (k < n0) pv(0, sv, k == 0, false, k + 1 == n0);
            if (k + 1 < n) {
              sk = stage();
              if (k + 1 < n0) qk(0, dq, sk, false, false);
            }
            pv(1, sv, k == 0, true, k + 1 == n);
            if (k + 1 < n) qk(1, dq1, sk, true, k + 2 == n);
          }
        } else {
          // the units take the tiles in turn
          for (int k = 0; k < min(n, 2); ++k) {
            const int s = stage();
            qk(k, dq, s, true, k + 1 == n);
          }
          for (int k = 0; k < n; ++k) {
            if (dead()) break;
            const int sv = stage();
            pv(k & 1, sv, k < 2, true, k + 2 >= n);
            if (k + 2 < n) {
              const int sk = stage();
              qk(k & 1, dq, sk, true, k + 3 == n);
            }
          }
        }
        __syncwarp();
      }
      __syncwarp();
      // every product issued has completed once this commit lands
      volatile int quiet = 0;
      if (tc::elect_one()) tc::umma_commit(&S.drained);
      __syncwarp();
      tc::mbar_wait_bounded(&S.drained, 0, &quiet, P.wait_ns);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    tc::regs_grow<kRegsSoftmax>();
    const int u = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                        // query row of the tile = lane of tensor memory
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + u * kTile, t_o = tmem + lanes + Y::kColO + u * DH;
    const float c = a.scale_log2;
    const uint64_t c2 = pair(c, c);
    int n_s = 0, n_o = 0, n_o0 = 0, n_x = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait_short(bar, par, abort_flag, P.wait_ns));
      tc::tc_fence_after();
      return ok;
    };
    for (int i = 0; ok; ++i) {
      if (!wait(&S.item_full[i & 1], (i >> 1) & 1)) break;
      const Item it = S.item[i & 1];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
      if (it.tiles == 0) break;
      if (threadIdx.x == 0 && it.split >= 0) ++S.cut;
      const int tile = it.tiles == 2 ? u : 0;
      const int first_tok = it.tok0 + tile * P.per_tile;
      const int tok = first_tok + r / a.g;
      const bool live = r < P.per_tile * a.g && tok < it.n;
      const int vis = it.L - it.n + tok;                         // last slot this row sees
      const int vis_min = it.L - it.n + first_tok;               // every row of the tile sees slots up to here
      const int steps = unit_steps(it, u, P.per_tile);
      const bool exchange = it.tiles == 1 && it.kv1 - it.kv0 > 1;

      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < steps; ++k) {
        if (!wait(&S.s_full[u], n_s & 1)) break;
        ++n_s;
        const int t0 = unit_tile(it, u, k) * kTile;
        if (t0 + kTile - 1 > vis_min) {
          // tokens that a row does not see: masked in tensor memory, so that the common tile's code stays short
          const int lim = vis - t0;
#pragma unroll 1
          for (int x = 0; x < kTile; x += 32) {
            uint32_t w[32];
            tc::tmem_ld32_nowait(t_s + x, w);
            tc::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 32; ++y) w[y] = x + y > lim ? 0xff800000u : w[y];
            tc::tmem_st32(t_s + x, w);
          }
          tc::tmem_st_wait();
        }
        float s[kTile];
#pragma unroll
        for (int x = 0; x < 4; ++x) tc::tmem_ld32_nowait(t_s + x * 32, reinterpret_cast<uint32_t*>(s) + x * 32);
        tc::tmem_ld_wait();
        float mx[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) mx[y] = fmaxf(s[y], s[y + 4]);
#pragma unroll
        for (int x = 8; x < kTile; x += 8) {
#pragma unroll
          for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[x + y], s[x + 4 + y]);
        }
        const float top = softmax_base<BF16>(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c, kLift);
        const bool raise = top > m + kRaise;                     // true on the first finite score
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? top : m;
          const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - mn);
          m = mn;
          l *= f;
          if (k > 0) {   // s_full also says that the product before it, into O, has completed
#pragma unroll 1
            for (int x = 0; x < DH; x += 16) {
              uint32_t o[16];
              tc::tmem_ld16_nowait(t_o + x, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc::tmem_st16(t_o + x, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;             // nothing seen yet: every p is 2^-inf = 0
        const uint64_t n2 = pair(neg, neg);
        uint64_t sum2[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float2 e = unpair(fma2(pair(s[x * 32 + 2 * y], s[x * 32 + 2 * y + 1]), c2, n2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            sum2[y & 1] = add2(sum2[y & 1], pair(p0, p1));
            p[y] = pack2<BF16>(p0, p1);
          }
          tc::tmem_st16(t_s + x * 16, p);
          if (x & 1) {                                           // 64 tokens' weights: the product may begin
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.p_full[u][x >> 1]);
          }
        }
        const float2 z = unpair(add2(sum2[0], sum2[1]));
        l += z.x + z.y;
      }
      if (!ok) break;

      // the unit's row: O / l, or its partial
      if (steps > 0) {
        if (!wait(&S.o_full[u], n_o & 1)) break;
        ++n_o;
      }
      float* xs = reinterpret_cast<float*>(smem);                // [d / 4][128 rows][4] in the queries' space
      if (u == 1 && unit_steps(it, 0, P.per_tile) > 0) ++n_o0;
      if (exchange && u == 1) {
        if (!wait(&S.o_full[0], (n_o0 - 1) & 1)) break;          // unit 0's products read the queries too
#pragma unroll 1
        for (int x = 0; x < DH / 32; ++x) {
          uint32_t o[32];
          tc::tmem_ld32_nowait(t_o + x * 32, o);
          tc::tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 8; ++y)
            *reinterpret_cast<uint4*>(xs + ((x * 8 + y) * kTile + r) * 4) =
                make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        }
        S.ml[r] = make_float2(m, l);
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.x_full);
        continue;
      }
      if (it.tiles == 1 && u == 1) continue;                     // a single step: unit 0 has all of it
      float f0 = 1.f, f1 = 0.f;
      if (exchange) {
        if (!wait(&S.x_full, n_x & 1)) break;
        ++n_x;
        const float2 o1 = S.ml[r];
        const float mn = fmaxf(m, o1.x), b0 = mn == -INFINITY ? 0.f : mn;
        f0 = exp2f(m - b0);
        f1 = exp2f(o1.x - b0);
        l = fmaf(l, f0, o1.y * f1);
        m = mn;
      }
      const int64_t row = (int64_t)(it.q0 + tok) * a.n_heads + it.h * a.g + r % a.g;
      const int64_t slot = ((int64_t)it.split * a.n_kv + it.h) * 2 + tile;
      if (it.split < 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f0 *= inv;
        f1 *= inv;
        if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        if (live) a.part_ml[slot * kTile + r] = make_float2(m, l);
      }
#pragma unroll 1
      for (int x = 0; x < DH / 32; ++x) {
        float o[32];
        if (steps > 0) {
          tc::tmem_ld32_nowait(t_o + x * 32, reinterpret_cast<uint32_t*>(o));
          tc::tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] *= f0;
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0.f;
        }
        if (exchange) {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float4 v = *reinterpret_cast<const float4*>(xs + ((x * 8 + y) * kTile + r) * 4);
            o[4 * y] = fmaf(v.x, f1, o[4 * y]);
            o[4 * y + 1] = fmaf(v.y, f1, o[4 * y + 1]);
            o[4 * y + 2] = fmaf(v.z, f1, o[4 * y + 2]);
            o[4 * y + 3] = fmaf(v.w, f1, o[4 * y + 3]);
          }
        }
        if (it.split >= 0 && live) {
          float4* po = reinterpret_cast<float4*>(a.part_o) + (slot * (DH / 4) + x * 8) * kTile + r;
#pragma unroll
          for (int y = 0; y < 8; ++y) po[y * kTile] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        } else if (it.split < 0 && live) {
          uint16_t* out = static_cast<uint16_t*>(a.out) + row * DH + x * 32;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t w[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) w[z] = pack2<BF16>(o[16 * y + 2 * z], o[16 * y + 2 * z + 1]);
            store32(out + 16 * y, w, P.out_sectors);
          }
        }
      }
      tc::tc_fence_before();
      if (exchange) {                                            // the queries' space is read: TMA may fill it again
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.x_empty);
      }
    }
    // The join. Every item has been taken when a CTA comes here, by CTAs that run and wait for none: the wait for
    // their pieces ends whichever CTAs the GPU holds. All warps meet first, also after a wait that gave up.
    const auto any = [](bool bad) { return tc::named_bar_or(1, kJoinWarps * 32, bad); };
    if (!any(!ok) && S.plan.joins > 0) {
      Rows32 rows;
      rows_load(rows, a.rows, 0, P.per_tile);
      if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(&P.plan.head->pieces, S.cut);
        ok = pieces_wait(&P.plan.head->pieces, unsigned(S.plan.slots * a.n_kv), P.wait_ns);
        if (!ok) *abort_flag = 1;
      }
      // the queries' space is free: nothing is in flight behind the last item
      if (!any(!ok)) join_pieces<DH, BF16>(P, S.plan, rows, *reinterpret_cast<JoinShared*>(smem));
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (threadIdx.x == 0) {
    if (*abort_flag) record_error(a.err, kCodeTimeout, kErrWait, blockIdx.x, 0);
    // the last CTA to end sets the counters back for the next call; `done` wraps to zero by itself
    __threadfence();
    if (atomicInc(&P.plan.head->done, gridDim.x - 1) == gridDim.x - 1) P.plan.head->next = P.plan.head->pieces = 0;
  }
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

template <int DH, bool BF16> cudaError_t prepare_tc() {
  return cudaFuncSetAttribute(kv_attend_tc_kernel<DH, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Lay<DH>::kSmem);
}
template <int DH, bool BF16> cudaError_t launch_tc(const KvAttendArgs& a, const KvTcPlan& t, cudaStream_t st) {
  const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  TcParams P{};
  P.a = a;
  P.plan = t;
  P.per_tile = kTile / a.g;
  const int64_t rows = a.pages.n_pages * a.pages.page_size * a.n_kv;
  P.oob_row = rows;
  P.out_sectors = (uintptr_t)a.out % 32 == 0;
  P.wait_ns = t.wait_ns;
  CUtensorMap tm_q, tm_k, tm_v, tm_kb, tm_vb;
  {
    // queries [token][head][d]: boxes of 64 columns, one group's heads, a tile's tokens
    const cuuint64_t dims[3] = {DH, (cuuint64_t)a.n_heads, (cuuint64_t)a.rows.n_tokens};
    const cuuint64_t strides[2] = {DH * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)P.per_tile};
    if (!tma_encode(&tm_q, dt, 3, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  {
    // cached head rows [slot][kv head][d] as one list of rows, gathered four at a time
    const cuuint64_t dims[2] = {DH, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {DH * 2};
    const cuuint32_t box[2] = {64, 1};
    const cuuint64_t bdims[3] = {DH, (cuuint64_t)a.n_kv, (cuuint64_t)(a.pages.n_pages * a.pages.page_size)};
    const cuuint64_t bstrides[2] = {DH * 2, (cuuint64_t)a.n_kv * DH * 2};
    // A box must lie in one page: without a table a row is one page, else the largest power of two that divides it.
    // 512 new tokens at 8192: 77 us from pages of 64 and more, 80 of 16, 94 of 8, and 158 gathered from pages of 100 or 1.
    int box_tokens = a.rows.page_table ? a.pages.page_size & -a.pages.page_size : kTile;
    box_tokens = box_tokens > kTile ? kTile : box_tokens;
    P.box = box_tokens >= 8 ? box_tokens : 0;
    const cuuint32_t bbox[3] = {64, 1, (cuuint32_t)(P.box ? P.box : 8)};
    if (!tma_encode(&tm_kb, dt, 3, a.pages.k, bdims, bstrides, bbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tma_encode(&tm_vb, dt, 3, a.pages.v, bdims, bstrides, bbox, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    if (!tma_encode(&tm_k, dt, 2, a.pages.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    if (!tma_encode(&tm_v, dt, 2, a.pages.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  const int64_t most = ((int64_t)t.tile_cap + t.slots) * a.n_kv;
  const unsigned grid = (unsigned)(most < t.sm_count ? most : t.sm_count);
  return launch_early(kv_attend_tc_kernel<DH, BF16>, dim3(grid), kThreads, Lay<DH>::kSmem, st, tm_q, tm_k, tm_v, tm_kb,
                      tm_vb, P);
}

}  // namespace

cudaError_t prepare_kv_attend_tc(int head_dim, bool bf16) {
  if (head_dim == 128) return bf16 ? prepare_tc<128, true>() : prepare_tc<128, false>();
  return bf16 ? prepare_tc<64, true>() : prepare_tc<64, false>();
}

cudaError_t launch_kv_attend_tc(const KvAttendArgs& a, const KvTcPlan& t, cudaStream_t st) {
  if (!tma_available()) return cudaErrorNotSupported;
  if (a.head_dim == 128) return a.bf16 ? launch_tc<128, true>(a, t, st) : launch_tc<128, false>(a, t, st);
  return a.bf16 ? launch_tc<64, true>(a, t, st) : launch_tc<64, false>(a, t, st);
}

}  // namespace palu
