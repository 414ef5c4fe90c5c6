// What the tensor-core attention kernels share: the list of items that a call's rows make, and the join of what was cut.
#pragma once

#include "kv.h"
#include "internal.h"
#include "kv_tc_ptx.cuh"

namespace palu {

constexpr int kTile = 128;               // query rows of a tile, cached tokens of a step
constexpr int kWhole = kKvTcWhole;       // tiles of so few steps are not cut: the join would cost more
// log2 by which a score may exceed the running maximum before that is raised, and by which fp16 weights are lifted
// (softmax_base): together 15, the range of the type. An fp16 weight's rounding is then at most 2^-32 of the row's
// largest. Raised from 4 on, with a lift of 11, four prompts of 4096 took 481 us against 441; from 6 on, 453.
constexpr float kRaise = 8.f, kLift = 7.f;

struct Item {
  int q0, n, L, tok0, tiles, kv0, kv1, split, h, b;
};

struct Plan {
  int target;                             // longest piece, in steps of 128 cached tokens
  int items, joins, slots;                // of one head: items, cut tiles, pieces of cut tiles
};

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

// SUB: tiles of 128 rows that an item has at most.
template <int DH, bool BF16, int SUB = 2>
__device__ __forceinline__ void join_pieces(const TcParams& P, const Plan& plan, Rows32& rows, JoinShared& X) {
  const KvAttendArgs& a = P.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  rows.items = rows.slots = rows.joins = 0;
  rows_cut(rows, plan.target);
  // unit: columns fastest, then heads, tiles, and last the row groups of which a tile may have none
  constexpr int kParts = DH / 16;
  const int per = P.per_tile / (SUB / 2);                          // tokens of 128 rows
  const int inner = plan.joins * a.n_kv * kParts;
  const int live = (min(SUB * per, a.rows.max_new) * a.g + kJoinRows - 1) / kJoinRows;
  const bool share = plan.slots >= 2 * kJoinWarps * plan.joins && (int64_t)inner * live <= gridDim.x;
  const int first = share ? blockIdx.x : blockIdx.x + gridDim.x * warp, step = gridDim.x * (share ? 1 : kJoinWarps);
  for (int un = first; un < inner * SUB * (kTile / kJoinRows); un += step) {
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
    const int tok0 = (__shfl_sync(0xffffffffu, x.tiles, src) - 1 - in_row) * SUB * per;
    const int h = in_group / kParts % a.n_kv, tile = group % SUB, r0 = group / SUB * kJoinRows, r = r0 + lane;
    const int c0 = in_group % kParts * 4;
    if (tok0 + tile * per >= n || r0 >= per * a.g || tok0 + tile * per + r0 / a.g >= n) continue;
    const int i = tok0 + tile * per + r / a.g;
    const bool live_row = r < per * a.g && i < n;
    const int64_t s0 = ((int64_t)slot * a.n_kv + h) * SUB + tile;
    const int64_t pitch = (int64_t)SUB * a.n_kv * kTile;           // rows between two pieces' partials
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

}  // namespace palu
