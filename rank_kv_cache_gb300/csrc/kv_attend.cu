// Attention of few new tokens over a paged KV cache: decode steps, drafted tokens.
//
//   o = softmax(q K^T / sqrt(d)) V over slots 0 .. L - n + i of the query's row,  lse = ln sum e^s.
//
// A unit is (row, key/value head): query row r = i g + j of its n g <= 16 is new token i under head j of
// the g heads that share the key/value head. Bound: HBM, each cached row is read once for the whole
// group. The query rows are those of 16-row matrix instructions (mma.sync m16n8k16, fp32 accumulation):
// the 128-row tcgen05 shapes would leave 7/8 of their rows empty here, and the rate needed, 16 rows
// for every 4 d cached bytes, is a few per cent of what this instruction gives.
//
// The units' steps of 64 cached tokens (d = 64: 128) are cut into pieces of about one length, so many that
// they fill the GPU in whole waves, two CTAs an SM (one's start and join hide behind the other's stream).
// The lengths are read on the device: rows of unlike lengths give unlike numbers of pieces. The last CTA of
// a cut unit to finish joins its pieces in their order.
//
// A CTA's four warps take 16 tokens (d = 64: 32) in turn, each with its own online softmax (fp32 maximum,
// sum and output) and its own three-stage ring of cp.async copies, so no barrier stands between the warps
// until they are joined. Rows past the end are written as zeros into shared memory and masked, never
// read. The weights p are rounded to the cache's type for the product with V, as the matrix instruction
// takes it (fp16: up to 2^15, see softmax_base); the sum is of the unrounded p.
//
// Measured on a GB300 with states in turn, 32 / 8 heads of 128, bf16: one token of four sequences at 65536 (1.07 GB)
// 162 to 166 us, 6450 to 6600 GB/s; of 64 sequences at 4096 165 us from pages of 64, 174 of 16; of 256 at 1024 186.
// 32 / 32 heads, one sequence at 4096 (67 MB): 20 us, 16.5 with the cache in L2, of which the start and the join are
// half. 8 / 8 heads of 64, one at 512: 8 us.
#include "kv.h"

namespace palu {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr float kLift = 15.f;            // log2 of the largest fp16 weight

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int DH> struct Sm {
  static constexpr int kTok = kKvFewTokens / kWarps * 128 / DH;   // tokens a warp takes at once: 16, or 32 of d = 64
  static constexpr int kStep = kWarps * kTok;
  static constexpr int kRow = DH * 2;                       // bytes of a token's head row
  static constexpr int kTile = kTok * kRow;                 // one warp's K (or V) stage
  static constexpr int kWarp = kStages * 2 * kTile;
  static constexpr int kBytes = kWarps * kWarp;
  static_assert(kKvFewRows * 2 * kKvFewMostCtas * 4 <= kBytes && kWarps * kKvFewRows * DH * 4 <= kBytes, "joins");
};

// Rows are stored with their 16-byte chunks exchanged by the row's low three bits, so that the eight
// rows of an ldmatrix fall into different banks.
template <int DH> __device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return uint32_t(row * (DH * 2) + ((chunk ^ (row & 7)) << 4));
}

// How the rows' steps are cut: the pieces of each row (32 rows at a time, one a lane) and the numbers of the first
// of them among all pieces, and among those of cut units. Every warp works it out for itself, alike.
struct Cut {
  int per;          // steps of a piece, at most
  int pieces;       // of this lane's row, for each of its key/value heads
  int start, cut;   // pieces (of one head) of the rows before it; those of cut units
  int total, total_cut;
};

__device__ __forceinline__ void cut_rows(int steps, int per, Cut& c, int base, int base_cut) {
  const int lane = threadIdx.x & 31;
  c.per = per;
  c.pieces = (steps + per - 1) / per;
  int x = c.pieces, y = c.pieces > 1 ? c.pieces : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  c.start = base + x - c.pieces;
  c.cut = base_cut + y - (c.pieces > 1 ? c.pieces : 0);
  c.total = base + __shfl_sync(0xffffffffu, x, 31);
  c.total_cut = base_cut + __shfl_sync(0xffffffffu, y, 31);
}

template <int DH, bool BF16>
__global__ void __launch_bounds__(kWarps * 32, 2) kv_attend_few_kernel(const KvAttendArgs a) {
  using S = Sm<DH>;
  constexpr int kTok = S::kTok, kNT = kTok / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 ml_s[kWarps][kKvFewRows];
  __shared__ float wgt[kWarps][kKvFewRows];
  __shared__ float2 tot[kKvFewRows];
  __shared__ int last_cta;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const KvRows& R = a.rows;
  grid_wait();
  grid_release();

  // steps of a row (0: nothing to do); one without cached tokens takes a step too, for its empty outputs
  auto row_steps = [&](int b, bool report) -> int {
    if (b >= R.batch) return 0;
    int q0, n, L;
    unsigned bad;
    const bool use = kv_row(R, b, q0, n, L, bad);
    if (bad && report) record_error(a.err, kCodeDevice, bad, b, b);
    return !use || n == 0 ? 0 : max(1, (L + S::kStep - 1) / S::kStep);
  };
  const int steps0 = row_steps(lane, blockIdx.x == 0 && warp == 0);
  int64_t all = __reduce_add_sync(0xffffffffu, steps0);
  for (int b0 = 32; b0 < R.batch; b0 += 32)
    all += __reduce_add_sync(0xffffffffu, row_steps(b0 + lane, blockIdx.x == 0 && warp == 0));
  if (all == 0) return;
  // A piece's length: at least an equal share of all CTAs that the GPU holds. Up to 32 rows, each lane weighs one
  // length, from that share to three times it or 31 steps more: the waves of CTAs times the length and what a CTA's
  // start and end cost (eight steps), and the join of what is cut (four; with eight, 8 sequences at 1000 took 12.3 us
  // against 9.6; with lengths up to twice a share of one step only, 300 tokens of two sequences 7.6 against 6.5). More
  // rows are cut a quarter longer than the share. The quarter alone took 169 us against 136 for 32 ragged rows up to
  // 8192 and 137 against 119 for 20 of 7000, and up to 1 us less for few equal rows (48.4 against 50.3, one of 65536).
  const int64_t work = all * a.n_kv;
  const int share = work < (1 << 30) ? (int(work) + a.ctas - 1) / a.ctas : int((work + a.ctas - 1) / a.ctas);
  int per = share + share / 4;
  if (R.batch <= 32) {
    const int mine = share + lane * max(1, share / 16);
    const float inv = 1.f / mine;
    int count = 0, cuts = 0;
    for (int b = 0; b < R.batch; ++b) {
      const int p = int(ceilf(__shfl_sync(0xffffffffu, steps0, b) * inv));
      count += p;
      cuts |= p > 1;
    }
    const unsigned est = unsigned((count * a.n_kv + a.ctas - 1) / a.ctas) * unsigned(mine + 8) + (cuts ? 4u : 0u);
    const unsigned least = __reduce_min_sync(0xffffffffu, est);
    per = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, est == least)) - 1);
  }
  Cut cut0;
  cut_rows(steps0, per, cut0, 0, 0);
  int pieces_all = cut0.total;
  if (R.batch > 32) {
    Cut x = cut0;
    for (int b0 = 32; b0 < R.batch; b0 += 32) cut_rows(row_steps(b0 + lane, false), per, x, x.total, x.total_cut);
    pieces_all = x.total;
  }

  // the 32 rows of the piece: a CTA's pieces only go on, so they are looked for from the last one's. (From the first row
  // each time 4096 rows of 16 tokens and 8 heads took 2437 us against 432.)
  Cut x = cut0;
  int row0 = 0;
  for (int idx = blockIdx.x; idx < pieces_all * a.n_kv; idx += gridDim.x) {
    // the piece's row b, head h and number among the unit's np, and its place among those of cut units
    unsigned at;
    while (!(at = __ballot_sync(0xffffffffu, idx < (x.start + x.pieces) * a.n_kv))) {
      row0 += 32;
      cut_rows(row_steps(row0 + lane, false), per, x, x.total, x.total_cut);
    }
    const int src = __ffs(at) - 1, b = row0 + src;
    const int np = __shfl_sync(0xffffffffu, x.pieces, src);
    const int in_row = idx - __shfl_sync(0xffffffffu, x.start, src) * a.n_kv;
    const int h = in_row / np, piece = in_row % np;
    const int first_slot = __shfl_sync(0xffffffffu, x.cut, src) * a.n_kv + h * np;
    int q0, n, L;
    unsigned bad;
    kv_row(R, b, q0, n, L, bad);
    const int rows = n * a.g;
    int len = (L + S::kStep - 1) / S::kStep;                       // the row's steps, cut evenly
    len = (len + np - 1) / np * S::kStep;
    const int t0 = min(L, piece * len), t1 = min(L, t0 + len);

    float o[DH / 8][4];
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    uint8_t* ring = smem + warp * S::kWarp;
    const uint32_t ring_a = smem_u32(ring);
    const int first = t0 + warp * kTok;
    const int n_it = first < t1 ? (t1 - first + S::kStep - 1) / S::kStep : 0;
    const uint16_t* kb = static_cast<const uint16_t*>(a.pages.k) + h * DH;
    const uint16_t* vb = static_cast<const uint16_t*>(a.pages.v) + h * DH;
    const int64_t tok_stride = (int64_t)a.n_kv * DH;

    // slot of this lane's token of step `it` (-1: past the range, or a page outside the pool)
    auto slot_of = [&](int it) -> int {
      const int t = first + it * S::kStep + lane;
      if (it >= n_it || lane >= kTok || t >= t1) return -1;
      const int64_t s = kv_slot(R, a.pages, b, t);
      if (s < 0) record_error(a.err, kCodeDevice, kErrPage, t, b);
      return int(s);
    };
    auto load = [&](int it, int slot) {
      if (it < n_it) {
        const uint32_t st = ring_a + (it % kStages) * 2 * S::kTile;
        constexpr int kCh = DH / 8;                                  // 16-byte chunks of a row
#pragma unroll
        for (int x = 0; x < kTok * kCh / 32; ++x) {
          const int row = (x * 32 + lane) / kCh, ch = lane % kCh;
          const int s = __shfl_sync(0xffffffffu, slot, row);
          const int64_t off = s < 0 ? 0 : s * tok_stride + ch * 8;
          const int bytes = s < 0 ? 0 : 16;
          cp16(st + swz<DH>(row, ch), kb + off, bytes);
          cp16(st + S::kTile + swz<DH>(row, ch), vb + off, bytes);
        }
      }
      cp_commit();
    };

    int next = slot_of(0);
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) {
      const int cur = next;
      next = slot_of(it + 1);
      load(it, cur);
    }

    // query rows as the A operand: row = lane / 4 and + 8, column pairs by lane % 4
    const int r0 = lane >> 2, cp = lane & 3;
    uint32_t qf[DH / 16][4];
    int vis[2];                                                      // last slot the two query rows see
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rr = r0 + 8 * x;
      const bool ok = rr < rows;
      const int i = rr / a.g, head = h * a.g + rr % a.g;
      vis[x] = ok ? L - n + i : -1;
      const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                            (int64_t)(q0 + i) * a.q_stride + head * DH);
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        qf[k][x] = ok ? p[k * 8 + cp] : 0u;
        qf[k][2 + x] = ok ? p[k * 8 + 4 + cp] : 0u;
      }
    }
    const int vis_min = L - n;                                       // every row sees slots up to here

    for (int it = 0; it < n_it; ++it) {
      {
        const int cur = next;
        next = slot_of(it + kStages);
        load(it + kStages - 1, cur);
      }
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t ks = ring_a + (it % kStages) * 2 * S::kTile, vs = ks + S::kTile;
      float s[kNT][4];
#pragma unroll
      for (int i = 0; i < kNT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      const int tr = ((lane >> 4) & 1) * 8 + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
#pragma unroll
        for (int p = 0; p < kNT / 2; ++p) {
          uint32_t f[4];
          ldsm4(f, ks + swz<DH>(p * 16 + tr, k * 2 + kc));
          mma<BF16>(s[2 * p], qf[k], f[0], f[1]);
          mma<BF16>(s[2 * p + 1], qf[k], f[2], f[3]);
        }
      }
      const int tb = first + it * S::kStep;
      if (tb + kTok > t1 || tb + kTok - 1 > vis_min) {
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = tb + i * 8 + cp * 2 + (e & 1);
            if (t >= t1 || t > vis[e >> 1]) s[i][e] = -INFINITY;
          }
      }
      float al[2], base[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(s[0][2 * x], s[0][2 * x + 1]);
#pragma unroll
        for (int i = 1; i < kNT; ++i) mx = fmaxf(mx, fmaxf(s[i][2 * x], s[i][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[x], softmax_base<BF16>(mx * a.scale_log2, kLift));
        base[x] = mn == -INFINITY ? 0.f : mn;                        // nothing seen yet: every p is 2^-inf = 0
        al[x] = ex2(m[x] - base[x]);
        m[x] = mn;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kNT; ++i) {
          s[i][2 * x] = ex2(fmaf(s[i][2 * x], a.scale_log2, -base[x]));
          s[i][2 * x + 1] = ex2(fmaf(s[i][2 * x + 1], a.scale_log2, -base[x]));
          sum += s[i][2 * x] + s[i][2 * x + 1];
        }
        l[x] = fmaf(l[x], al[x], sum);
      }
      if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          o[i][0] *= al[0];
          o[i][1] *= al[0];
          o[i][2] *= al[1];
          o[i][3] *= al[1];
        }
      }
      const int vr = ((lane >> 3) & 1) * 8 + (lane & 7), vc = lane >> 4;
#pragma unroll
      for (int k = 0; k < kNT / 2; ++k) {
        const uint32_t pf[4] = {pack2<BF16>(s[2 * k][0], s[2 * k][1]), pack2<BF16>(s[2 * k][2], s[2 * k][3]),
                                pack2<BF16>(s[2 * k + 1][0], s[2 * k + 1][1]),
                                pack2<BF16>(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) {
          uint32_t f[4];
          ldsm4t(f, vs + swz<DH>(k * 16 + vr, 2 * i + vc));
          mma<BF16>(o[2 * i], pf, f[0], f[1]);
          mma<BF16>(o[2 * i + 1], pf, f[2], f[3]);
        }
      }
      __syncwarp();
    }
    cp_wait<0>();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
    __syncthreads();

    // join the warps: each leaves its output rows in the (now free) ring
    float* ob = reinterpret_cast<float*>(smem) + warp * kKvFewRows * DH;
    if (cp == 0) {
      ml_s[warp][r0] = make_float2(m[0], l[0]);
      ml_s[warp][r0 + 8] = make_float2(m[1], l[1]);
    }
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) {
      *reinterpret_cast<float2*>(ob + r0 * DH + i * 8 + cp * 2) = make_float2(o[i][0], o[i][1]);
      *reinterpret_cast<float2*>(ob + (r0 + 8) * DH + i * 8 + cp * 2) = make_float2(o[i][2], o[i][3]);
    }
    __syncthreads();
    if (threadIdx.x < kKvFewRows) {
      const int r = threadIdx.x;
      float M = -INFINITY, Lsum = 0.f;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml_s[w][r].x);
      for (int w = 0; w < kWarps; ++w) {
        const float x = M == -INFINITY ? 0.f : ex2(ml_s[w][r].x - M);
        wgt[w][r] = x;
        Lsum = fmaf(ml_s[w][r].y, x, Lsum);
      }
      tot[r] = make_float2(M, Lsum);
    }
    __syncthreads();

    const float* of = reinterpret_cast<const float*>(smem);
    auto write_lse = [&](int r, float M, float Lsum) {
      if (a.lse)
        a.lse[(int64_t)(q0 + r / a.g) * a.n_heads + h * a.g + r % a.g] =
            Lsum == 0.f ? -INFINITY : (M + log2f(Lsum)) * 0.69314718055994531f;
    };
    auto out_at = [&](int r) -> int64_t { return ((int64_t)(q0 + r / a.g) * a.n_heads + h * a.g + r % a.g) * DH; };
    const bool whole = np == 1;
    float* po = a.part_o + (int64_t)(first_slot + piece) * kKvFewRows * DH;
    for (int x = tid; x < rows * (DH / 2); x += kWarps * 32) {
      const int r = x / (DH / 2), cl = x % (DH / 2) * 2;
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kWarps; ++y) {
        const float2 u = *reinterpret_cast<const float2*>(of + (y * kKvFewRows + r) * DH + cl);
        v.x = fmaf(u.x, wgt[y][r], v.x);
        v.y = fmaf(u.y, wgt[y][r], v.y);
      }
      if (whole) {
        const float Lsum = tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + out_at(r) + cl) = pack2<BF16>(v.x * inv, v.y * inv);
        if (cl == 0) write_lse(r, tot[r].x, Lsum);
      } else {
        *reinterpret_cast<float2*>(po + r * DH + cl) = v;
      }
    }
    if (!whole) {
      if (tid < rows) a.part_ml[(int64_t)(first_slot + piece) * kKvFewRows + tid] = tot[tid];
      __threadfence();
      __syncthreads();
      if (tid == 0) last_cta = atomicAdd(&a.counters[first_slot], 1u) == unsigned(np - 1);
      __syncthreads();
      if (last_cta) {
        __threadfence();
        // join the pieces, in their order
        float* wr = reinterpret_cast<float*>(smem);                  // [rows][np] weights
        auto slot = [&](int k) { return (int64_t)(first_slot + k) * kKvFewRows; };
        for (int r = warp; r < rows; r += kWarps) {
          float M = -INFINITY, Lsum = 0.f;
          for (int k = lane; k < np; k += 32) M = fmaxf(M, __ldcg(&a.part_ml[slot(k) + r]).x);
          M = warp_max(M);
          for (int k = lane; k < np; k += 32) {
            const float2 v = __ldcg(&a.part_ml[slot(k) + r]);
            const float x = M == -INFINITY ? 0.f : ex2(v.x - M);
            wr[r * np + k] = x;
            Lsum = fmaf(v.y, x, Lsum);
          }
          Lsum = warp_sum(Lsum);
          if (lane == 0) tot[r] = make_float2(M, Lsum);
        }
        __syncthreads();
        for (int x = tid; x < rows * (DH / 4); x += kWarps * 32) {
          const int r = x / (DH / 4), cl = x % (DH / 4) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k0 = 0; k0 < np; k0 += 8) {                   // eight pieces' loads in flight
            float4 u[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (k0 + y < np)
                u[y] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot(k0 + y) + r) * DH + cl));
#pragma unroll
            for (int y = 0; y < 8; ++y)
              if (k0 + y < np) {
                const float f = wr[r * np + k0 + y];
                v.x = fmaf(u[y].x, f, v.x);
                v.y = fmaf(u[y].y, f, v.y);
                v.z = fmaf(u[y].z, f, v.z);
                v.w = fmaf(u[y].w, f, v.w);
              }
          }
          const float Lsum = tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_at(r) + cl) =
              make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
          if (cl == 0) write_lse(r, tot[r].x, Lsum);
        }
        if (tid == 0) a.counters[first_slot] = 0u;
      }
    }
    __syncthreads();                                                 // the joins' space becomes the ring again
  }
}

template <int DH, bool BF16> cudaError_t prepare_few() {
  return cudaFuncSetAttribute(kv_attend_few_kernel<DH, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Sm<DH>::kBytes);
}
template <int DH, bool BF16> cudaError_t launch_few(const KvAttendArgs& a, int ctas, cudaStream_t st) {
  return launch_early(kv_attend_few_kernel<DH, BF16>, dim3(ctas), kWarps * 32, Sm<DH>::kBytes, st, a);
}

}  // namespace

cudaError_t prepare_kv_attend_few(int head_dim, bool bf16) {
  if (head_dim == 128) return bf16 ? prepare_few<128, true>() : prepare_few<128, false>();
  return bf16 ? prepare_few<64, true>() : prepare_few<64, false>();
}

cudaError_t launch_kv_attend_few(KvAttendArgs a, int sm_count, cudaStream_t st) {
  // the cut aims at the CTAs that the GPU holds; no more are launched than the rows' bounds give steps
  a.ctas = kKvFewCtas * sm_count < kKvFewMostCtas ? kKvFewCtas * sm_count : kKvFewMostCtas;
  const int step = kKvFewTokens * 128 / a.head_dim;
  const int64_t steps = (((int64_t)a.rows.max_kv_len + step - 1) / step + 1) * a.rows.batch * a.n_kv;
  const int grid = steps < a.ctas ? (int)steps : a.ctas;
  if (a.head_dim == 128) return a.bf16 ? launch_few<128, true>(a, grid, st) : launch_few<128, false>(a, grid, st);
  return a.bf16 ? launch_few<64, true>(a, grid, st) : launch_few<64, false>(a, grid, st);
}

}  // namespace palu
