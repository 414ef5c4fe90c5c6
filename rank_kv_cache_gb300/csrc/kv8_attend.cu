// Attention of few new tokens over a paged KV cache held in 8 bits: decode steps, drafted tokens.
//
//   x_t = log2(e) / sqrt(d) s_k(t) q . c_k(t),   o = sum_t 2^x_t s_v(t) c_v(t) / sum_t 2^x_t,   lse = ln sum_t 2^x_t,
//
// c the e4m3 codes of slot t, s_k and s_v the scales of its block of 16 slots. The work is cut as for 16-bit caches
// (kv_attend.cu: units of up to 24 query rows of a key/value head, pieces over all CTAs, four warps with a ring of cp.async
// copies each); what differs lies between shared memory and the matrix instructions.
//   * The products are turned over: S^T = K Q^T and O^T = V^T P^T, tokens and then columns of the head being the 16 rows of
//     a matrix instruction (mma.sync m16n8k16) and query rows its 8 columns. So query rows count in eights, one to three
//     of them (NB), and codes, made fp16 in registers once, serve all.
//   * Codes become fp16 exactly, two an instruction. The order of a product's inner index is free, so a lane reads 16
//     consecutive codes of a key in one access and the queries' registers are loaded to match; of values, pairs of codes
//     are transposed as if they were 16-bit elements, and each pair parted by one byte permutation.
//   * bf16 queries become fp16, lifted by a power of two of their row so that the largest lies in [2^14, 2^15).
//   * s_k multiplies 16 scores at once. s_v belongs into the weights of the product with c_v, not into their sum: with
//     y_t = x_t + log2 s_v(t) and a running maximum M of y, weights are w_t = 2^(y_t - M), o = sum w c_v and
//     l = sum over blocks of (sum w) / s_v, so that one exponential serves both and the fp16 weights are relative to the
//     largest weight that enters the product, whatever the scales (up to 2^15 of it, see softmax_base).
//
// Bound: HBM; half the bytes of a 16-bit cache in as many copies (four tokens at 65536, 8 heads of 128, 4 query rows each: 91
// us, 5.9 TB/s of 6.8; 103 with two CTAs an SM and three stages). With more query rows the warps' own steps bound it: eight
// rows of 20 at 1600 to 16384 take 65 us at 44 % of the bandwidth. Two warps sharing their tokens took 80 us there, rows as
// the 16 of a matrix instruction (two blocks of it, half of the second empty) 67.
#include "kv8.h"
#include "kv_few.cuh"

namespace palu {
namespace {

constexpr int kWarps = kFewWarps;
constexpr float kLift = 15.f;            // log2 of the largest weight

// NB: query rows in eights. One leaves registers for three CTAs an SM, whose copies in flight then need fewer stages.
template <int DH, int NB> struct Sm {
  static constexpr int kTok = 4096 / DH;                    // tokens a warp takes at once: 32, or 64 of d = 64
  static constexpr int kBlocks = kTok / kKv8Block;
  static constexpr int kRows = 8 * NB;
  static constexpr int kCtas = NB == 1 ? 3 : 2;             // of an SM
  static constexpr int kStages = NB == 1 ? 2 : 3;
  static constexpr int kStep = kWarps * kTok;
  static constexpr int kTile = kTok * DH;                   // one warp's K (or V) stage
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kOffQ = kWarps * kRing;
  static constexpr bool kQueries = NB > 2;                  // their queries stand in shared memory: registers are short
  static constexpr int kBytes = kOffQ + (kQueries ? kRows * DH * 2 : 0);
  // a unit has at most as many pieces as the call aims at CTAs
  static_assert(kRows * (kKvFewMostCtas + 1) * 4 <= kOffQ && kWarps * kRows * DH * 4 <= kOffQ, "joins");
};

// Places of 16-byte chunks in a tile. Keys are read as 16 bytes of two tokens by eight lanes, four chunks each; values as
// eight rows of one chunk. Both then fall into different banks. Rows are 8 (d = 128) or 4 chunks long.
template <int DH> __device__ __forceinline__ uint32_t key_at(int row, int chunk) {
  return uint32_t(row * DH + ((DH == 128 ? chunk ^ (row & 1) << 2 : chunk) << 4));
}
template <int DH> __device__ __forceinline__ uint32_t value_at(int row, int chunk) {
  return uint32_t(row * DH + ((chunk ^ (DH == 128 ? row & 7 : (row >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// 4 bytes global -> shared; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// an 8 x 8 matrix of 16-bit elements, two of a row a lane, turned over
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int DH, bool BF16, int NB>
__global__ void __launch_bounds__(kWarps * 32, (Sm<DH, NB>::kCtas)) kv8_attend_few_kernel(const Kv8AttendArgs A) {
  using S = Sm<DH, NB>;
  constexpr int kTok = S::kTok, kBlocks = S::kBlocks, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FewJoin<S::kRows> X;
  __shared__ float scales[kWarps][kStages][2][kBlocks];
  const KvAttendArgs& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  const int per = piece_length(steps0, all, R.batch, a.n_kv, a.ctas);
  Cut cut0;
  cut_rows(steps0, per, cut0, 0, 0);
  int pieces_all = cut0.total;
  if (R.batch > 32) {
    Cut x = cut0;
    for (int b0 = 32; b0 < R.batch; b0 += 32) cut_rows(row_steps(b0 + lane, false), per, x, x.total, x.total_cut);
    pieces_all = x.total;
  }

  // the 32 rows of the piece: a CTA's pieces only go on, so they are looked for from the last one's
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

    float o[NB][DH / 16][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int z = 0; z < NB; ++z) {
#pragma unroll
      for (int i = 0; i < DH / 16; ++i) o[z][i][0] = o[z][i][1] = o[z][i][2] = o[z][i][3] = 0.f;
      m[z][0] = m[z][1] = -INFINITY;
      l[z][0] = l[z][1] = 0.f;
    }

    const uint32_t ring_a = smem_u32(smem + warp * S::kRing);
    const int first = t0 + warp * kTok;
    const uint8_t* kb = static_cast<const uint8_t*>(a.pages.k) + h * DH;
    const uint8_t* vb = static_cast<const uint8_t*>(a.pages.v) + h * DH;
    const int64_t tok_stride = (int64_t)a.n_kv * DH;

    // This lane's block of 16 tokens of the step that is looked up next; its slot, or -1: past the range, or a page
    // outside the pool. A step is kStep tokens on from the last, so its page is found without a division.
    const int ps = a.pages.page_size, step_pages = S::kStep / ps, step_rest = S::kStep % ps;
    int look_t = first + lane * kKv8Block;
    int look_pg = R.page_table ? look_t / ps : 0, look_off = look_t - look_pg * ps;
    const int32_t* table = R.page_table ? R.page_table + (int64_t)b * R.table_pages : nullptr;
    auto slot_next = [&]() -> int {
      int slot = -1;
      if (lane < kBlocks && look_t < t1) {
        int page = b;
        if (table) page = look_pg < R.table_pages ? table[look_pg] : -1;
        if (page >= 0 && page < a.pages.n_pages) slot = page * ps + look_off;
        else record_error(a.err, kCodeDevice, kErrPage, look_t, b);
      }
      look_t += S::kStep;
      if (table) {
        look_pg += step_pages;
        look_off += step_rest;
        if (look_off >= ps) {
          look_off -= ps;
          ++look_pg;
        }
      } else {
        look_off += S::kStep;
      }
      return slot;
    };
    // a lane copies the 16-byte chunk `ch` of every kRows-th row, from `row0` on: all places are constants apart
    constexpr int kCh = DH / 16, kRows = 32 / kCh, kPer = kKv8Block / kRows;
    const int row0_l = lane / kCh, ch = lane % kCh;
    const int64_t lane_off = (int64_t)row0_l * tok_stride + ch * 16, row_off = kRows * tok_stride;
    const uint32_t k_to = key_at<DH>(row0_l, ch), v_to = value_at<DH>(row0_l, ch);
    auto load = [&](int stage, int rest, int slot) {                 // rest: tokens of the step that are there
      if (rest > 0) {
        const uint32_t st = ring_a + stage * (2 * S::kTile);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int s = __shfl_sync(0xffffffffu, slot, i);
          const int64_t off = s < 0 ? 0 : s * tok_stride + lane_off;
          const int in = s < 0 ? 0 : rest - i * kKv8Block - row0_l;  // rows of the block that are there, those x kRows below it
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            const int row = i * kKv8Block + x * kRows;               // and row0_l
            // the chunk's exchange by the row's low bits: those of row0_l, and for rows of eight chunks bit 2 of 4 x
            const uint32_t flip = DH == 128 ? uint32_t(row & 4) << 4 : 0u;
            const int bytes = x * kRows < in ? 16 : 0;
            const int64_t o = bytes ? off + x * row_off : 0;
            cp16(st + row * DH + k_to, kb + o, bytes);
            cp16(st + S::kTile + row * DH + (v_to ^ flip), vb + o, bytes);
          }
        }
        if (lane < kBlocks) {
          const int64_t off = slot < 0 ? 0 : (int64_t)(slot / kKv8Block) * a.n_kv + h;
          cp4(smem_u32(&scales[warp][stage][0][lane]), A.k_scale + off, slot < 0 ? 0 : 4);
          cp4(smem_u32(&scales[warp][stage][1][lane]), A.v_scale + off, slot < 0 ? 0 : 4);
        }
      }
      cp_commit();
    };

    int next = slot_next();
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) {
      const int cur = next;
      next = slot_next();
      load(it, t1 - first - it * S::kStep, cur);
    }

    // Query rows as the B operand: column lane / 4 of an eight; inner index: lane % 4 has the elements [16 c + 4 w, + 4) of
    // every 64 in the product w of the four that they take, as a key's chunk gives them. Of scores and outputs a lane has
    // the columns 2 (lane % 4) and the next.
    const int r0 = lane >> 2, cp = lane & 3;
    uint32_t qf[S::kQueries ? 1 : NB][DH / 16][2];
    uint2* q_s = reinterpret_cast<uint2*>(smem + S::kOffQ) + lane;   // [NB][DH / 16][32 lanes]
    float scale[NB][2];                                              // log2(e) / sqrt(d), without the row's lift
    int vis[NB][2];                                                  // last slot the query rows see
#pragma unroll
    for (int z = 0; z < NB; ++z) {
      const int rr = z * 8 + r0, zq = S::kQueries ? 0 : z;
      const bool ok = rr < rows;
      const int head = h * a.g + rr % a.g;
      const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) +
                                                      (int64_t)(q0 + rr / a.g) * a.q_stride + head * DH + cp * 16);
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        const uint2 v = ok ? p[k / 4 * 16 + k % 4] : make_uint2(0u, 0u);
        qf[zq][k][0] = v.x;
        qf[zq][k][1] = v.y;
      }
      float lift = 1.f;
      if constexpr (BF16) {
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int k = 0; k < DH / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&qf[zq][k][e])));
        float big = fmaxf(__low2float(top), __high2float(top));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        lift = lift_of(big);
#pragma unroll
        for (int k = 0; k < DH / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) qf[zq][k][e] = lifted(qf[zq][k][e], lift);
      }
      if constexpr (S::kQueries) {
        if (warp == z % kWarps) {
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) q_s[(z * (DH / 16) + k) * 32] = make_uint2(qf[0][k][0], qf[0][k][1]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = z * 8 + 2 * cp + x;
        scale[z][x] = a.scale_log2 * (1.f / __shfl_sync(0xffffffffu, lift, (2 * cp + x) * 4));   // powers of two
        vis[z][x] = r < rows ? L - n + r / a.g : -1;
      }
    }
    if constexpr (S::kQueries) __syncthreads();
    const int vis_min = L - n;                                       // every row sees slots up to here

    int stage = 0;
    for (int tb = first; tb < t1; tb += S::kStep) {
      cp_wait<kStages - 2>();
      __syncwarp();                                                  // the stage is there, the one before it has been read
      {
        const int cur = next;
        next = slot_next();
        load(stage == 0 ? kStages - 1 : stage - 1, t1 - tb - (kStages - 1) * S::kStep, cur);
      }
      const uint32_t ks = ring_a + stage * (2 * S::kTile), vs = ks + S::kTile;
      float s[NB][kBlocks][4];                                       // of tokens r0 and r0 + 8, two query rows each
#pragma unroll
      for (int z = 0; z < NB; ++z)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) s[z][i][0] = s[z][i][1] = s[z][i][2] = s[z][i][3] = 0.f;
      // two blocks at a time: products in a row belong to different ones
#pragma unroll
      for (int i0 = 0; i0 < kBlocks; i0 += 2) {
#pragma unroll
        for (int c = 0; c < DH / 64; ++c) {
          uint4 v[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) v[i][x] = lds16(ks + key_at<DH>((i0 + i) * 16 + x * 8 + r0, c * 4 + cp));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t f[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w = k == 0 ? v[i][x].x : k == 1 ? v[i][x].y : k == 2 ? v[i][x].z : v[i][x].w;
                f[i][x] = f16_of_codes(uint16_t(w));
                f[i][2 + x] = f16_of_codes(uint16_t(w >> 16));
              }
#pragma unroll
            for (int z = 0; z < NB; ++z) {
              uint2 q;
              if constexpr (S::kQueries) q = q_s[(z * (DH / 16) + c * 4 + k) * 32];
              else q = make_uint2(qf[z][c * 4 + k][0], qf[z][c * 4 + k][1]);
#pragma unroll
              for (int i = 0; i < 2; ++i) mma<false>(s[z][i0 + i], f[i], q.x, q.y);
            }
          }
        }
      }
      if (tb + kTok > t1 || tb + kTok - 1 > vis_min) {
#pragma unroll
        for (int z = 0; z < NB; ++z)
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = tb + i * 16 + (e >> 1) * 8 + r0;
              if (t >= t1 || t > vis[z][e & 1]) s[z][i][e] = -INFINITY;
            }
      }
      float k_s[kBlocks], v_log[kBlocks], v_inv[kBlocks];
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        k_s[i] = scale_or_one(scales[warp][stage][0][i]);
        const float y = scale_or_one(scales[warp][stage][1][i]);
        v_log[i] = lg2(y);
        v_inv[i] = rcp(y);
      }
      uint32_t pf[NB][kBlocks][2];
#pragma unroll
      for (int z = 0; z < NB; ++z) {
        float al[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
            mx = fmaxf(mx, fmaf(fmaxf(s[z][i][x], s[z][i][2 + x]), factor_of<BF16>(scale[z][x], k_s[i]), v_log[i]));
#pragma unroll
          for (int e = 4; e < 32; e *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
          const float mn = fmaxf(m[z][x], softmax_base<false>(mx, kLift));
          const float base = mn == -INFINITY ? 0.f : mn;             // nothing seen yet: every weight is 2^-inf = 0
          al[x] = ex2(m[z][x] - base);
          m[z][x] = mn;
          l[z][x] *= al[x];
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            const float c = factor_of<BF16>(scale[z][x], k_s[i]), d = v_log[i] - base;
            s[z][i][x] = ex2(fmaf(s[z][i][x], c, d));
            s[z][i][2 + x] = ex2(fmaf(s[z][i][2 + x], c, d));
            l[z][x] = fmaf(s[z][i][x] + s[z][i][2 + x], v_inv[i], l[z][x]);
          }
        }
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          pf[z][i][0] = turned(pack2<false>(s[z][i][0], s[z][i][1]));
          pf[z][i][1] = turned(pack2<false>(s[z][i][2], s[z][i][3]));
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            o[z][i][0] *= al[0];
            o[z][i][1] *= al[1];
            o[z][i][2] *= al[0];
            o[z][i][3] *= al[1];
          }
        }
      }
      const int vr = ((lane >> 3) & 1) * 8 + (lane & 7), vc = lane >> 4;
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) {
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          uint32_t f[4];                                             // tokens 0 - 7 and 8 - 15 of two chunks
          ldsm4t(f, vs + value_at<DH>(k * 16 + vr, 2 * i + vc));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            // two tokens of an even and an odd column, parted: the even columns are a product's rows 0 to 7, the odd 8 to 15
            const uint32_t b0 = __byte_perm(f[2 * y], 0u, 0x3120), b1 = __byte_perm(f[2 * y + 1], 0u, 0x3120);
            const uint32_t v[4] = {f16_of_codes(uint16_t(b0)), f16_of_codes(uint16_t(b0 >> 16)),
                                   f16_of_codes(uint16_t(b1)), f16_of_codes(uint16_t(b1 >> 16))};
#pragma unroll
            for (int z = 0; z < NB; ++z) mma<false>(o[z][2 * i + y], v, pf[z][k][0], pf[z][k][1]);
          }
        }
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncthreads();

    // join the warps: each leaves its output rows in the (now free) ring
    float* ob = reinterpret_cast<float*>(smem) + warp * S::kRows * DH;
#pragma unroll
    for (int z = 0; z < NB; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = z * 8 + 2 * cp + x;
#pragma unroll
        for (int e = 4; e < 32; e *= 2) l[z][x] += __shfl_xor_sync(0xffffffffu, l[z][x], e);
        if (r0 == 0) X.ml[warp][r] = make_float2(m[z][x], l[z][x]);
#pragma unroll
        for (int i = 0; i < DH / 16; ++i)
          *reinterpret_cast<float2*>(ob + r * DH + i * 16 + 2 * r0) = make_float2(o[z][i][x], o[z][i][2 + x]);
      }
    __syncthreads();
    finish_piece<DH, BF16>(a, X, smem, q0, rows, h, np, piece, first_slot);
    __syncthreads();                                                 // the joins' space becomes the ring again
  }
}

template <int DH, bool BF16, int NB> cudaError_t prepare_few() {
  return cudaFuncSetAttribute(kv8_attend_few_kernel<DH, BF16, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Sm<DH, NB>::kBytes);
}
template <int DH, bool BF16> cudaError_t prepare_all() {
  cudaError_t e = prepare_few<DH, BF16, 1>();
  if (e == cudaSuccess) e = prepare_few<DH, BF16, 2>();
  if (e == cudaSuccess) e = prepare_few<DH, BF16, 3>();
  return e;
}
template <int DH, bool BF16, int NB> cudaError_t launch_few(Kv8AttendArgs A, int sm_count, cudaStream_t st) {
  using S = Sm<DH, NB>;
  KvAttendArgs& a = A.a;
  // the cut aims at the CTAs that the GPU holds; no more are launched than the rows' bounds give steps
  a.ctas = S::kCtas * sm_count < kKvFewMostCtas ? S::kCtas * sm_count : kKvFewMostCtas;
  const int64_t steps = (((int64_t)a.rows.max_kv_len + S::kStep - 1) / S::kStep + 1) * a.rows.batch * a.n_kv;
  const int grid = steps < a.ctas ? (int)steps : a.ctas;
  return launch_early(kv8_attend_few_kernel<DH, BF16, NB>, dim3(grid), kWarps * 32, S::kBytes, st, A);
}
template <int DH, bool BF16> cudaError_t launch_rows(const Kv8AttendArgs& A, int sm_count, cudaStream_t st) {
  switch ((A.a.rows.max_new * A.a.g + 7) / 8) {
    case 0:
    case 1: return launch_few<DH, BF16, 1>(A, sm_count, st);
    case 2: return launch_few<DH, BF16, 2>(A, sm_count, st);
    default: return launch_few<DH, BF16, 3>(A, sm_count, st);
  }
}

}  // namespace

cudaError_t prepare_kv8_attend_few(int head_dim, bool bf16) {
  if (head_dim == 128) return bf16 ? prepare_all<128, true>() : prepare_all<128, false>();
  return bf16 ? prepare_all<64, true>() : prepare_all<64, false>();
}

cudaError_t launch_kv8_attend_few(const Kv8AttendArgs& A, int sm_count, cudaStream_t st) {
  if (A.a.head_dim == 128) return A.a.bf16 ? launch_rows<128, true>(A, sm_count, st) : launch_rows<128, false>(A, sm_count, st);
  return A.a.bf16 ? launch_rows<64, true>(A, sm_count, st) : launch_rows<64, false>(A, sm_count, st);
}

}  // namespace palu
