// Attention of few new tokens over a paged KV cache: decode steps, drafted tokens.
//
//   o = softmax(q K^T / sqrt(d)) V over slots 0 .. L - n + i of the query's row,  lse = ln sum e^s.
//
// A unit is (row, key/value head, 16 query rows): query row r = i g + j is new token i under head j of
// the g heads that share the key/value head. Bound: HBM, each cached row is read once for the whole
// group. The g heads are the rows of 16-row matrix instructions (mma.sync m16n8k16, fp32 accumulation):
// the 128-row tcgen05 shapes would leave 7/8 of their rows empty here, and the rate needed, 16 rows
// for every 4 d cached bytes, is a few per cent of what this instruction gives.
//
// A unit's cached tokens are cut into n_splits ranges, one CTA each, two CTAs an SM (so that one's start
// and join hide behind the other's stream); a CTA's four warps take 16 tokens (d = 64: 32) in turn, each
// with its own online softmax (fp32 maximum, sum and output) and its own three-stage ring of cp.async
// copies, so no barrier stands between the warps until they are joined. Rows past the end are
// written as zeros into shared memory and masked, never read. The last CTA of a unit to finish joins
// the ranges in a fixed order. The weights p are rounded to the cache's type for the product with V, as
// the matrix instruction takes it; the sum is of the unrounded p.
#include "kv.h"

namespace palu {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;

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
  static_assert(kKvFewRows * kKvFewSplits * 4 <= kBytes && kWarps * kKvFewRows * DH * 4 <= kBytes, "joins");
};

// Rows are stored with their 16-byte chunks exchanged by the row's low three bits, so that the eight
// rows of an ldmatrix fall into different banks.
template <int DH> __device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return uint32_t(row * (DH * 2) + ((chunk ^ (row & 7)) << 4));
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.n_splits;
  const int uy = blockIdx.x / a.n_splits;
  const int h = uy % a.n_kv, rt = uy / a.n_kv, b = blockIdx.y;
  const KvRows& R = a.rows;

  int q0, n, L;
  unsigned bad;
  const bool use = kv_row(R, b, q0, n, L, bad);
  if (bad && split == 0 && uy == 0 && threadIdx.x == 0) record_error(a.err, kCodeDevice, bad, b, b);
  if (!use) return;
  const int rows = min(n * a.g - rt * kKvFewRows, kKvFewRows);
  if (rows <= 0) return;
  const int i_last = (rt * kKvFewRows + rows - 1) / a.g;           // the unit's last new token
  const int seen = max(0, min(L, L - n + i_last + 1));             // cached tokens it attends to
  // the row's own ranges: n_splits at most, whole steps of the CTA
  int per = (seen + a.n_splits - 1) / a.n_splits;
  per = (per + S::kStep - 1) / S::kStep * S::kStep;
  const int ns = per > 0 ? (seen + per - 1) / per : 1;
  if (split >= ns) return;
  const int t0 = split * per, t1 = min(seen, t0 + per);

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
    const int rr = rt * kKvFewRows + r0 + 8 * x;
    const bool ok = r0 + 8 * x < rows;
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
  const int vis_min = L - n + rt * kKvFewRows / a.g;               // every row sees slots up to here

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
      const float mn = fmaxf(m[x], mx * a.scale_log2);
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
  const int64_t unit = (int64_t)b * (gridDim.x / a.n_splits) + uy;
  auto write_lse = [&](int r, float M, float Lsum) {
    const int rr = rt * kKvFewRows + r;
    if (a.lse)
      a.lse[(int64_t)(q0 + rr / a.g) * a.n_heads + h * a.g + rr % a.g] =
          Lsum == 0.f ? -INFINITY : (M + log2f(Lsum)) * 0.69314718055994531f;
  };
  auto out_at = [&](int r) -> int64_t {
    const int rr = rt * kKvFewRows + r;
    return ((int64_t)(q0 + rr / a.g) * a.n_heads + h * a.g + rr % a.g) * DH;
  };
  if (ns == 1) {
    for (int x = threadIdx.x; x < rows * (DH / 2); x += kWarps * 32) {
      const int r = x / (DH / 2), c = x % (DH / 2) * 2;
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 u = *reinterpret_cast<const float2*>(of + (w * kKvFewRows + r) * DH + c);
        v.x = fmaf(u.x, wgt[w][r], v.x);
        v.y = fmaf(u.y, wgt[w][r], v.y);
      }
      const float Lsum = tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + out_at(r) + c) = pack2<BF16>(v.x * inv, v.y * inv);
      if (c == 0) write_lse(r, tot[r].x, Lsum);
    }
    return;
  }
  float* po = a.part_o + (unit * a.n_splits + split) * kKvFewRows * DH;
  for (int x = threadIdx.x; x < rows * (DH / 2); x += kWarps * 32) {
    const int r = x / (DH / 2), c = x % (DH / 2) * 2;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 u = *reinterpret_cast<const float2*>(of + (w * kKvFewRows + r) * DH + c);
      v.x = fmaf(u.x, wgt[w][r], v.x);
      v.y = fmaf(u.y, wgt[w][r], v.y);
    }
    *reinterpret_cast<float2*>(po + r * DH + c) = v;
  }
  if (threadIdx.x < rows) a.part_ml[(unit * a.n_splits + split) * kKvFewRows + threadIdx.x] = tot[threadIdx.x];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last_cta = atomicAdd(&a.counters[unit], 1u) == unsigned(ns - 1);
  __syncthreads();
  if (!last_cta) return;
  __threadfence();
  // join the ranges, in their order
  float* wr = reinterpret_cast<float*>(smem);                       // [rows][ns] weights
  const float2* pm = a.part_ml + unit * a.n_splits * kKvFewRows;
  for (int r = warp; r < rows; r += kWarps) {
    float M = -INFINITY, Lsum = 0.f;
    for (int k = lane; k < ns; k += 32) M = fmaxf(M, __ldcg(&pm[k * kKvFewRows + r]).x);
    M = warp_max(M);
    for (int k = lane; k < ns; k += 32) {
      const float2 v = __ldcg(&pm[k * kKvFewRows + r]);
      const float x = M == -INFINITY ? 0.f : ex2(v.x - M);
      wr[r * ns + k] = x;
      Lsum = fmaf(v.y, x, Lsum);
    }
    Lsum = warp_sum(Lsum);
    if (lane == 0) tot[r] = make_float2(M, Lsum);
  }
  __syncthreads();
  const float* pb = a.part_o + unit * a.n_splits * kKvFewRows * DH;
  for (int x = threadIdx.x; x < rows * (DH / 2); x += kWarps * 32) {
    const int r = x / (DH / 2), c = x % (DH / 2) * 2;
    float2 v = make_float2(0.f, 0.f);
    for (int k = 0; k < ns; ++k) {
      const float2 u = __ldcg(reinterpret_cast<const float2*>(pb + ((int64_t)k * kKvFewRows + r) * DH + c));
      v.x = fmaf(u.x, wr[r * ns + k], v.x);
      v.y = fmaf(u.y, wr[r * ns + k], v.y);
    }
    const float Lsum = tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + out_at(r) + c) = pack2<BF16>(v.x * inv, v.y * inv);
    if (c == 0) write_lse(r, tot[r].x, Lsum);
  }
  if (threadIdx.x == 0) a.counters[unit] = 0u;
}

template <int DH, bool BF16> cudaError_t prepare_few() {
  return cudaFuncSetAttribute(kv_attend_few_kernel<DH, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Sm<DH>::kBytes);
}
template <int DH, bool BF16> cudaError_t launch_few(const KvAttendArgs& a, cudaStream_t st) {
  const int64_t tiles = ((int64_t)a.rows.max_new * a.g + kKvFewRows - 1) / kKvFewRows;
  const dim3 grid((unsigned)(tiles * a.n_kv * a.n_splits), (unsigned)a.rows.batch);
  kv_attend_few_kernel<DH, BF16><<<grid, kWarps * 32, Sm<DH>::kBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_kv_attend_few(int head_dim, bool bf16) {
  if (head_dim == 128) return bf16 ? prepare_few<128, true>() : prepare_few<128, false>();
  return bf16 ? prepare_few<64, true>() : prepare_few<64, false>();
}

cudaError_t launch_kv_attend_few(const KvAttendArgs& a, cudaStream_t st) {
  if (a.head_dim == 128) return a.bf16 ? launch_few<128, true>(a, st) : launch_few<128, false>(a, st);
  return a.bf16 ? launch_few<64, true>(a, st) : launch_few<64, false>(a, st);
}

}  // namespace palu
