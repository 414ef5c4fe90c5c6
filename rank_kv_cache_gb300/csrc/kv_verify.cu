// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
//   a = the first draft i with u_i q_i(x_i) >= p_i(x_i) (or all of them);  w = max(p_a - q_a, 0), or p_a where every draft
//   was accepted, or where that is zero;  token = min { v : sum_{j <= v} w_j > u sum_j w_j }.
//
// The comparison of a draft is exact (the product of two fp32 numbers with its rounding error). A token is drawn from sums of
// up to 2^20 numbers, of which fp32 would misplace about vocab 2^-24 of the draws: every sum is an unevaluated one of two
// fp32 numbers (Knuth's two-sum), to which a difference p - q with its rounding error (exact for p >= q >= 0) is added;
// 48 bits misplace about vocab 2^-46. fp64 would be bound by that unit: an instruction of a warp takes it 64 cycles.
//
// Bound: HBM, one target and one draft row of each batch row. A cluster of 1 to 8 CTAs takes a row; a warp a segment of
// 512 values, a lane 16 of them in four loads (64 rows of 131072 tokens, fp32: 17 us, 3.9 TB/s of 6.8, of which the drafts'
// look-ups, the exchange and the second look take 5; four rows of 32000 7.5 us in a graph). The CTAs exchange their sums
// through distributed shared memory; the one that holds the draw finds the segment by its running sums, and one warp reads
// that segment again (from L2) for the token.
#include <cooperative_groups.h>

#include "kv8.h"

namespace palu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSeg = 512, kVec = 4, kSteps = kSeg / (32 * kVec);   // values of a segment, of a lane's load; loads
constexpr int kMostCtas = 8, kCtas = 4;                            // of a cluster; of an SM

// the cluster's CTAs have all started: before that their shared memory is not written
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// hi + lo, the second at most half a step of the first
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)), rest));
    hi = s;
  }
  __device__ __forceinline__ void carry() {
    const float s = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(s, hi));
    hi = s;
  }
  __device__ __forceinline__ Sum plus(const Sum& o) const {
    Sum r = *this;
    r.add(o.hi, o.lo);
    r.carry();
    return r;
  }
  __device__ __forceinline__ Sum times(float u) const {
    Sum r;
    r.hi = __fmul_rn(hi, u);
    r.lo = __fmaf_rn(lo, u, __fmaf_rn(hi, u, -r.hi));
    r.carry();
    return r;
  }
  __device__ __forceinline__ bool over(const Sum& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};
// two such sums, whose numbers are added by packed instructions
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return fma2(b, pair(-1.f, -1.f), a); }
struct Sum2 {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t x, uint64_t rest) {
    const uint64_t s = add2(hi, x), b = sub2(s, hi);
    lo = add2(lo, add2(add2(sub2(hi, sub2(s, b)), sub2(x, b)), rest));
    hi = s;
  }
  __device__ __forceinline__ Sum both() const {
    const float2 h = unpair(hi), l = unpair(lo);
    Sum r{h.x, l.x};
    r.add(h.y, l.y);
    return r;
  }
};
__device__ __forceinline__ Sum shfl(const Sum& s, int lane) {
  return Sum{__shfl_sync(0xffffffffu, s.hi, lane), __shfl_sync(0xffffffffu, s.lo, lane)};
}
// sums of this and the lanes below
__device__ __forceinline__ Sum running(Sum s) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum z{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
    if ((threadIdx.x & 31) >= o) s = s.plus(z);
  }
  return s;
}
// a random number as one of [0, 1): what is not below 1, NaN too, as 1 - 2^-24
__device__ __forceinline__ float uniform_of(float u) { return u < 1.f ? fmaxf(u, 0.f) : 0.99999994f; }
// u q < p
__device__ __forceinline__ bool below_p(float u, float q, float p) {
  const float x = __fmul_rn(u, q);
  if (x < 1e-20f) return double(u) * double(q) < double(p);   // the error of so small a product might be cut off
  return x < p || (x == p && __fmaf_rn(u, q, -x) < 0.f);
}

constexpr int kWide = 1;               // both rows' loads are aligned
constexpr int kUp = 2, kDown = 4;      // weights are lifted by 2^100, lowered by 2^32
// What the token is drawn from, of a lane's values of a segment: max(p - q, 0) as a difference and its rounding error.
struct Weights {
  float d[kSteps][kVec], e[kSteps][kVec];
};
template <typename T> struct Source {
  const T* p;
  const T* q;        // nullptr: none
  int certain;       // a draft that was certain: its weight is 0 (or -1)
  int vocab;
  int flags;         // kWide, and of kUp and kDown one for sums outside the range

  template <bool WIDE> __device__ __forceinline__ void row(float (&x)[kSteps][kVec], const T* r, int v) const {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int at = v + k * 32 * kVec;
      if constexpr (WIDE) {
        if constexpr (sizeof(T) == 4) {
          const float4 f = *reinterpret_cast<const float4*>(r + at);
          x[k][0] = f.x, x[k][1] = f.y, x[k][2] = f.z, x[k][3] = f.w;
        } else {
          const uint2 f = *reinterpret_cast<const uint2*>(r + at);
          const T* e = reinterpret_cast<const T*>(&f);
#pragma unroll
          for (int i = 0; i < kVec; ++i) x[k][i] = to_f32(e[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[k][i] = at + i < vocab ? to_f32(r[at + i]) : 0.f;
      }
    }
  }
  // A lane's values of the segment at v0: 4 at v0 + 4 lane, and every 128 on. Whole segments of aligned rows come without a
  // branch between the loads, so that all are under way at once.
  __device__ __forceinline__ void load(Weights& w, int v0) const {
    const int v = v0 + (threadIdx.x & 31) * kVec;
    if ((flags & kWide) && v0 + kSeg <= vocab) {
      row<true>(w.d, p, v);
      if (q) row<true>(w.e, q, v);
    } else {
      row<false>(w.d, p, v);
      if (q) row<false>(w.e, q, v);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        // NaN: 0. What q is above p does not count: both results are then 0.
        const float x0 = fmaxf(w.d[k][i], 0.f), x1 = fmaxf(w.d[k][i + 1], 0.f);
        const float y0 = q ? fminf(fmaxf(w.e[k][i], 0.f), x0) : 0.f, y1 = q ? fminf(fmaxf(w.e[k][i + 1], 0.f), x1) : 0.f;
        const uint64_t x = pair(x0, x1), y = pair(y0, y1), d = sub2(x, y);
        const float2 d2 = unpair(d), e2 = unpair(sub2(sub2(x, d), y));
        w.d[k][i] = d2.x, w.d[k][i + 1] = d2.y;
        w.e[k][i] = e2.x, w.e[k][i + 1] = e2.y;
      }
    if (unsigned(certain - v0) < unsigned(kSeg) || flags >= kUp) {
      // a rejected draft's p is below its 1, and its rounding error is 0, as there is no q
      const float lift = flags < kUp ? 1.f : flags & kUp ? 0x1p100f : 0x1p-32f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          w.d[k][i] = v + k * 32 * kVec + i == certain ? 0.f : w.d[k][i] * lift;
          w.e[k][i] *= lift;
        }
    }
  }
};

template <typename T> __global__ void __launch_bounds__(kThreads, kCtas) kv_verify_kernel(const KvVerifyArgs a) {
  extern __shared__ __align__(16) Sum seg[];            // sums of the CTA's segments
  __shared__ float2 part[kMostCtas];                    // sums of the cluster's CTAs
  __shared__ int taken_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int b = blockIdx.x / ctas;
  cluster_arrive();
  grid_wait();
  grid_release();

  // the row's drafts; the first 32 come beside the row's bounds
  const int32_t* drafts = a.draft_tokens + (int64_t)b * a.max_draft;
  const float* u = a.uniforms + (int64_t)b * (a.max_draft + 1);
  const int x0 = lane < a.max_draft ? drafts[lane] : 0;
  const float u0 = lane < a.max_draft ? u[lane] : 0.f;
  const float u1 = uniform_of(u[a.max_draft]);
  const int start = a.row_start[b], end = a.row_start[b + 1];
  const bool row_ok = start >= 0 && end >= start && end <= a.n_tokens;
  const int brought = row_ok ? end - start : 0;         // tokens that are in the cached length
  if (rank == 0 && tid == 0 && (!row_ok || brought - 1 > a.max_draft)) record_error(a.err, kCodeDevice, kErrRows, b, b);
  const int n = min(brought, a.max_draft + 1);
  int32_t* out = a.tokens + (int64_t)b * (a.max_draft + 1);
  const T* target = static_cast<const T*>(a.target) + (int64_t)start * a.target_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + (int64_t)b * a.max_draft * a.draft_stride : nullptr;
  if (n == 0) {                                         // the whole cluster
    cluster_wait();
    if (rank == 0) {
      for (int i = tid; i <= a.max_draft; i += kThreads) out[i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        if (a.kv_len_out) a.kv_len_out[b] = a.kv_len[b];
      }
    }
    return;
  }
  if (warp == 0) {
    int taken = n - 1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool no = false;
      if (i < n - 1) {
        const int x = i0 == 0 ? x0 : drafts[i];
        no = x < 0 || x >= a.vocab;
        if (no) {
          if (rank == 0) record_error(a.err, kCodeDevice, kErrToken, x, b);
        } else {
          const float p = fmaxf(to_f32(target[(int64_t)i * a.target_stride + x]), 0.f);
          const float q = draft ? fmaxf(to_f32(draft[(int64_t)i * a.draft_stride + x]), 0.f) : 1.f;
          no = !below_p(uniform_of(i0 == 0 ? u0 : u[i]), q, p);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, no);
      if (m) {
        taken = i0 + __ffs(m) - 1;
        break;
      }
    }
    if (lane == 0) taken_s = taken;
  }
  __syncthreads();
  cluster_wait();
  const int taken = taken_s;
  const bool rejected = taken < n - 1;
  if (rank == 0) {
    for (int i = tid; i <= a.max_draft; i += kThreads)
      if (i != taken) out[i] = i < taken ? drafts[i] : -1;
    if (tid == 0) {
      a.accepted[b] = taken;
      if (a.kv_len_out) a.kv_len_out[b] = a.kv_len[b] - (brought - 1 - taken);
    }
  }

  Source<T> src;
  src.p = target + (int64_t)taken * a.target_stride;
  src.q = rejected && draft ? draft + (int64_t)taken * a.draft_stride : nullptr;
  src.certain = rejected && !draft ? drafts[taken] : -1;
  src.vocab = a.vocab;
  src.flags = ((uintptr_t)src.p | (uintptr_t)src.q) % (kVec * sizeof(T)) == 0 ? kWide : 0;
  const int segs = (a.vocab + kSeg - 1) / kSeg, per = (segs + ctas - 1) / ctas;
  const int s0 = min(segs, rank * per), mine = min(segs, s0 + per) - s0;

  Sum total, below;
  for (;;) {
    for (int s = warp; s < mine; s += kWarps) {
      Weights w;
      src.load(w, (s0 + s) * kSeg);
      Sum2 two;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < kVec; i += 2) two.add(pair(w.d[k][i], w.d[k][i + 1]), pair(w.e[k][i], w.e[k][i + 1]));
      Sum sum = two.both();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
        sum.add(hi, lo);
      }
      sum.carry();
      if (lane == 0) seg[s] = sum;
    }
    __syncthreads();
    if (warp == 0) {                                    // in the segments' order by lanes, then over the lanes
      Sum own;
      for (int s = lane; s < mine; s += 32) own = own.plus(seg[s]);
      own = shfl(running(own), 31);
      if (lane < ctas) *cluster.map_shared_rank(&part[rank], lane) = make_float2(own.hi, own.lo);
    }
    cluster.sync();
    total = below = Sum{};
    for (int c = 0; c < ctas; ++c) {
      if (c == rank) below = total;
      total = total.plus(Sum{part[c].x, part[c].y});
    }
    if (total.hi == 0.f) {
      if (!src.q && src.certain < 0) break;
      src.q = nullptr;                                  // nothing is left of p - q: from p
      src.certain = -1;
    } else {
      // Below 2^-100 the second number's bits would fall under the least subnormal, u times the sum would round to the sum
      // itself, and nothing would exceed it; past the largest number sums are NaN. Such a row is summed anew, lifted by 2^100
      // or lowered by 2^32 (2^20 numbers are then in range, and what that rounds lies far below the sum's last bit).
      if (src.flags >= kUp || (total.hi >= 0x1p-100f && total.hi < INFINITY)) break;
      src.flags |= total.hi < 1.f ? kUp : kDown;
    }
    cluster.sync();                                     // every CTA has read the sums
  }
  if (!(total.hi > 0.f)) {
    if (rank == 0 && tid == 0) {
      out[taken] = -1;
      record_error(a.err, kCodeDevice, kErrToken, -1, b);
    }
    return;
  }
  // The draw falls to the first CTA whose running sum exceeds it; those are the same numbers in every CTA.
  const Sum t = total.times(u1);
  const Sum own{part[rank].x, part[rank].y};
  if (warp != 0 || mine == 0 || below.over(t) || !below.plus(own).over(t)) return;
  // the segment: the first whose running sum exceeds it, or by another order of rounding the last that holds anything
  Sum run = below, from = below;
  int at = -1;
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const Sum x = i0 + lane < mine ? seg[i0 + lane] : Sum{};
    const Sum y = run.plus(running(x));
    const unsigned holds = __ballot_sync(0xffffffffu, x.hi > 0.f), over = __ballot_sync(0xffffffffu, x.hi > 0.f && y.over(t));
    const int pick = over ? __ffs(over) - 1 : 31 - __clz(holds);
    if (holds) {
      at = i0 + pick;
      const Sum before = shfl(y, max(pick - 1, 0));     // what lies before the segment
      from = pick ? before : run;
    }
    if (over) break;
    run = shfl(y, 31);
  }
  // the token within it, alike
  Weights w;
  src.load(w, (s0 + at) * kSeg);
  run = from;
  int token = -1;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    Sum sum;
#pragma unroll
    for (int i = 0; i < kVec; ++i) sum.add(w.d[k][i], w.e[k][i]);
    sum.carry();
    const Sum to = run.plus(running(sum));              // behind this lane's four; before them: behind the lane below's
    Sum x{__shfl_up_sync(0xffffffffu, to.hi, 1), __shfl_up_sync(0xffffffffu, to.lo, 1)};
    if (lane == 0) x = run;
    int first = -1, last = -1;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      x.add(w.d[k][i], w.e[k][i]);
      x.carry();
      if (w.d[k][i] > 0.f) {
        last = i;
        if (first < 0 && x.over(t)) first = i;
      }
    }
    const unsigned over = __ballot_sync(0xffffffffu, first >= 0), holds = __ballot_sync(0xffffffffu, last >= 0);
    if (over) {
      const int l = __ffs(over) - 1;
      token = (s0 + at) * kSeg + k * 32 * kVec + l * kVec + __shfl_sync(0xffffffffu, first, l);
      break;
    }
    if (holds) {
      const int l = 31 - __clz(holds);
      token = (s0 + at) * kSeg + k * 32 * kVec + l * kVec + __shfl_sync(0xffffffffu, last, l);
    }
    run = shfl(to, 31);
  }
  if (lane == 0) out[taken] = token;
}

template <typename T> cudaError_t launch_typed(const KvVerifyArgs& a, int sm_count, cudaStream_t st) {
  // The row's segments are shared by 1 to 8 CTAs, of the numbers with which the GPU holds all rows' CTAs at once the least whose
  // warps take the fewest segments one after the other. One row over 131072 tokens: 7.3 us by 8 CTAs, 9.9 by 4, 15.9 by 2, 28.3
  // by one; 128 rows: 23.6 by 4, 27.0 by 2, 40.2 by one; 80 rows 18.9 by 7 against 22.3 by 4, 180 rows 30.7 by 3 against 39.4
  // by 2. 80 rows over 32000: 10.8 by 4, 12.0 by 7, two segments a warp either way.
  const int segs = (a.vocab + kSeg - 1) / kSeg;
  auto rounds = [&](int c) { return ((segs + c - 1) / c + kWarps - 1) / kWarps; };
  int ctas = kMostCtas;
  while (ctas > 1 && (int64_t)a.batch * ctas > (int64_t)sm_count * kCtas) --ctas;
  while (ctas > 1 && rounds(ctas - 1) == rounds(ctas)) --ctas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Sum) * ((segs + ctas - 1) / ctas);   // at most 16 KB
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_kv_verify(const KvVerifyArgs& a, int sm_count, cudaStream_t st) {
  if (a.dtype == kF32) return launch_typed<float>(a, sm_count, st);
  if (a.dtype == kF16) return launch_typed<__half>(a, sm_count, st);
  return launch_typed<__nv_bfloat16>(a, sm_count, st);
}

}  // namespace palu
