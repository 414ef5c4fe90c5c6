// The plan of a step's rows and pages: admission, packed rows, page table entries from a ring of free pages, and the place
// and slot of every packed token.
//
//   pages(b) = max(0, ceil((L_b + n_b) / page) - held_b),  row_start = running sum of the admitted n_b,
//   admitted: the running sums of pages and tokens, over all rows up to b, stay within what is free.
//
// Bound: latency (a step of 64 rows moves a few KB: 4.7 us in a graph; 512 rows, 20 of them ended: 9.3). One launch, one cluster of 1 to 8 CTAs: every CTA loads the rows, one
// or four a thread, and works out the three running sums (pages taken, tokens, pages given back) for itself in shared memory;
// then the CTAs share the writes, each finding its rows by bisection of those sums. Nothing is read that
// another CTA writes: pages are read from the ring's front and written behind its end, table entries are read below
// `held` and written from there on, and what is replaced in place (lengths, held, the ring's state) is written behind a
// barrier of the cluster. A ring in which the pages given back would reach round to its front is known before the first
// write and left alone.
#include <cooperative_groups.h>

#include "kv8.h"

namespace palu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kRows = 4 * kThreads;   // rows of a chunk, at most
constexpr int kMostCtas = 8;
// Tokens and pages that a CTA writes alone: past it the work goes to a cluster. 256 rows of up to 128 new tokens take 5.6 us
// (7.2 from 4096 on, and by one CTA), 512 of 256 5.8 us (7.7 and 14.6); from 512 on, 64 rows of 128 take 5.2 us against 4.9.
constexpr int kWritesPerCta = 2048;

struct Sums {
  int64_t pages, tokens, back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.pages + b.pages, a.tokens + b.tokens, a.back + b.back};
}

// the last of the `n` ascending numbers x[0 .. n) that is <= v (x[0] is)
__device__ __forceinline__ int last_at_most(const int* x, int n, int v) {
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Shared {
  Sums warp[kWarps], most[kWarps];
  // of the chunk's rows: running sums before the row (one more: behind the last), relative to the chunk's beginning
  int tokens[kRows + 1], pages[kRows + 1], back[kRows + 1];
  int len[kRows], held[kRows];
};

// the sum of this lane's and all lower lanes' numbers
__device__ __forceinline__ Sums running(Sums s) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y{__shfl_up_sync(0xffffffffu, s.pages, o), __shfl_up_sync(0xffffffffu, s.tokens, o),
                 __shfl_up_sync(0xffffffffu, s.back, o)};
    if ((threadIdx.x & 31) >= o) s = s + y;
  }
  return s;
}
__device__ __forceinline__ Sums of_lane(const Sums& s, int lane) {
  return Sums{__shfl_sync(0xffffffffu, s.pages, lane), __shfl_sync(0xffffffffu, s.tokens, lane),
              __shfl_sync(0xffffffffu, s.back, lane)};
}

// kPer: rows of a thread
template <int kPer> __global__ void __launch_bounds__(kThreads) kv_plan_kernel(const KvPlanArgs a) {
  constexpr int kRows = kThreads * kPer;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& S = *reinterpret_cast<Shared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  grid_wait();
  grid_release();
  const int head0 = a.state[0], count0 = a.state[1];
  auto ring_at = [&](int64_t i) {      // of 0 .. n_pages, in a ring that adds up
    const int64_t x = head0 + i;
    return (int)(x < a.n_pages ? x : x - a.n_pages);
  };
  // The ring adds up: its numbers do, and the pages of all ended rows have a place in it. Else no page is taken or given back.
  auto adds_up = [&](int64_t back) {
    const bool ok = head0 >= 0 && head0 < a.n_pages && count0 >= 0 && count0 + back <= a.n_pages;
    if (!ok && rank == 0 && tid == 0)
      record_error(a.err, kCodeDevice, kErrPool, (int)min(count0 + back, (int64_t)INT32_MAX), head0);
    return ok;
  };
  auto held_right = [&](int held) { return held >= 0 && held <= a.table_pages; };
  bool ring_ok = true;                 // one chunk: from its sums
  if (a.batch > kRows) {
    int64_t back = 0;
    for (int b = tid; b < a.batch; b += kThreads) {
      const int held = a.held[b];
      if (a.fresh[b] < 0 && held_right(held)) back += held;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) back += __shfl_xor_sync(0xffffffffu, back, o);
    if (lane == 0) S.warp[warp].back = back;
    __syncthreads();
    back = 0;
    for (int w = 0; w < kWarps; ++w) back += S.warp[w].back;
    ring_ok = adds_up(back);
    __syncthreads();
  }

  Sums wanted{0, 0, 0};                // of all rows before the chunk, admitted or not
  int64_t taken = 0, tokens = 0;       // of the admitted ones
  if (rank == 0 && tid == 0) a.row_start[0] = 0;
  for (int row0 = 0; row0 < a.batch; row0 += kRows) {
    const int rows = min(kRows, a.batch - row0);
    int n[kPer], L[kPer], held[kPer];
    Sums w[kPer], run{0, 0, 0};
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int r = tid * kPer + e, b = row0 + r;
      n[e] = L[e] = held[e] = 0;
      w[e] = Sums{0, 0, 0};
      if (r < rows) {
        n[e] = a.fresh[b];
        L[e] = a.kv_len[b];
        held[e] = a.held[b];
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int r = tid * kPer + e, b = row0 + r;
      bool bad = !held_right(held[e]);
      if (n[e] < 0) {
        if (bad) n[e] = 0;
        else w[e].back = held[e];
      } else {
        const int64_t end = (int64_t)L[e] + n[e];
        bad = bad || L[e] < 0 || n[e] > a.max_new || end > a.max_kv_len || L[e] > (int64_t)held[e] * a.page_size;
        if (bad) n[e] = 0;
        if (n[e] > 0) {
          w[e].tokens = n[e];
          w[e].pages = max(0, (int)((end + a.page_size - 1) / a.page_size) - held[e]);
        }
      }
      if (bad && rank == 0) record_error(a.err, kCodeDevice, kErrRows, b, b);
      run = run + w[e];
    }
    // the running sums over the CTA
    const Sums scan = running(run);
    if (lane == 31) S.warp[warp] = scan;
    __syncthreads();
    const Sums warps = running(lane < kWarps ? S.warp[lane] : Sums{0, 0, 0});
    Sums all = of_lane(warps, 31);
    const Sums lower = of_lane(warps, max(warp - 1, 0));
    Sums before = warp ? lower : Sums{0, 0, 0};
    if (a.batch <= kRows) ring_ok = adds_up(all.back);
    if (!ring_ok) all.back = 0;
    const int count = ring_ok ? count0 : 0;
    before = Sums{before.pages + scan.pages - run.pages, before.tokens + scan.tokens - run.tokens,
                  before.back + scan.back - run.back};
    // Admission falls off once: from the first row that does not fit on. Sums of rows behind it are those of the last one
    // that fits, so that admitted tokens and pages count on from 0.
    Sums at = before;
    int most_tokens = 0, most_pages = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const Sums to = at + w[e];
      if (wanted.pages + to.pages <= count && wanted.tokens + to.tokens <= a.n_tokens) {
        most_tokens = (int)to.tokens;
        most_pages = (int)to.pages;
      } else {
        n[e] = min(n[e], 0);
      }
      at = to;
    }
    // what the chunk admits in all: the sums ascend, so the largest that fits is the last
    most_tokens = __reduce_max_sync(0xffffffffu, most_tokens);
    most_pages = __reduce_max_sync(0xffffffffu, most_pages);
    if (lane == 0) S.most[warp] = Sums{most_pages, most_tokens, 0};
    __syncthreads();
    const Sums top = lane < kWarps ? S.most[lane] : Sums{0, 0, 0};
    most_tokens = __reduce_max_sync(0xffffffffu, (int)top.tokens);
    most_pages = __reduce_max_sync(0xffffffffu, (int)top.pages);
    at = before;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int r = tid * kPer + e;
      if (r < rows) {
        S.tokens[r] = (int)min(at.tokens, (int64_t)most_tokens);
        S.pages[r] = (int)min(at.pages, (int64_t)most_pages);
        S.back[r] = ring_ok ? (int)at.back : 0;
        S.len[r] = L[e];
        S.held[r] = held[e];
      }
      at = at + w[e];
    }
    if (tid == 0) {
      S.tokens[rows] = most_tokens;
      S.pages[rows] = most_pages;
      S.back[rows] = (int)all.back;
    }
    // every CTA has read the chunk's rows: they may be replaced
    if (ctas > 1) cluster.sync();
    else __syncthreads();

    // numbers of pages and tokens reach 2^31 - 1, and a thread's last step past it: unsigned
    const unsigned step = ctas * kThreads, me = rank * kThreads + tid;
    if (rank == 0) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int r = tid * kPer + e, b = row0 + r;
        if (r >= rows) continue;
        const bool ended = n[e] < 0 && ring_ok;
        a.row_start[b + 1] = (int)tokens + S.tokens[r + 1];
        a.kv_len_out[b] = ended ? 0 : L[e] + max(n[e], 0);
        a.held_out[b] = ended ? 0 : held[e] + S.pages[r + 1] - S.pages[r];
      }
    }
    // pages taken: from the ring into the table
    for (unsigned j = me; j < (unsigned)most_pages; j += step) {
      const int r = last_at_most(S.pages, rows + 1, j);
      const int page = a.ring[ring_at(taken + j)];
      a.table[(int64_t)(row0 + r) * a.table_pages + S.held[r] + j - S.pages[r]] = page;
      if (page < 0 || page >= a.n_pages) record_error(a.err, kCodeDevice, kErrPage, page, row0 + r);
    }
    // pages given back: from the table into the ring
    for (unsigned j = me; j < (unsigned)all.back; j += step) {
      const int r = last_at_most(S.back, rows + 1, j);
      a.ring[ring_at(count + wanted.back + j)] = a.table[(int64_t)(row0 + r) * a.table_pages + j - S.back[r]];
    }
    // the tokens' places, four at a time: their pages' loads are under way together
    if (a.positions || a.slots) {
      const bool wide = tokens % 4 == 0 && (uintptr_t)a.positions % 16 == 0 && (uintptr_t)a.slots % 16 == 0;
      for (unsigned j = me * 4; j < (unsigned)most_tokens; j += step * 4) {
        const int j0 = (int)j;
        int r = last_at_most(S.tokens, rows + 1, j0);
        int pos = S.len[r] + j0 - S.tokens[r], pg = pos / a.page_size, off = pos - pg * a.page_size;
        int place[4], slot[4];
        const int32_t* from[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int more = pg - S.held[r];
          place[e] = pos;
          slot[e] = off;
          from[e] = more < 0 ? a.table + (int64_t)(row0 + r) * a.table_pages + pg : a.ring + ring_at(taken + S.pages[r] + more);
          if (most_tokens - j0 <= e + 1) continue;                // the last one's is looked up again
          if (S.tokens[r + 1] > j0 + e + 1) {
            ++pos;
            if (++off == a.page_size) {
              off = 0;
              ++pg;
            }
          } else {
            do ++r;
            while (S.tokens[r + 1] <= j0 + e + 1);
            pos = S.len[r];
            pg = pos / a.page_size;
            off = pos - pg * a.page_size;
          }
        }
        const int n = min(4, most_tokens - j0);
        if (a.slots) {
          int page[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) page[e] = *from[e];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool ok = page[e] >= 0 && page[e] < a.n_pages;
            slot[e] = ok ? page[e] * a.page_size + slot[e] : -1;
            if (!ok) record_error(a.err, kCodeDevice, kErrPage, page[e], row0);
          }
        }
        if (wide && n == 4) {
          if (a.positions) *reinterpret_cast<int4*>(a.positions + tokens + j0) = make_int4(place[0], place[1], place[2], place[3]);
          if (a.slots) *reinterpret_cast<int4*>(a.slots + tokens + j0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (e >= n) break;
            if (a.positions) a.positions[tokens + j0 + e] = place[e];
            if (a.slots) a.slots[tokens + j0 + e] = slot[e];
          }
        }
      }
    }
    tokens += most_tokens;
    taken += most_pages;
    wanted = wanted + all;
    __syncthreads();                   // the sums' space is written anew
  }
  for (int64_t t = tokens + rank * kThreads + tid; t < a.n_tokens; t += (int64_t)ctas * kThreads) {
    if (a.positions) a.positions[t] = 0;
    if (a.slots) a.slots[t] = -1;
  }
  // The state is written when every CTA has read it: they have met since.
  if (rank == 0 && tid == 0) {
    a.state_out[0] = ring_ok ? ring_at(taken) : head0;
    a.state_out[1] = ring_ok ? (int)(count0 - taken + wanted.back) : count0;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st) {
  // CTAs by what there may be to write: tokens, and the pages they can take
  const int64_t writes = (int64_t)a.n_tokens + a.n_tokens / a.page_size + a.batch;
  unsigned ctas = 1;
  while (ctas < kMostCtas && writes > (int64_t)ctas * kWritesPerCta) ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return a.batch <= kThreads ? cudaLaunchKernelEx(&cfg, kv_plan_kernel<1>, a) : cudaLaunchKernelEx(&cfg, kv_plan_kernel<4>, a);
}

}  // namespace palu
