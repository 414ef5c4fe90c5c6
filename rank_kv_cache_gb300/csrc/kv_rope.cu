// Norm and rotation of queries and keys, and the append of rotated keys and values into a paged
// KV cache, in one pass.
//
// For every head vector x of a token at position p:
//   y = R(p) (x * rsqrt(mean(x^2) + eps) * w),   R rotates the pairs (j, j + d/2) by p theta^(-2j/d).
// Without weights the norm is left out; values are copied. All arithmetic is fp32 from the inputs
// as stored; each output is rounded once, to the pages' type.
//
// Bound: HBM. Each input is read once and each output written once, with 16-byte accesses. A lane
// holds elements [8j, 8j + 8) and [d/2 + 8j, d/2 + 8j + 8) of a head, so both halves of its eight
// pairs are its own: the rotation needs no shuffle, the norm's sum three (d = 128) or two. d / 16
// lanes make a head, and a warp takes 4 (d = 128) or 8 heads at once. The angles of a token are the
// same for all of its heads: a warp computes its lanes' eight sines and cosines once and walks over
// the token's heads with them, the next heads' loads under way (the first ones' while it looks up the
// token's place). Phases are 64-bit fractions of a turn, so far positions keep theirs. The arithmetic
// is packed two fp32 to an instruction: unpacked it was bound by issue.
//
// Measured on a GB300: 16384 tokens of 32 + 8 heads of 128, bf16, normed: 58 us, 5800 GB/s, as a
// plain copy of the same bytes (57.3 us); 4096 19.4 us, 4350 GB/s; 512 8 us. Four prompts of 12831 tokens
// appended, with the queries: 59 us, 5360 GB/s; 4096 tokens 23.7. 8192 tokens in fp32: 55 us, 6090 GB/s.
// Eight tokens of 32 + 32 heads: 2.6 us, one launch.
#include "kv_vec.cuh"

namespace palu {
namespace {

constexpr int kThreads = 128;

// Row of packed token t: the first that ends behind it (batch: none does), so that a row out of order behind it changes
// nothing. Warp-wide: 32 row ends a step.
__device__ __forceinline__ int row_of_token(const KvRows& r, int t) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < r.batch; base += 32) {
    const int i = base + lane;
    const unsigned m = __ballot_sync(0xffffffffu, i < r.batch && r.row_start[i + 1] > t);
    if (m) return base + __ffs(m) - 1;
  }
  return r.batch;
}

// Records what the attention would of the rows: bounds that do not hold, a row_start that decreases. A warp of its own
// does it, beside those of the tokens.
__device__ __noinline__ void check_rows(const KvRopeArgs& a) {
  for (int b = threadIdx.x & 31; b < a.rows.batch; b += 32) {
    int q0, n, L;
    unsigned bad;
    kv_row(a.rows, b, q0, n, L, bad);
    if (bad) record_error(a.err, kCodeDevice, bad, b, b);
  }
}

template <typename TI, typename TO, int DH>
__global__ void __launch_bounds__(kThreads) kv_rope_kernel(const KvRopeArgs a, const __grid_constant__ KvFreq f,
                                                           int parts, int chunks_per_part) {
  constexpr int kLanes = DH / 16;          // lanes of a head
  constexpr int kHeads = 32 / kLanes;      // heads a warp takes at once: a chunk, of one side (queries, keys or values)
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31, j = lane % kLanes, hl = lane / kLanes;
  // the same for the warp, and told so
  const unsigned unit = __shfl_sync(0xffffffffu, blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), 0);
  const int t = int(unit / unsigned(parts)), part = int(unit % unsigned(parts));
  if (t >= a.n_tokens) {
    if (a.append && unit == unsigned(a.n_tokens) * unsigned(parts)) check_rows(a);
    return;
  }
  const int nq = (a.heads[0] + kHeads - 1) / kHeads, nk = (a.heads[1] + kHeads - 1) / kHeads;   // chunks
  const int c0 = part * chunks_per_part, c1 = min(c0 + chunks_per_part, nq + nk + (a.heads[2] + kHeads - 1) / kHeads);

  auto side_of = [&](int c) { return c < nq ? 0 : c < nq + nk ? 1 : 2; };
  auto head_of = [&](int c, int side) { return (c - (side == 0 ? 0 : side == 1 ? nq : nq + nk)) * kHeads + hl; };
  Vec8<TI> lo, hi;                         // the chunk that comes next
  auto load = [&](int c) {
    const int side = side_of(c), h = head_of(c, side);
    if (c < c1 && h < a.heads[side]) {
      const TI* p = static_cast<const TI*>(a.src[side]) + (int64_t)t * a.src_stride[side] + (h * DH + j * 8);
      lo.load(p, 0);
      hi.load(p, DH / 2);
    }
  };
  load(c0);                                // under way while the token's place and angles are found

  // the token's position and, for the append, its slot in the pages
  int pos = 0;
  int64_t slot = -1;
  if (a.append) {
    const int b = row_of_token(a.rows, t);
    if (b >= a.rows.batch) return;         // behind the last row
    const int start = a.rows.row_start[b];
    if (t < start) return;                 // in front of the first row
    pos = a.rows.kv_len[b] - a.rows.row_start[b + 1] + t;
    if (pos >= 0) slot = kv_slot(a.rows, a.pages, b, pos);
    if (slot < 0 && part == 0 && lane == 0) record_error(a.err, kCodeDevice, kErrSlot, pos, b);
  }
  if (a.positions) pos = a.positions[t];
  uint64_t cs[4], sn[4];
  // values alone need no angles
  if (a.rotate && c0 < nq + nk) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float c[2], s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // turns * 2^64, in [-1/2, 1/2); half turns: * 2^-63
        const int64_t phase = (int64_t)(uint64_t((int64_t)pos) * f.turn[j * 8 + 2 * e + k]);
        sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &s[k], &c[k]);
      }
      cs[e] = pair(c[0], c[1]);
      sn[e] = pair(s[0], s[1]);
    }
  }

  uint64_t gl[4], gu[4];                   // this lane's norm weights of the side
  const void* w = nullptr;
  TO* dst = nullptr;
  bool rotate = false;
  for (int c = c0; c < c1; ++c) {
    const Vec8<TI> xl = lo, xh = hi;
    load(c + 1);
    const int side = side_of(c), h = head_of(c, side);
    if (c == c0 || c == nq || c == nq + nk) {   // the side's first chunk here: its weights and its place
      w = side < 2 ? a.w[side] : nullptr;
      if (w) {
        Vec8<TI> g;
        g.load(w, j * 8);
        g.get(gl);
        g.load(w, j * 8 + DH / 2);
        g.get(gu);
      }
      rotate = a.rotate && side < 2;
      if (side == 0 || !a.append)
        dst = static_cast<TO*>(a.dst[side]) + (int64_t)t * a.dst_stride[side];
      else
        dst = slot < 0 ? nullptr : static_cast<TO*>(side == 1 ? a.pages.k : a.pages.v) + slot * a.heads[1] * DH;
    }
    uint64_t l[4], u[4];
    xl.get(l);
    xh.get(u);
    if (w) {
      uint64_t ss2 = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss2 = fma2(l[e], l[e], fma2(u[e], u[e], ss2));
      const float2 s = unpair(ss2);
      float ss = s.x + s.y;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * (1.f / DH) + a.eps);
      const uint64_t r2 = pair(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[e] = mul2(mul2(l[e], r2), gl[e]);
        u[e] = mul2(mul2(u[e], r2), gu[e]);
      }
    }
    if (rotate) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t p = l[e], q = u[e];
        l[e] = fma2(p, cs[e], mul2(q, sn[e]) ^ 0x8000000080000000ull);
        u[e] = fma2(q, cs[e], mul2(p, sn[e]));
      }
    }
    if (h < a.heads[side] && dst) {
      Vec8<TO> y;
      y.set(l);
      y.store(dst, h * DH + j * 8);
      y.set(u);
      y.store(dst, h * DH + j * 8 + DH / 2);
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_typed(const KvRopeArgs& a, const KvFreq& f, int sm_count, cudaStream_t st) {
  const int per = a.head_dim == 128 ? 4 : 8;
  const int chunks = (a.heads[0] + per - 1) / per + (a.heads[1] + per - 1) / per + (a.heads[2] + per - 1) / per;
  // Few tokens: one chunk of heads a warp, so that the call takes one load's latency. Many: a warp
  // keeps its token's angles for all of the heads.
  int parts = chunks;
  while (parts > 1 && (int64_t)a.n_tokens * parts > (int64_t)sm_count * 64) parts = (parts + 1) / 2;
  const int cpp = (chunks + parts - 1) / parts;
  parts = (chunks + cpp - 1) / cpp;
  const int64_t units = (int64_t)a.n_tokens * parts + (a.append ? 1 : 0);   // one to check the rows
  const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32));
  if (a.head_dim == 128) return launch_early(kv_rope_kernel<TI, TO, 128>, dim3(grid), kThreads, 0, st, a, f, parts, cpp);
  return launch_early(kv_rope_kernel<TI, TO, 64>, dim3(grid), kThreads, 0, st, a, f, parts, cpp);
}

template <typename TI>
cudaError_t launch_from(const KvRopeArgs& a, const KvFreq& f, int sm_count, cudaStream_t st) {
  if (a.dtype == kF32) return launch_typed<TI, float>(a, f, sm_count, st);
  if (a.dtype == kF16) return launch_typed<TI, __half>(a, f, sm_count, st);
  return launch_typed<TI, __nv_bfloat16>(a, f, sm_count, st);
}

}  // namespace

cudaError_t launch_kv_rope(const KvRopeArgs& a, const KvFreq& f, int sm_count, cudaStream_t st) {
  if (a.n_tokens == 0 || a.heads[0] + a.heads[1] + a.heads[2] == 0) return cudaSuccess;
  if (a.x_dtype == kF32) return launch_from<float>(a, f, sm_count, st);
  if (a.x_dtype == kF16) return launch_from<__half>(a, f, sm_count, st);
  return launch_from<__nv_bfloat16>(a, f, sm_count, st);
}

}  // namespace palu
