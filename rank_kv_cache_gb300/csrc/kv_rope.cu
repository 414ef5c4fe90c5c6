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
// the token's heads with them. Phases are 64-bit fractions of a turn, so far positions lose nothing.
#include "kv.h"

namespace palu {
namespace {

constexpr int kThreads = 256;

// eight consecutive elements as floats
template <typename T> struct Vec8 {
  static __device__ __forceinline__ void load(const void* base, int64_t i, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + i);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = to_f32(e[j]);
  }
  static __device__ __forceinline__ void store(void* base, int64_t i, const float (&x)[8]) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = from_f32<T>(x[j]);
    *reinterpret_cast<uint4*>(static_cast<T*>(base) + i) = u;
  }
};
template <> struct Vec8<float> {
  static __device__ __forceinline__ void load(const void* base, int64_t i, float (&x)[8]) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* base, int64_t i, const float (&x)[8]) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Row of packed token t: the number of rows that end at or before it (row_start does not decrease).
// Warp-wide: 32 row ends a step.
__device__ __forceinline__ int row_of_token(const KvRows& r, int t) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int base = 0; base < r.batch; base += 32) {
    const int i = base + lane;
    const bool past = i < r.batch && r.row_start[i + 1] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, past);
    b += __popc(m);
    if (m != 0xffffffffu) break;
  }
  return b;
}

template <typename TI, typename TO, int DH>
__global__ void __launch_bounds__(kThreads) kv_rope_kernel(const KvRopeArgs a, const __grid_constant__ KvFreq f,
                                                           int parts, int chunks_per_part) {
  constexpr int kLanes = DH / 16;          // lanes of a head
  constexpr int kHeads = 32 / kLanes;      // heads a warp takes at once
  const int lane = threadIdx.x & 31, j = lane % kLanes, hl = lane / kLanes;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = int(unit / parts), part = int(unit % parts);
  if (t >= a.n_tokens) return;

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

  float cs[8], sn[8];
  if (a.rotate) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t phase = (int64_t)(uint64_t((int64_t)pos) * f.turn[j * 8 + e]);   // turns * 2^64, in [-1/2, 1/2)
      sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &sn[e], &cs[e]);     // half turns: * 2^-63
    }
  }

  const int nq = a.heads[0], nk = a.heads[1], total = nq + nk + a.heads[2];
  const int c1 = min((part + 1) * chunks_per_part, (total + kHeads - 1) / kHeads);
#pragma unroll 2
  for (int c = part * chunks_per_part; c < c1; ++c) {
    const int h = c * kHeads + hl;
    const int side = h < nq ? 0 : h < nq + nk ? 1 : 2;
    const int hs = h - (side == 0 ? 0 : side == 1 ? nq : nq + nk);   // head within its side
    const bool live = h < total;
    float lo[8], hi[8];
    if (live) {
      const int64_t at = (int64_t)t * a.src_stride[side] + (int64_t)hs * DH + j * 8;
      Vec8<TI>::load(a.src[side], at, lo);
      Vec8<TI>::load(a.src[side], at + DH / 2, hi);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) lo[e] = hi[e] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], ss));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!live) continue;
    if (side < 2) {
      if (a.w[side]) {
        const float r = rsqrtf(ss * (1.f / DH) + a.eps);
        float wl[8], wh[8];
        Vec8<TI>::load(a.w[side], j * 8, wl);
        Vec8<TI>::load(a.w[side], j * 8 + DH / 2, wh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] *= r * wl[e];
          hi[e] *= r * wh[e];
        }
      }
      if (a.rotate) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = lo[e], y = hi[e];
          lo[e] = x * cs[e] - y * sn[e];
          hi[e] = y * cs[e] + x * sn[e];
        }
      }
    }
    void* dst;
    int64_t at;
    if (side == 0 || !a.append) {
      dst = a.dst[side];
      at = (int64_t)t * a.dst_stride[side] + (int64_t)hs * DH + j * 8;
    } else {
      if (slot < 0) continue;
      dst = side == 1 ? a.pages.k : a.pages.v;
      at = (slot * nk + hs) * DH + j * 8;
    }
    Vec8<TO>::store(dst, at, lo);
    Vec8<TO>::store(dst, at + DH / 2, hi);
  }
}

template <typename TI, typename TO>
cudaError_t launch_typed(const KvRopeArgs& a, const KvFreq& f, int sm_count, cudaStream_t st) {
  const int per = a.head_dim == 128 ? 4 : 8;
  const int chunks = (a.heads[0] + a.heads[1] + a.heads[2] + per - 1) / per;
  // Few tokens: one chunk of heads a warp, so that the call takes one load's latency. Many: a warp
  // keeps its token's angles for all of the heads.
  int parts = chunks;
  while (parts > 1 && (int64_t)a.n_tokens * parts > (int64_t)sm_count * 64) parts = (parts + 1) / 2;
  const int cpp = (chunks + parts - 1) / parts;
  parts = (chunks + cpp - 1) / cpp;
  const int64_t units = (int64_t)a.n_tokens * parts;
  const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32));
  if (a.head_dim == 128)
    kv_rope_kernel<TI, TO, 128><<<grid, kThreads, 0, st>>>(a, f, parts, cpp);
  else
    kv_rope_kernel<TI, TO, 64><<<grid, kThreads, 0, st>>>(a, f, parts, cpp);
  return cudaGetLastError();
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
