// Norm and rotation of queries and keys, and the append of keys and values into a paged cache held in 8 bits, in one pass.
//
// As kv_rope.cu for the arithmetic up to the rotated key; then, for each head and each block of 16 slots,
//   s = 2^ceil(log2(max |y| / 448)) over the call's new tokens of the block, at least the scale of older tokens in it,
//   code = e4m3(y / s).
// s is a power of two, so y / s is exact (but for what falls under the least subnormal) and codes, being floating
// point, lose nothing against a scale of full precision: their steps follow each value's own exponent. It also keeps
// older codes whole when a block's scale grows under them: only their exponents move.
//
// A group is a row's new tokens of one block. A CTA takes the groups that begin among 16 packed tokens: one or two of a
// prompt, 16 of a decode step. It computes the sines and cosines of their tokens (31 at most) once, in shared memory;
// then a warp takes one group and head at a time. The 16 tokens' rows of a head come by cp.async while the warp works at
// the ones before them; their halves then stay in registers (16 elements of a token a lane, as in kv_rope.cu) over norm,
// rotation and the maximum to the codes. Old codes are read only where a scale grows.
//
// Bound: HBM; each input is read once and each output written once (four prompts, up to 4096 tokens of 32 + 2 x 8 heads of 128:
// 61 us, 4.7 TB/s of 6.8; one token of eight requests 4.6 us in a graph, latency). 128 threads of 128 registers, four CTAs an
// SM (of fp32 heads of 128 two, for their shared memory; the parts of a chunk are chosen as if four): with 256 threads the prompts took 104 us at 160 registers and more (one CTA), 91 at 128 (spilled). A token's angles
// are worked out a pair a thread: read by lanes from different places, the parameters' frequencies came one after another.
#include "kv8.h"
#include "kv_vec.cuh"

namespace palu {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kCtas = 4;   // CTAs of an SM
constexpr int kChunk = kKv8Block;          // packed tokens whose groups a CTA takes

struct Group {
  int t0, n;        // packed tokens
  int pos0;         // slot of the first in its row; the block begins at pos0 & ~15
  int slot0;        // its slot in the pages, or -1
};

template <int DH, int E> struct Sm {              // E: bytes of an element as it comes
  static constexpr int kHalf = DH / 2, kTokens = 2 * kChunk - 1;
  uint8_t rows[kWarps][2][kKv8Block * DH * E];    // a warp's task and its next one's
  float cs[kTokens][kHalf], sn[kTokens][kHalf];   // pairs 8 j + e of a token at (e / 4) (kHalf / 2) + 4 j + e % 4
  Group group[kChunk];
  int groups, t0, n;                              // the groups' tokens: t0 .. t0 + n - 1
};

// The first row that ends behind packed token t (batch: none does): of row ends that ascend. Warp-wide, 32 at a time.
__device__ __forceinline__ int find_row(const KvRows& r, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = r.batch;                        // among rows lo .. lo + n - 1, or lo + n
  while (n > 0) {
    const int step = (n + 31) / 32;               // each lane looks at the last row of its share
    const int i = min(lane * step + step, n) - 1;
    const unsigned m = __ballot_sync(0xffffffffu, r.row_start[lo + i + 1] > t);
    if (!m) return lo + n;
    const int k = __ffs(m) - 1;
    const int first = k * step, last = min(first + step, n) - 1;
    lo += first;
    n = last - first;                             // row lo + n ends behind t
  }
  return lo;
}

// the least k, from -64 to 64, with top <= 448 * 2^k; top = 1.f * 2^e and 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_exponent(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int k = int(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return min(64, max(-64, k));
}

// Records what the attention would of the rows: bounds that do not hold, a row_start that decreases.
__device__ __noinline__ void check_rows(const KvRopeArgs& a) {
  for (int b = threadIdx.x; b < a.rows.batch; b += kThreads) {
    int q0, n, L;
    unsigned bad;
    kv_row(a.rows, b, q0, n, L, bad);
    if (bad) record_error(a.err, kCodeDevice, bad, b, b);
  }
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

template <typename TI, typename TO, int DH>
__global__ void __launch_bounds__(kThreads, kCtas) kv8_append_kernel(const KvRopeArgs a, const Kv8Pages P,
                                                                     const __grid_constant__ KvFreq f) {
  constexpr int kLanes = DH / 16;          // lanes of a token's head
  constexpr int kTok = 32 / kLanes;        // tokens that a warp takes at once
  constexpr int kPass = kKv8Block / kTok;
  constexpr int kQuarter = DH / 4;
  constexpr int kRow = DH * sizeof(TI), kCh = kRow / 16;   // bytes and 16-byte chunks of a row
  extern __shared__ __align__(16) uint8_t smem[];
  Sm<DH, sizeof(TI)>& S = *reinterpret_cast<Sm<DH, sizeof(TI)>*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = lane % kLanes, tl = lane / kLanes;
  const KvRows& R = a.rows;
  grid_wait();
  grid_release();
  const int parts = gridDim.y, part = blockIdx.y, heads = a.heads[0] + a.heads[1] + a.heads[2];
  if ((int64_t)blockIdx.x * kChunk >= a.n_tokens) {
    if (part == 0) check_rows(a);
    return;
  }

  // the groups that begin here
  if (warp == 0) {
    const int c0 = blockIdx.x * kChunk, t = c0 + lane;
    int base = find_row(R, c0), row = R.batch;
    int e = base + lane < R.batch ? R.row_start[base + lane + 1] : INT_MAX;
    for (int i = 0; i < kChunk; ++i) {
      unsigned m;
      while (!(m = __ballot_sync(0xffffffffu, e > c0 + i))) {       // a lane past the last row ends the search
        base += 32;
        e = base + lane < R.batch ? R.row_start[base + lane + 1] : INT_MAX;
      }
      if (lane == i) row = min(base + __ffs(m) - 1, R.batch);
    }
    bool first = false;
    Group g{t, 0, 0, -1};
    if (lane < kChunk && row < R.batch && t < a.n_tokens) {
      const int start = R.row_start[row], end = min(R.row_start[row + 1], a.n_tokens);
      if (t >= start) {
        g.pos0 = R.kv_len[row] - R.row_start[row + 1] + t;
        first = t == start || (g.pos0 & (kKv8Block - 1)) == 0;
        if (first) {
          g.n = min(end - t, kKv8Block - (g.pos0 & (kKv8Block - 1)));
          if (g.pos0 >= 0) g.slot0 = (int)kv_slot(R, P.codes, row, g.pos0);
          if (g.slot0 < 0 && part == 0) record_error(a.err, kCodeDevice, kErrSlot, g.pos0, row);
        }
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (first) S.group[__popc(m & ((1u << lane) - 1))] = g;
    const int lead = m ? __ffs(m) - 1 : 0, last = m ? 31 - __clz(m) : 0;
    const int end = __shfl_sync(0xffffffffu, t + g.n, last);
    if (lane == 0) {
      S.groups = __popc(m);
      S.t0 = c0 + lead;
      S.n = m ? end - c0 - lead : 0;
    }
  }
  __syncthreads();
  const int t0 = S.t0, tasks = S.groups * heads;
  // a task: head h of a side (queries, keys, values) of a group
  auto side_of = [&](int task, int& h) {
    h = task % heads;
    const int side = h < a.heads[0] ? 0 : h < a.heads[0] + a.heads[1] ? 1 : 2;
    h -= side == 0 ? 0 : side == 1 ? a.heads[0] : a.heads[0] + a.heads[1];
    return side;
  };
  // this CTA's tasks lie in a row, so that few groups' angles serve them
  const int per = (tasks + parts - 1) / parts, first = part * per, end = min(tasks, first + per);
  if (first >= end) return;
  auto fetch = [&](int task, int stage) {
    if (task < end) {
      const Group& g = S.group[task / heads];
      int h;
      const int side = side_of(task, h), n = g.n;
      const void* src = side == 0 ? a.src[0] : side == 1 ? a.src[1] : a.src[2];
      const int64_t pitch = (side == 0 ? a.src_stride[0] : side == 1 ? a.src_stride[1] : a.src_stride[2]) * (int64_t)sizeof(TI);
      const uint8_t* x = static_cast<const uint8_t*>(src) + g.t0 * pitch + h * kRow;
#pragma unroll
      for (int i = 0; i < kKv8Block * kCh / 32; ++i) {
        const int tok = (i * 32 + lane) / kCh, c = (i * 32 + lane) % kCh;
        if (tok < n) cp16(&S.rows[warp][stage][tok * kRow + c * 16], x + tok * pitch + c * 16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int task = first + warp, stage = 0;
  fetch(task, 0);                                  // under way while the angles are computed

  if (a.rotate) {
    const int g0 = first / heads, g1 = (end - 1) / heads;
    const int from = S.group[g0].t0 - t0, n = S.group[g1].t0 + S.group[g1].n - t0 - from;
    const int k = tid % (DH / 2);                  // this thread's pair: lanes that read different parameters take turns
    const uint64_t turn = f.turn[k];
    for (int tok = from + tid / (DH / 2); tok < from + n; tok += kThreads / (DH / 2)) {
      int pos;
      if (a.positions) {
        pos = a.positions[t0 + tok];
      } else {
        int g = g0;                                // the group that holds the token: they are in order
        while (g < g1 && S.group[g + 1].t0 <= t0 + tok) ++g;
        pos = S.group[g].pos0 + t0 + tok - S.group[g].t0;
      }
      // turns * 2^64, in [-1/2, 1/2); half turns: * 2^-63
      const int64_t phase = (int64_t)(uint64_t((int64_t)pos) * turn);
      const int at = (k & 4) / 4 * kQuarter + k / 8 * 4 + (k & 3);
      sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &S.sn[tok][at], &S.cs[tok][at]);
    }
    __syncthreads();
  }

  for (; task < end; task += kWarps, stage ^= 1) {
    const Group g = S.group[task / heads];
    int h;
    const int side = side_of(task, h);
    __syncwarp();                                  // the other stage has been read
    fetch(task + kWarps, stage ^ 1);
    const TI* rows = reinterpret_cast<const TI*>(S.rows[warp][stage]) + j * 8;
    const int64_t block = g.slot0 < 0 ? 0 : g.slot0 / kKv8Block;
    const int older = g.pos0 & (kKv8Block - 1);    // older tokens of the block
    float* scale = side == 0 ? nullptr : (side == 1 ? P.scale[0] : P.scale[1]) + block * a.heads[1] + h;
    float was = 0.f;
    if (side != 0 && g.slot0 >= 0 && older > 0) was = *scale;
    uint64_t gl[4], gu[4];                         // this lane's norm weights
    const void* w = side == 0 ? a.w[0] : side == 1 ? a.w[1] : nullptr;
    if (w) {
      Vec8<TI> v;
      v.load(w, j * 8);
      v.get(gl);
      v.load(w, j * 8 + DH / 2);
      v.get(gu);
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    uint64_t l[kPass][4], u[kPass][4];
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int tok = p * kTok + tl;
      if (p * kTok >= g.n) break;
      Vec8<TI> x;
      x.load(rows, tok * DH);
      x.get(l[p]);
      x.load(rows, tok * DH + DH / 2);
      x.get(u[p]);
      if (w) {
        uint64_t ss2 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss2 = fma2(l[p][e], l[p][e], fma2(u[p][e], u[p][e], ss2));
        const float2 s = unpair(ss2);
        float ss = s.x + s.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / DH) + a.eps);
        const uint64_t r2 = pair(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[p][e] = mul2(mul2(l[p][e], r2), gl[e]);
          u[p][e] = mul2(mul2(u[p][e], r2), gu[e]);
        }
      }
      if (a.rotate && side < 2) {
        const int at = min(g.t0 - t0 + tok, S.n - 1);
        const uint64_t* cp = reinterpret_cast<const uint64_t*>(S.cs[at]);
        const uint64_t* sp = reinterpret_cast<const uint64_t*>(S.sn[at]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e / 2 * (kQuarter / 2) + j * 2 + e % 2;
          const uint64_t p0 = l[p][e], p1 = u[p][e], cs = cp[i], sn = sp[i];
          l[p][e] = fma2(p0, cs, mul2(p1, sn) ^ 0x8000000080000000ull);
          u[p][e] = fma2(p1, cs, mul2(p0, sn));
        }
      }
      if (side == 0) {
        if (tok < g.n) {
          TO* dst = static_cast<TO*>(a.dst[0]) + (int64_t)(g.t0 + tok) * a.dst_stride[0];
          Vec8<TO> y;
          y.set(l[p]);
          y.store(dst, h * DH + j * 8);
          y.set(u[p]);
          y.store(dst, h * DH + j * 8 + DH / 2);
        }
      } else if (tok < g.n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = unpair(l[p][e]), z = unpair(u[p][e]);
          top = fmaxf(fmaxf(fmaxf(top, fabsf(y.x)), fabsf(y.y)), fmaxf(fabsf(z.x), fabsf(z.y)));
        }
      }
    }
    if (side == 0 || g.slot0 < 0) continue;

    top = warp_max(top);
    float s = __uint_as_float(uint32_t(scale_exponent(top) + 127) << 23);
    uint8_t* codes = static_cast<uint8_t*>(side == 1 ? P.codes.k : P.codes.v);
    const int64_t pitch = (int64_t)a.heads[1] * DH;                    // bytes between slots
    if (older > 0) {
      was = was >= kKv8ScaleMin ? fminf(was, kKv8ScaleMax) : kKv8ScaleMin;
      if (s > was) {                                                   // the older codes under the larger scale
        const float r = was / s;
        uint8_t* c = codes + block * kKv8Block * pitch + h * DH;
        for (int i = lane; i < older * (DH / 16); i += 32) {
          uint4* at = reinterpret_cast<uint4*>(c + i / (DH / 16) * pitch + i % (DH / 16) * 16);
          uint4 v = *at;
          uint16_t* e = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t y = f16_of_codes(e[k]);
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&y));
            e[k] = codes_of(z.x * r, z.y * r);
          }
          *at = v;
        }
      }
      s = fmaxf(s, was);
    }
    const float inv = 1.f / s;                                         // exact where s is a power of two
    uint8_t* c = codes + (int64_t)g.slot0 * pitch + h * DH + j * 8;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int tok = p * kTok + tl;
      if (tok >= g.n) continue;
      uint16_t y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = unpair(l[p][e]), z = unpair(u[p][e]);
        y[e] = codes_of(v.x * inv, v.y * inv);
        y[4 + e] = codes_of(z.x * inv, z.y * inv);
      }
      *reinterpret_cast<uint2*>(c + tok * pitch) = make_uint2(y[0] | uint32_t(y[1]) << 16, y[2] | uint32_t(y[3]) << 16);
      *reinterpret_cast<uint2*>(c + tok * pitch + DH / 2) =
          make_uint2(y[4] | uint32_t(y[5]) << 16, y[6] | uint32_t(y[7]) << 16);
    }
    if (lane == 0) *scale = s;
  }
}

template <typename TI, typename TO>
cudaError_t launch_typed(const KvRopeArgs& a, const Kv8Pages& p, const KvFreq& f, int sm_count, cudaStream_t st) {
  const int heads = a.heads[0] + a.heads[1] + a.heads[2];
  const int chunks = (int)(((int64_t)a.n_tokens + kChunk - 1) / kChunk);
  // How many CTAs share a chunk: the waves of them, times a warp's tasks and what a CTA's start costs (kStart tasks). Few
  // chunks get one head of one group a warp, so that the call takes one load's latency; many keep their angles for more
  // heads. A chunk has one group of a prompt, 16 of a decode step. With more parts the prompts above took 64 us against
  // 61.
  constexpr int kStart = 2;
  const int groups = kChunk / min(kChunk, max(1, a.rows.max_new)), tasks = groups * heads, held = sm_count * kCtas;
  const int most = (tasks + kWarps - 1) / kWarps;
  int parts = most;
  if ((int64_t)chunks * most > held) {
    int least = INT_MAX;
    for (int p = 1; p <= min(most, 64) && (p == 1 || chunks <= 4 * held / p); ++p) {
      const int waves = (int)(((int64_t)chunks * p + held - 1) / held);
      const int time = waves * ((tasks + p * kWarps - 1) / (p * kWarps) + kStart);
      if (time < least) {
        least = time;
        parts = p;
      }
    }
  }
  const dim3 grid((unsigned)chunks + 1, (unsigned)parts);              // one to check the rows
  auto go = [&](auto kernel, size_t smem) -> cudaError_t {
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, grid, kThreads, smem, st, a, p, f);
  };
  if (a.head_dim == 128) return go(kv8_append_kernel<TI, TO, 128>, sizeof(Sm<128, sizeof(TI)>));
  return go(kv8_append_kernel<TI, TO, 64>, sizeof(Sm<64, sizeof(TI)>));
}

template <typename TI>
cudaError_t launch_from(const KvRopeArgs& a, const Kv8Pages& p, const KvFreq& f, int sm_count, cudaStream_t st) {
  if (a.dtype == kF16) return launch_typed<TI, __half>(a, p, f, sm_count, st);
  return launch_typed<TI, __nv_bfloat16>(a, p, f, sm_count, st);
}

}  // namespace

cudaError_t launch_kv8_append(const KvRopeArgs& a, const Kv8Pages& p, const KvFreq& f, int sm_count, cudaStream_t st) {
  if (a.x_dtype == kF32) return launch_from<float>(a, p, f, sm_count, st);
  if (a.x_dtype == kF16) return launch_from<__half>(a, p, f, sm_count, st);
  return launch_from<__nv_bfloat16>(a, p, f, sm_count, st);
}

}  // namespace palu
