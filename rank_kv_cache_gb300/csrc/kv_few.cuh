// What the attention kernels for few query rows share: copies, matrix instructions, and the cut of the rows into pieces.
#pragma once

#include "kv.h"

namespace palu {

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

// A piece's length: at least an equal share of all CTAs that the GPU holds. Up to 32 rows, each lane weighs one
// length, from that share to three times it or 31 steps more: the waves of CTAs times the length and what a CTA's
// start and end cost (eight steps), and the join of what is cut (four; with eight, 8 sequences at 1000 took 12.3 us
// against 9.6; with lengths up to twice a share of one step only, 300 tokens of two sequences 7.6 against 6.5). More
// rows are cut a quarter longer than the share. The quarter alone took 169 us against 136 for 32 ragged rows up to
// 8192 and 137 against 119 for 20 of 7000, and up to 1 us less for few equal rows (48.4 against 50.3, one of 65536).
__device__ __forceinline__ int piece_length(int steps0, int64_t all, int batch, int n_kv, int ctas) {
  const int lane = threadIdx.x & 31;
  const int64_t work = all * n_kv;
  const int share = work < (1 << 30) ? (int(work) + ctas - 1) / ctas : int((work + ctas - 1) / ctas);
  int per = share + share / 4;
  if (batch <= 32) {
    const int mine = share + lane * max(1, share / 16);
    const float inv = 1.f / mine;
    int count = 0, cuts = 0;
    for (int b = 0; b < batch; ++b) {
      const int p = int(ceilf(__shfl_sync(0xffffffffu, steps0, b) * inv));
      count += p;
      cuts |= p > 1;
    }
    const unsigned est = unsigned((count * n_kv + ctas - 1) / ctas) * unsigned(mine + 8) + (cuts ? 4u : 0u);
    const unsigned least = __reduce_min_sync(0xffffffffu, est);
    per = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, est == least)) - 1);
  }
  return per;
}

constexpr int kFewWarps = 4;             // warps of a CTA
template <int ROWS = kKvFewRows> struct FewJoin {
  float2 ml[kFewWarps][ROWS];            // of each warp's rows: maximum (log2 units) and sum
  float wgt[kFewWarps][ROWS];
  float2 tot[ROWS];
  int last_cta;
};

// A piece's end: joins the outputs of the warps, which took its tokens in turn and whose rows stand in
// shared memory as fp32 [warp][row][d] with their maxima and sums in X (the CTA has met since), and writes the unit's
// rows or its partial; the last CTA of a cut unit joins its pieces.
template <int DH, bool BF16, int ROWS>
__device__ __forceinline__ void finish_piece(const KvAttendArgs& a, FewJoin<ROWS>& X, uint8_t* smem, int q0, int rows, int h, int np,
                                             int piece, int first_slot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (threadIdx.x < ROWS) {
    const int r = threadIdx.x;
    float M = -INFINITY, Lsum = 0.f;
    for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, X.ml[w][r].x);
    for (int w = 0; w < kFewWarps; ++w) {
      const float x = M == -INFINITY ? 0.f : ex2(X.ml[w][r].x - M);
      X.wgt[w][r] = x;
      Lsum = fmaf(X.ml[w][r].y, x, Lsum);
    }
    X.tot[r] = make_float2(M, Lsum);
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
  float* po = a.part_o + (int64_t)(first_slot + piece) * ROWS * DH;
  for (int x = tid; x < rows * (DH / 2); x += kFewWarps * 32) {
    const int r = x / (DH / 2), cl = x % (DH / 2) * 2;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kFewWarps; ++y) {
      const float2 u = *reinterpret_cast<const float2*>(of + (y * ROWS + r) * DH + cl);
      v.x = fmaf(u.x, X.wgt[y][r], v.x);
      v.y = fmaf(u.y, X.wgt[y][r], v.y);
    }
    if (whole) {
      const float Lsum = X.tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + out_at(r) + cl) = pack2<BF16>(v.x * inv, v.y * inv);
      if (cl == 0) write_lse(r, X.tot[r].x, Lsum);
    } else {
      *reinterpret_cast<float2*>(po + r * DH + cl) = v;
    }
  }
  if (!whole) {
    if (tid < rows) a.part_ml[(int64_t)(first_slot + piece) * ROWS + tid] = X.tot[tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) X.last_cta = atomicAdd(&a.counters[first_slot], 1u) == unsigned(np - 1);
    __syncthreads();
    if (X.last_cta) {
      __threadfence();
      // join the pieces, in their order
      float* wr = reinterpret_cast<float*>(smem);                  // [rows][np] weights
      auto slot = [&](int k) { return (int64_t)(first_slot + k) * ROWS; };
      for (int r = warp; r < rows; r += kFewWarps) {
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
        if (lane == 0) X.tot[r] = make_float2(M, Lsum);
      }
      __syncthreads();
      for (int x = tid; x < rows * (DH / 4); x += kFewWarps * 32) {
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
        const float Lsum = X.tot[r].y, inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_at(r) + cl) =
            make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
        if (cl == 0) write_lse(r, X.tot[r].x, Lsum);
      }
      if (tid == 0) a.counters[first_slot] = 0u;
    }
  }
}

}  // namespace palu
