// Internal interface of the paged dense KV cache's operators: the norm and rotation of queries and
// keys, the append into the pages, and the attention of new tokens over them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace palu {

// what this cache's operators record beside ErrWhere's
constexpr unsigned kErrPage = 6;   // a page table entry outside the page pool
constexpr unsigned kErrRows = 7;   // row_start decreases, or a row has more new tokens than the call's bound

constexpr int kKvMaxHalf = 64;   // pairs of a head: head_dim / 2

// Rotation frequencies: F_k = frac(theta^(-2k/d) / 2 pi) as a 64-bit fraction of a turn, rounded to nearest.
// pos * F_k mod 2^64 is then the phase of position pos: of the product nothing is lost, and the rounding of
// F_k moves it by at most 2^-34 turns for any int32 position.
struct KvFreq {
  uint64_t turn[kKvMaxHalf];
};

// The new tokens and caches of a batch (device arrays as the C ABI describes them).
struct KvRows {
  const int32_t* row_start;    // [batch + 1]
  const int32_t* kv_len;       // [batch]
  const int32_t* page_table;   // [batch][table_pages]; nullptr: row b is page b
  int batch;
  int n_tokens;
  int max_new;
  int max_kv_len;
  int64_t table_pages;
};
struct KvPages {
  void* k;
  void* v;
  int64_t n_pages;
  int page_size;
};

// Slot index (page * page_size + offset) of token t of row b, or -1 where the page table gives no page.
__device__ __forceinline__ int64_t kv_slot(const KvRows& r, const KvPages& p, int b, int t) {
  if (!r.page_table) return t < p.page_size ? (int64_t)b * p.page_size + t : -1;
  const int pg = t / p.page_size;
  if (pg >= r.table_pages) return -1;
  const int page = r.page_table[(int64_t)b * r.table_pages + pg];
  if (page < 0 || page >= p.n_pages) return -1;
  return (int64_t)page * p.page_size + (t - pg * p.page_size);
}

// The kernels here are launched to start while the one ahead of them in the stream still runs: every thread first
// waits for that one's end (grid_wait, before anything of it is read or its memory written), and says at once that the
// next one may set itself up. A few microseconds of launch latency hide behind the work.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                         const Args&... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Row b's first packed token, new tokens and cached length, clamped to the call's bounds; false where the row
// is skipped. `bad`: what to record (an ErrWhere), or 0.
__device__ __forceinline__ bool kv_row(const KvRows& r, int b, int& q0, int& n, int& L, unsigned& bad) {
  q0 = r.row_start[b];
  const int q1 = r.row_start[b + 1];
  const int len = r.kv_len[b];
  const bool skip = q0 < 0 || q1 < q0 || q1 > r.n_tokens;
  n = skip ? 0 : q1 - q0;
  bad = skip || n > r.max_new ? kErrRows : len < 0 || len > r.max_kv_len ? kErrSeqLen : 0u;
  n = min(n, r.max_new);
  L = max(0, min(len, r.max_kv_len));
  return !skip;
}

// 2^x by the special function unit (relative error 2^-22; 2^-inf = 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 values in one 64-bit register, and the packed arithmetic on them
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What the exponents of a softmax's weights are taken from, for a largest score `top` (log2 units): p = 2^(s - base).
// The weights are rounded to the cache's type for the product with V, while their sum is not. In fp16 a weight below
// 2^-25 would vanish from the product alone: behind a score 17.4 (natural) above the others, as attention sinks have,
// 65536 tokens would lose 2^-9 of that score's weight, and all of their own. So fp16 weights are lifted to use the
// type's range, the largest 2^lift; a shift of the base changes neither o / l nor m + log2 l. Scores past 2^20, whose
// fp32 steps could carry the largest weight out of range, are not lifted. bf16 has the range of fp32.
template <bool BF16> __device__ __forceinline__ float softmax_base(float top, float lift) {
  if constexpr (BF16) return top;
  return fabsf(top) < 1048576.f ? top - lift : top;
}

template <bool BF16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// norm_rope and append: one kernel over packed tokens and the heads of q, k and (append) v
struct KvRopeArgs {
  const void* src[3];          // q, k, v (nullptr: absent)
  int64_t src_stride[3];       // elements between tokens
  void* dst[2];                // q out, k out (norm_rope; append: k goes to the pages)
  int64_t dst_stride[2];
  const void* w[2];            // norm weights of q and k, x_dtype (nullptr: no norm)
  int heads[3];                // heads of q, k, v (0: absent)
  int head_dim;
  int x_dtype, dtype;
  int rotate;
  float eps;
  const int32_t* positions;    // [n_tokens]; nullptr (append): the token's slot in its row
  int n_tokens;
  int append;
  KvRows rows;                 // append
  KvPages pages;
  ErrWord* err;
};
cudaError_t launch_kv_rope(const KvRopeArgs& a, const KvFreq& f, int sm_count, cudaStream_t st);

// attention of new tokens over the pages
struct KvAttendArgs {
  const void* q;               // [n_tokens][n_heads][d], token stride q_stride elements
  int64_t q_stride;
  void* out;                   // [n_tokens][n_heads][d]
  float* lse;                  // [n_tokens][n_heads] or nullptr
  KvRows rows;
  KvPages pages;
  int n_heads, n_kv, g;        // g = n_heads / n_kv query heads share a key/value head
  int head_dim;
  int bf16;
  float scale_log2;            // log2(e) / sqrt(d)
  float* part_o;               // fp32 partial outputs, not yet divided by their sums
  float2* part_ml;             // their running maxima (log2 units) and sums
  unsigned* counters;          // few rows: [piece of a cut unit], zero between calls
  int ctas;                    // few rows: CTAs that the GPU holds at once
  ErrWord* err;
};
// Query rows (token, head of the group) of a unit: what one matrix instruction takes, and the most that run here.
// 16 rows took 169 us here against 179 on the tensor-core kernel (64 sequences at 4096), 64 against 66 (one at
// 65536) and 12.0 against 11.3 (16 at 256); 20 rows, in two passes, 120 against 82 (eight ragged up to 16384).
constexpr int kKvFewRows = 16;
constexpr int kKvFewTokens = 64;         // cached tokens of 128 elements that a CTA's warps take together
constexpr int kKvFewCtas = 2;            // CTAs of an SM; one takes 237 us where two take 160 (four at 65536)
constexpr int kKvFewMostCtas = 512;      // most CTAs of a call; cut units have at most twice as many pieces
// once a handle, on its device: what the kernel's launches need set
cudaError_t prepare_kv_attend_few(int head_dim, bool bf16);
cudaError_t launch_kv_attend_few(KvAttendArgs a, int sm_count, cudaStream_t st);   // max_new g <= 16

// the tensor-core kernel
constexpr int kKvTcRows = 128;           // query rows of a tile
// Steps of 128 cached tokens up to which a tile is not cut. With 4, calls of 5 and 6 steps took 0.3 to 0.9 us more
// (16 sequences of 32 at 700: 35.8 against 34.9); with 12, 64 new tokens at 1024 took 19.7 us against 16.1.
constexpr int kKvTcWhole = 6;
struct KvPlanHead {
  unsigned next;     // the next item to take; zero between calls
  unsigned done;     // CTAs that have ended; zero between calls
  unsigned pieces;   // pieces of cut tiles that are stored; zero between calls
};
struct KvTcPlan {
  KvPlanHead* head;
  int tile_cap;      // most tiles (or pairs of tiles) the call's packed tokens can make
  int slots;         // most pieces x key/value heads whose partials the workspace holds
  int sm_count;
  int test_stall;    // failure-detection test hook: the value loader issues nothing
  uint64_t wait_ns;  // bound of the kernel's waits
};
cudaError_t prepare_kv_attend_tc(int head_dim, bool bf16);
cudaError_t launch_kv_attend_tc(const KvAttendArgs& a, const KvTcPlan& t, cudaStream_t st);

}  // namespace palu
