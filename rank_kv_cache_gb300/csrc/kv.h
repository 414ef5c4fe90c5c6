// Internal interface of the paged dense KV cache's operators: the norm and rotation of queries and
// keys, the append into the pages, and the attention of new tokens over them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace palu {

constexpr int kKvMaxHalf = 64;   // pairs of a head: head_dim / 2

// Rotation frequencies: F_k = frac(theta^(-2k/d) / 2 pi) as a 64-bit fraction of a turn, so that
// pos * F_k mod 2^64 is the phase of position pos, range-reduced exactly for every int32 position.
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
  int n_splits;                // ranges a row's cached tokens are cut into
  float* part_o;               // [unit][n_splits][16][d] fp32 partial outputs, normalised by nothing
  float2* part_ml;             // [unit][n_splits][16]: running maximum (log2 units) and sum
  unsigned* counters;          // [unit], zero between calls
  ErrWord* err;
};
constexpr int kKvFewRows = 16;           // query rows (token, head of the group) of a unit
constexpr int kKvFewStep = 128;          // cached tokens the unit's warps take together
cudaError_t launch_kv_attend_few(const KvAttendArgs& a, cudaStream_t st);

}  // namespace palu
