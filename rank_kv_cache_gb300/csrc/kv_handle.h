// The handle of the paged KV cache's operators, and what its host files share.
#pragma once

#include <math.h>

#include "palu_attn.h"
#include "kv.h"

namespace palu {

// Partials of a call: work that is cut takes a slot for each piece. The cuts keep to these numbers, so the
// workspace does not grow with the call. The two kernels' partials share the space.
constexpr int kPartSlots = 2 * kKvFewMostCtas;   // few rows: pieces of 16 query rows (24 over 8-bit pages)
constexpr int kTcSlots = 456;      // tensor-core kernel: pieces x key/value heads, of two 128-row tiles

struct KvLayout {
  size_t err, head, counters, part_ml, part_o, total;
};

// tiles (or pairs of tiles) that n_tokens packed new tokens of `batch` rows make at most
inline int64_t tc_tile_cap(const palu_kv_desc& d, int64_t n_tokens, int64_t batch) {
  const int64_t per = 2 * (kKvTcRows / (d.n_heads / d.n_kv_heads));
  return (n_tokens + per - 1) / per + batch;
}

inline int64_t elem_size(palu_dtype_t t) { return t == PALU_F32 ? 4 : 2; }

// a [tokens][heads][head_dim] array: 16-byte aligned, tokens a multiple of 16 bytes apart and not overlapping
inline bool bad_view(const void* p, int64_t stride, int heads, int head_dim, palu_dtype_t t) {
  return !p || (uintptr_t)p % 16 || stride < (int64_t)heads * head_dim || stride > (int64_t(1) << 31) ||
         stride * elem_size(t) % 16;
}

// the workspace's device for the length of a call; the thread's own comes back afterwards
struct DeviceGuard {
  int before = -1;
  bool ok;
  explicit DeviceGuard(int device) {
    ok = cudaGetDevice(&before) == cudaSuccess && (before == device || cudaSetDevice(device) == cudaSuccess);
    if (before == device) before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};

}  // namespace palu

struct palu_kv {
  palu_kv_desc d;
  char* ws;
  palu::KvLayout L;
  int device;
  int sm_count;
  palu::KvFreq freq;
};

namespace palu {

inline palu_status_t check_pages_rows(const palu_kv* h, const palu_kv_pages* p, const palu_kv_rows* r) {
  if (!h || !p || !r) return PALU_ERR_INVALID_ARG;
  if (r->batch < 0 || r->batch > h->d.max_batch || r->n_tokens < 0 || r->n_tokens > h->d.max_tokens)
    return PALU_ERR_INVALID_ARG;
  if (r->max_new < 0 || r->max_kv_len < 0) return PALU_ERR_INVALID_ARG;
  if (!p->k || !p->v || (uintptr_t)p->k % 16 || (uintptr_t)p->v % 16) return PALU_ERR_INVALID_ARG;
  if (p->n_pages <= 0 || p->page_size <= 0) return PALU_ERR_INVALID_ARG;
  if (p->n_pages >= (int64_t(1) << 31) || p->n_pages * p->page_size >= (int64_t(1) << 31)) return PALU_ERR_UNSUPPORTED;
  if (r->batch == 0 || r->n_tokens == 0) return PALU_OK;
  if (!r->row_start || !r->kv_len || (uintptr_t)r->row_start % 4 || (uintptr_t)r->kv_len % 4 ||
      (uintptr_t)r->page_table % 4 || (uintptr_t)r->positions % 4)
    return PALU_ERR_INVALID_ARG;
  if (r->page_table) {
    if (r->table_pages <= 0 || r->table_pages >= (int64_t(1) << 31)) return PALU_ERR_INVALID_ARG;
    if (r->max_kv_len > r->table_pages * p->page_size) return PALU_ERR_INVALID_ARG;
  } else if (r->max_kv_len > p->page_size || r->batch > p->n_pages) {
    return PALU_ERR_INVALID_ARG;
  }
  if (r->max_kv_len >= (int64_t(1) << 30)) return PALU_ERR_UNSUPPORTED;
  return PALU_OK;
}

inline KvRows rows_of(const palu_kv_rows& r) {
  KvRows o{};
  o.row_start = r.row_start;
  o.kv_len = r.kv_len;
  o.page_table = r.page_table;
  o.batch = r.batch;
  o.n_tokens = (int)r.n_tokens;
  o.max_new = r.max_new < r.n_tokens ? r.max_new : (int)r.n_tokens;
  o.max_kv_len = (int)r.max_kv_len;
  o.table_pages = r.table_pages;
  return o;
}

inline void rope_args(const palu_kv* h, KvRopeArgs& a) {
  a.head_dim = h->d.head_dim;
  a.x_dtype = (int)h->d.x_dtype;
  a.dtype = (int)h->d.dtype;
  a.rotate = h->d.rope_theta > 0.0;
  a.eps = (float)h->d.norm_eps;
  a.err = reinterpret_cast<ErrWord*>(h->ws + h->L.err);
}

// everything but the pages
inline void attend_args(const palu_kv* h, const palu_kv_rows& rows, const void* q, int64_t q_stride, void* out, float* lse,
                        KvAttendArgs& a) {
  const palu_kv_desc& d = h->d;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.rows = rows_of(rows);
  a.n_heads = d.n_heads;
  a.n_kv = d.n_kv_heads;
  a.g = d.n_heads / d.n_kv_heads;
  a.head_dim = d.head_dim;
  a.bf16 = d.dtype == PALU_BF16;
  a.scale_log2 = float(1.4426950408889634 / sqrt((double)d.head_dim));
  a.part_o = reinterpret_cast<float*>(h->ws + h->L.part_o);
  a.part_ml = reinterpret_cast<float2*>(h->ws + h->L.part_ml);
  a.counters = reinterpret_cast<unsigned*>(h->ws + h->L.counters);
  a.err = reinterpret_cast<ErrWord*>(h->ws + h->L.err);
}

inline KvTcPlan tc_plan(const palu_kv* h, const palu_kv_rows& rows) {
  KvTcPlan t{};
  t.head = reinterpret_cast<KvPlanHead*>(h->ws + h->L.head);
  t.tile_cap = (int)tc_tile_cap(h->d, rows.n_tokens, rows.batch);
  t.slots = kTcSlots;
  t.sm_count = h->sm_count;
  t.test_stall = (h->d.flags & PALU_FLAG_TEST_STALL) != 0;
  t.wait_ns = t.test_stall ? 50000000ull : 1000000000ull;   // bound of every device wait
  return t;
}

}  // namespace palu
