// C ABI of the 8-bit paged KV cache, of the plan of a step's rows and pages, and of the verification of drafts: validation
// and launches. Host code only.
#include "kv8.h"
#include "kv_handle.h"

using namespace palu;

namespace {

// the codes as the pages that the shared checks and look-ups know
palu_status_t check_pages8(const palu_kv* h, const palu_kv8_pages* p, const palu_kv_rows* r) {
  if (!h || !p || !r) return PALU_ERR_INVALID_ARG;
  const palu_kv_pages codes{p->k, p->v, p->n_pages, p->page_size};
  const palu_status_t st = check_pages_rows(h, &codes, r);
  if (st != PALU_OK) return st;
  if (p->page_size % kKv8Block) return PALU_ERR_INVALID_ARG;
  if (!p->k_scale || !p->v_scale || (uintptr_t)p->k_scale % 4 || (uintptr_t)p->v_scale % 4) return PALU_ERR_INVALID_ARG;
  return h->d.dtype == PALU_F32 ? PALU_ERR_UNSUPPORTED : PALU_OK;
}

KvPages codes_of_pages(const palu_kv8_pages& p) { return KvPages{p.k, p.v, p.n_pages, p.page_size}; }

// Which kernel. The streaming one holds up to 24 query rows and reads the cache at up to the full rate, but its warps take their
// steps one after the other, the longer the more rows there are: while the call's bounds promise an SM few steps of 128
// cached tokens, the tensor-core kernel is sooner done. 32 / 8 heads of 128, 24 query rows: one sequence at 4096 (1.7 steps an SM)
// 34 us against 18, two at 16384 (13.5) 45 against 38, four at 16384 (27) 56 against 64, eight (54) 87 against 110. 16 rows: one
// at 4096 24 against 18, two 24 against 21, at 16384 34 against 37, four at 4096 (6.7) 25 against 26. Heads of 64, 24 rows: one
// at 4096 19 against 16, two at 16384 30 against 33, four at 1000 16 against 19.
bool streams(const KvAttendArgs& a, int sms) {
  const int64_t rows = (int64_t)a.rows.max_new * a.g, units = (int64_t)a.rows.batch * a.n_kv;
  const int64_t steps = units * ((a.rows.max_kv_len + 127) / 128);
  if (rows > kKv8FewRows) return false;
  if (rows > 16 && a.head_dim == 128) return steps > (int64_t)16 * sms;
  return rows <= (a.head_dim == 128 ? 12 : 16) || units > 16 || steps > (int64_t)7 * sms;
}

bool bad_ints(const void* p) { return !p || (uintptr_t)p % 4; }

}  // namespace

extern "C" {

palu_status_t palu_append_kv8(palu_kv_t h, const palu_kv8_pages* pages, const palu_kv_rows* rows, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const void* q_norm, const void* k_norm, void* q_out, palu_stream_t stream) {
  const palu_status_t st = check_pages8(h, pages, rows);
  if (st != PALU_OK) return st;
  if (rows->batch == 0 || rows->n_tokens == 0) return PALU_OK;
  const palu_kv_desc& d = h->d;
  if (bad_view(k, k_stride, d.n_kv_heads, d.head_dim, d.x_dtype) ||
      bad_view(v, v_stride, d.n_kv_heads, d.head_dim, d.x_dtype))
    return PALU_ERR_INVALID_ARG;
  if (!q != !q_out) return PALU_ERR_INVALID_ARG;
  if (q && (bad_view(q, q_stride, d.n_heads, d.head_dim, d.x_dtype) || (uintptr_t)q_out % 16)) return PALU_ERR_INVALID_ARG;
  const int64_t packed = (int64_t)d.n_heads * d.head_dim;
  if (q && q == q_out && (d.dtype != d.x_dtype || q_stride != packed)) return PALU_ERR_INVALID_ARG;
  if ((uintptr_t)q_norm % 16 || (uintptr_t)k_norm % 16) return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  KvRopeArgs a{};
  rope_args(h, a);
  a.src[0] = q;
  a.src[1] = k;
  a.src[2] = v;
  a.src_stride[0] = q_stride;
  a.src_stride[1] = k_stride;
  a.src_stride[2] = v_stride;
  a.dst[0] = q_out;
  a.dst_stride[0] = packed;
  a.w[0] = q_norm;
  a.w[1] = k_norm;
  a.heads[0] = q ? d.n_heads : 0;
  a.heads[1] = a.heads[2] = d.n_kv_heads;
  a.positions = rows->positions;
  a.n_tokens = (int)rows->n_tokens;
  a.append = 1;
  a.rows = rows_of(*rows);
  const Kv8Pages p{codes_of_pages(*pages), {pages->k_scale, pages->v_scale}};
  const cudaError_t e = launch_kv8_append(a, p, h->freq, h->sm_count, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

palu_status_t palu_attend_kv8(palu_kv_t h, const palu_kv8_pages* pages, const palu_kv_rows* rows, const void* q,
                              int64_t q_stride, void* out, float* lse, palu_stream_t stream) {
  const palu_status_t st = check_pages8(h, pages, rows);
  if (st != PALU_OK) return st;
  const palu_kv_desc& d = h->d;
  if (rows->batch == 0 || rows->n_tokens == 0) return PALU_OK;
  if (bad_view(q, q_stride, d.n_heads, d.head_dim, d.dtype)) return PALU_ERR_INVALID_ARG;
  if (!out || (uintptr_t)out % 16 || (uintptr_t)lse % 4) return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  Kv8AttendArgs A{};
  A.k_scale = pages->k_scale;
  A.v_scale = pages->v_scale;
  KvAttendArgs& a = A.a;
  attend_args(h, *rows, q, q_stride, out, lse, a);
  a.pages = codes_of_pages(*pages);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (streams(a, h->sm_count)) {
    e = launch_kv8_attend_few(A, h->sm_count, s);
  } else {
    e = launch_kv8_attend_tc(A, tc_plan(h, *rows), s);
    if (e == cudaErrorNotSupported) return PALU_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

palu_status_t palu_plan_kv_rows(palu_kv_t h, const palu_kv_pool* pool, const int32_t* new_tokens, const int32_t* kv_len,
                                int batch, int64_t n_tokens, int max_new, int64_t max_kv_len, int32_t* row_start,
                                int32_t* kv_len_out, int32_t* held_out, int32_t* state_out, int32_t* positions,
                                int32_t* slots, palu_stream_t stream) {
  if (!h || !pool) return PALU_ERR_INVALID_ARG;
  if (batch < 0 || batch > h->d.max_batch || n_tokens < 0 || n_tokens > h->d.max_tokens) return PALU_ERR_INVALID_ARG;
  if (max_new < 0 || max_kv_len < 0) return PALU_ERR_INVALID_ARG;
  if (pool->n_pages <= 0 || pool->page_size <= 0 || pool->table_pages <= 0) return PALU_ERR_INVALID_ARG;
  if (pool->n_pages >= (int64_t(1) << 31) || pool->n_pages * pool->page_size >= (int64_t(1) << 31) ||
      pool->table_pages >= (int64_t(1) << 31) || max_kv_len >= (int64_t(1) << 30))
    return PALU_ERR_UNSUPPORTED;
  if (max_kv_len > pool->table_pages * pool->page_size) return PALU_ERR_INVALID_ARG;
  if (batch == 0) return PALU_OK;
  if (bad_ints(pool->page_table) || bad_ints(pool->held) || bad_ints(pool->free_pages) || bad_ints(pool->free_state) ||
      bad_ints(new_tokens) || bad_ints(kv_len) || bad_ints(row_start) || bad_ints(kv_len_out) ||
      (uintptr_t)held_out % 4 || (uintptr_t)state_out % 4 || (uintptr_t)positions % 4 || (uintptr_t)slots % 4)
    return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  KvPlanArgs a{};
  a.table = pool->page_table;
  a.table_pages = pool->table_pages;
  a.held = pool->held;
  a.ring = pool->free_pages;
  a.state = pool->free_state;
  a.n_pages = (int)pool->n_pages;
  a.page_size = pool->page_size;
  a.fresh = new_tokens;
  a.kv_len = kv_len;
  a.batch = batch;
  a.n_tokens = (int)n_tokens;
  a.max_new = max_new;
  a.max_kv_len = (int)max_kv_len;
  a.row_start = row_start;
  a.kv_len_out = kv_len_out;
  a.held_out = held_out ? held_out : pool->held;
  a.state_out = state_out ? state_out : pool->free_state;
  a.positions = positions;
  a.slots = slots;
  a.err = reinterpret_cast<ErrWord*>(h->ws + h->L.err);
  return launch_kv_plan(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

palu_status_t palu_verify_drafts(palu_kv_t h, const void* target, int64_t target_stride, const void* draft,
                                 int64_t draft_stride, palu_dtype_t p_dtype, int64_t vocab, const int32_t* row_start,
                                 int batch, int64_t n_tokens, const int32_t* draft_tokens, int max_draft,
                                 const float* uniforms, int32_t* tokens, int32_t* accepted, const int32_t* kv_len,
                                 int32_t* kv_len_out, palu_stream_t stream) {
  if (!h || batch < 0 || batch > h->d.max_batch || n_tokens < 0 || n_tokens > h->d.max_tokens) return PALU_ERR_INVALID_ARG;
  if ((unsigned)p_dtype > PALU_INT4 || vocab <= 0 || max_draft < 0) return PALU_ERR_INVALID_ARG;
  if (p_dtype == PALU_INT4 || vocab > (int64_t(1) << 20) || max_draft > (1 << 20)) return PALU_ERR_UNSUPPORTED;
  if (batch == 0) return PALU_OK;
  const int64_t e = elem_size(p_dtype), far = int64_t(1) << 31;
  if ((n_tokens > 0 && !target) || (uintptr_t)target % e || target_stride < vocab || target_stride > far)
    return PALU_ERR_INVALID_ARG;
  if (draft && ((uintptr_t)draft % e || draft_stride < vocab || draft_stride > far)) return PALU_ERR_INVALID_ARG;
  if (bad_ints(row_start) || bad_ints(uniforms) || bad_ints(tokens) || bad_ints(accepted) ||
      (max_draft > 0 && bad_ints(draft_tokens)) || !kv_len != !kv_len_out || (uintptr_t)kv_len % 4 ||
      (uintptr_t)kv_len_out % 4)
    return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  KvVerifyArgs a{};
  a.target = target;
  a.target_stride = target_stride;
  a.draft = draft;
  a.draft_stride = draft_stride;
  a.dtype = (int)p_dtype;
  a.vocab = (int)vocab;
  a.row_start = row_start;
  a.batch = batch;
  a.n_tokens = (int)n_tokens;
  a.draft_tokens = draft_tokens;
  a.max_draft = max_draft;
  a.uniforms = uniforms;
  a.tokens = tokens;
  a.accepted = accepted;
  a.kv_len = kv_len;
  a.kv_len_out = kv_len_out;
  a.err = reinterpret_cast<ErrWord*>(h->ws + h->L.err);
  return launch_kv_verify(a, h->sm_count, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

}  // extern "C"
