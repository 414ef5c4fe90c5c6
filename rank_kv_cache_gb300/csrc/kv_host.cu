// C ABI of the paged dense KV cache: validation, workspace layout, launch planning. Host code only.
#include <math.h>

#include <new>

#include "kv8.h"
#include "kv_handle.h"

using namespace palu;

namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

KvLayout kv_layout(const palu_kv_desc& d) {
  KvLayout L{};
  size_t off = 0;
  L.err = off;
  off = align256(off + 256);
  if (d.dtype != PALU_F32) {
    const size_t few = (size_t)kPartSlots * kKv8FewRows, tc = (size_t)kTcSlots * 2 * kKvTcRows;
    const size_t rows = few > tc ? few : tc;
    L.head = off;
    off = align256(off + sizeof(KvPlanHead));
    L.counters = off;
    off = align256(off + kPartSlots * sizeof(unsigned));
    L.part_ml = off;
    off = align256(off + rows * sizeof(float2));
    L.part_o = off;
    off = align256(off + rows * d.head_dim * sizeof(float));
  }
  L.total = off;
  return L;
}

palu_status_t check_kv_desc(const palu_kv_desc* d) {
  if (!d || d->abi_version != PALU_ABI_VERSION) return PALU_ERR_INVALID_ARG;
  if (d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads) return PALU_ERR_INVALID_ARG;
  if (d->head_dim <= 0 || (unsigned)d->dtype > PALU_INT4 || (unsigned)d->x_dtype > PALU_INT4)
    return PALU_ERR_INVALID_ARG;
  if (!(d->rope_theta >= 0.0) || !isfinite(d->rope_theta) || !(d->norm_eps >= 0.0) || !isfinite(d->norm_eps))
    return PALU_ERR_INVALID_ARG;
  if (d->max_batch <= 0 || d->max_tokens <= 0 || (d->flags & ~PALU_FLAG_TEST_STALL)) return PALU_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return PALU_ERR_UNSUPPORTED;
  if (d->dtype == PALU_INT4 || d->x_dtype == PALU_INT4) return PALU_ERR_UNSUPPORTED;
  if (d->n_heads / d->n_kv_heads > 64 || d->n_heads > 4096) return PALU_ERR_UNSUPPORTED;
  if (d->max_batch > 65535 || d->max_tokens >= (int64_t(1) << 31)) return PALU_ERR_UNSUPPORTED;
  return PALU_OK;
}

// An unevaluated sum of two doubles, the second at most half an ulp of the first: 106 bits (Dekker 1971). The leading
// product is kept from being fused with what follows.
struct Dd {
  double hi, lo;
};
Dd dd_sum(double a, double b) {            // |a| >= |b|
  volatile double s = a + b;
  return {s, b - (s - a)};
}
Dd dd_mul(Dd a, Dd b) {
  volatile double p = a.hi * b.hi;
  return dd_sum(p, fma(a.hi, b.hi, -p) + fma(a.hi, b.lo, a.lo * b.hi));
}
Dd dd_sqrt(Dd a) {                         // one Newton step from the double's root
  const double s = sqrt(a.hi);
  return dd_sum(s, (fma(-s, s, a.hi) + a.lo) / (2 * s));
}
Dd dd_inverse(Dd a) {
  const double q = 1 / a.hi;
  return dd_sum(q, q * fma(-q, a.lo, fma(-q, a.hi, 1.0)));
}

// turn[k] = theta^(-2k/d) / 2 pi in units of 2^-64 turns, rounded to a whole one (bases below 1 reach whole turns, which
// fall away). In doubles the 53 bits of a frequency are off by up to 3e-7 rad at the far end of the positions; here the
// root theta^(2/d) takes five or six square roots and each frequency one product, with 2^-96 of error.
void rope_turns(double theta, int half, uint64_t* turn) {
  Dd root{theta, 0.0};
  for (int n = half; n > 1; n /= 2) root = dd_sqrt(root);
  const Dd step = dd_inverse(root);
  Dd w{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};       // 1 / (2 pi)
  for (int k = 0; k < half; ++k, w = dd_mul(w, step)) {
    const double t = ldexp(w.hi - floor(w.hi), 64), whole = floor(t);
    const double rest = (t - whole) + ldexp(w.lo - floor(w.lo + 0.5), 64);
    turn[k] = isfinite(t) && fabs(rest) < 0x1p63 ? (whole < 0x1p64 ? (uint64_t)whole : 0) + (uint64_t)llrint(rest) : 0;
  }
}

}  // namespace

static KvPages pages_of(const palu_kv_pages& p) { return KvPages{p.k, p.v, p.n_pages, p.page_size}; }

extern "C" {

palu_status_t palu_kv_workspace_size(const palu_kv_desc* desc, size_t* bytes) {
  if (!bytes) return PALU_ERR_INVALID_ARG;
  const palu_status_t st = check_kv_desc(desc);
  if (st != PALU_OK) return st;
  *bytes = kv_layout(*desc).total;
  return PALU_OK;
}

palu_status_t palu_kv_create(const palu_kv_desc* desc, void* workspace, size_t workspace_bytes, palu_stream_t stream,
                             palu_kv_t* out) {
  if (!out) return PALU_ERR_INVALID_ARG;
  *out = nullptr;
  const palu_status_t st = check_kv_desc(desc);
  if (st != PALU_OK) return st;
  const KvLayout L = kv_layout(*desc);
  if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < L.total) return PALU_ERR_WORKSPACE;
  cudaPointerAttributes attr;
  if (cudaPointerGetAttributes(&attr, workspace) != cudaSuccess || attr.type != cudaMemoryTypeDevice) {
    cudaGetLastError();
    return PALU_ERR_WORKSPACE;
  }
  DeviceGuard dev(attr.device);
  int sms = 0;
  if (!dev.ok || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, attr.device) != cudaSuccess)
    return PALU_ERR_CUDA;
  palu_kv* h = new (std::nothrow) palu_kv();
  if (!h) return PALU_ERR_INVALID_ARG;
  h->d = *desc;
  h->ws = static_cast<char*>(workspace);
  h->L = L;
  h->device = attr.device;
  h->sm_count = sms;
  if (desc->rope_theta > 0.0) rope_turns(desc->rope_theta, desc->head_dim / 2, h->freq.turn);
  if (desc->dtype != PALU_F32) {
    const bool bf16 = desc->dtype == PALU_BF16;
    if (prepare_kv_attend_few(desc->head_dim, bf16) != cudaSuccess ||
        prepare_kv_attend_tc(desc->head_dim, bf16) != cudaSuccess ||
        prepare_kv8_attend_few(desc->head_dim, bf16) != cudaSuccess ||
        prepare_kv8_attend_tc(desc->head_dim, bf16) != cudaSuccess) {
      delete h;
      return PALU_ERR_CUDA;
    }
  }
  const size_t clear = desc->dtype == PALU_F32 ? 256 : L.part_ml;   // error word, list head and counters
  if (cudaMemsetAsync(h->ws, 0, clear, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    delete h;
    return PALU_ERR_CUDA;
  }
  *out = h;
  return PALU_OK;
}

palu_status_t palu_kv_destroy(palu_kv_t h) {
  delete h;
  return PALU_OK;
}

palu_status_t palu_kv_check(palu_kv_t h, palu_stream_t stream) {
  if (!h) return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ErrWord w{};
  if (cudaMemcpyAsync(&w, h->ws + h->L.err, sizeof(w), cudaMemcpyDeviceToHost, s) != cudaSuccess) return PALU_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return PALU_ERR_CUDA;
  if (w.code == 0) return PALU_OK;
  if (cudaMemsetAsync(h->ws + h->L.err, 0, sizeof(w), s) != cudaSuccess) return PALU_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return PALU_ERR_CUDA;
  return w.code == kCodeTimeout ? PALU_ERR_TIMEOUT : PALU_ERR_DEVICE;
}

palu_status_t palu_norm_rope(palu_kv_t h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* q_norm, const void* k_norm, const int32_t* positions, int64_t n_tokens,
                             void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                             palu_stream_t stream) {
  if (!h || n_tokens < 0 || n_tokens > h->d.max_tokens) return PALU_ERR_INVALID_ARG;
  if (n_tokens == 0) return PALU_OK;
  const palu_kv_desc& d = h->d;
  if (bad_view(q, q_stride, d.n_heads, d.head_dim, d.x_dtype) ||
      bad_view(q_out, q_out_stride, d.n_heads, d.head_dim, d.dtype))
    return PALU_ERR_INVALID_ARG;
  if (k && (bad_view(k, k_stride, d.n_kv_heads, d.head_dim, d.x_dtype) ||
            bad_view(k_out, k_out_stride, d.n_kv_heads, d.head_dim, d.dtype)))
    return PALU_ERR_INVALID_ARG;
  // in place: the output must cover the input element for element
  if ((q == q_out && (d.dtype != d.x_dtype || q_stride != q_out_stride)) ||
      (k && k == k_out && (d.dtype != d.x_dtype || k_stride != k_out_stride)))
    return PALU_ERR_INVALID_ARG;
  if ((uintptr_t)q_norm % 16 || (uintptr_t)k_norm % 16 || (uintptr_t)positions % 4) return PALU_ERR_INVALID_ARG;
  if (!positions && d.rope_theta > 0.0) return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  KvRopeArgs a{};
  rope_args(h, a);
  a.src[0] = q;
  a.src[1] = k;
  a.src_stride[0] = q_stride;
  a.src_stride[1] = k_stride;
  a.dst[0] = q_out;
  a.dst[1] = k_out;
  a.dst_stride[0] = q_out_stride;
  a.dst_stride[1] = k_out_stride;
  a.w[0] = q_norm;
  a.w[1] = k_norm;
  a.heads[0] = d.n_heads;
  a.heads[1] = k ? d.n_kv_heads : 0;
  a.positions = positions;
  a.n_tokens = (int)n_tokens;
  const cudaError_t e = launch_kv_rope(a, h->freq, h->sm_count, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

palu_status_t palu_append_kv(palu_kv_t h, const palu_kv_pages* pages, const palu_kv_rows* rows, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* q_norm, const void* k_norm, void* q_out, palu_stream_t stream) {
  const palu_status_t st = check_pages_rows(h, pages, rows);
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
  a.pages = pages_of(*pages);
  const cudaError_t e = launch_kv_rope(a, h->freq, h->sm_count, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

palu_status_t palu_attend_kv(palu_kv_t h, const palu_kv_pages* pages, const palu_kv_rows* rows, const void* q,
                             int64_t q_stride, void* out, float* lse, palu_stream_t stream) {
  const palu_status_t st = check_pages_rows(h, pages, rows);
  if (st != PALU_OK) return st;
  const palu_kv_desc& d = h->d;
  if (d.dtype == PALU_F32) return PALU_ERR_UNSUPPORTED;
  if (rows->batch == 0 || rows->n_tokens == 0) return PALU_OK;
  if (bad_view(q, q_stride, d.n_heads, d.head_dim, d.dtype)) return PALU_ERR_INVALID_ARG;
  if (!out || (uintptr_t)out % 16 || (uintptr_t)lse % 4) return PALU_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return PALU_ERR_CUDA;
  KvAttendArgs a{};
  attend_args(h, *rows, q, q_stride, out, lse, a);
  a.pages = pages_of(*pages);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if ((int64_t)a.rows.max_new * a.g <= kKvFewRows) {
    // 16 query rows hold every row's tokens: the few-row kernel streams the cache once
    e = launch_kv_attend_few(a, h->sm_count, s);
  } else {
    // the gathers index cached head rows with 31 bits
    if (pages->n_pages * pages->page_size * d.n_kv_heads >= (int64_t(1) << 31) - 1) return PALU_ERR_UNSUPPORTED;
    e = launch_kv_attend_tc(a, tc_plan(h, *rows), s);
    if (e == cudaErrorNotSupported) return PALU_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PALU_OK : PALU_ERR_CUDA;
}

}  // extern "C"
