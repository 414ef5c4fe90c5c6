// Internal interface of the 8-bit paged KV cache's operators: the quantising append, the attention over codes, the plan of a
// step's rows and pages, and the verification of drafted tokens.
#pragma once

#include <cuda_fp8.h>

#include "kv.h"

namespace palu {

// further things that these operators record
constexpr unsigned kErrPool = 8;    // a pool whose ring or page counts do not add up
constexpr unsigned kErrToken = 9;   // a drafted token outside the vocabulary, or nothing to draw from

constexpr int kKv8Block = 16;       // slots that share a scale, for each head
constexpr float kKv8ScaleMin = 5.4210108624275222e-20f, kKv8ScaleMax = 1.8446744073709552e19f;   // 2^-64, 2^64

// two e4m3 codes as fp16, exactly (an fp16 number holds every one); the first in the low half
__device__ __forceinline__ uint32_t f16_of_codes(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// two values as e4m3 codes, nearest even, past 448 the largest; `a` in the low byte
__device__ __forceinline__ uint16_t codes_of(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// A cache's scale as the attention takes it: what is not positive and finite (a block without tokens) counts as 1.
__device__ __forceinline__ float scale_or_one(float s) { return s > 0.f && s < INFINITY ? s : 1.f; }

// log2 and reciprocal by the special function unit (absolute error 2^-22, relative 2^-23; normal arguments)
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// bf16 queries enter fp16 products lifted by a power of two that brings their row's largest magnitude into [2^14, 2^15): exact
// for elements down to 2^-28 of it, and to 2^-39 of it below. Rows of zeros, and of NaN or infinities, are not lifted.
__device__ __forceinline__ float lift_of(float top) {
  const int e = int(__float_as_uint(top) >> 23);                 // of a magnitude: biased exponent
  return e == 0 || e == 255 ? 1.f : __uint_as_float(uint32_t(min(227, max(1, 127 + 14 + 127 - e))) << 23);
}
__device__ __forceinline__ uint32_t lifted(uint32_t bf16x2, float lift) {
  const float a = __uint_as_float(bf16x2 << 16) * lift, b = __uint_as_float(bf16x2 & 0xffff0000u) * lift;
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What the scores of a row and a block are multiplied by: its part of the row (log2(e) / sqrt(d) without the lift) times s_k. A bf16
// row's part alone reaches from 2^-103 to 2^111, s_k from 2^-64 to 2^64. Their product is kept a normal number, as a masked
// score, -infinity, times zero and a score of zero times infinity would be NaN; what this moves are scores below 2^-90, and
// those whose factor fp32 does not hold. fp16 rows are not lifted and need no bounds. 2048 tokens at 65536 take 1604 us with
// them and 1588 without; with a branch around them, for rows that some s_k leads out of the range, 1609.
template <bool BF16> __device__ __forceinline__ float factor_of(float row, float s_k) {
  const float f = row * s_k;
  return BF16 ? fminf(fmaxf(f, 0x1p-126f), 0x1.fffffep127f) : f;
}

struct Kv8Pages {
  KvPages codes;
  float* scale[2];              // of keys and values
};

cudaError_t launch_kv8_append(const KvRopeArgs& a, const Kv8Pages& p, const KvFreq& f, int sm_count, cudaStream_t st);

struct Kv8AttendArgs {
  KvAttendArgs a;               // its pages are the codes
  const float* k_scale;
  const float* v_scale;
};
cudaError_t prepare_kv8_attend_few(int head_dim, bool bf16);
constexpr int kKv8FewRows = 24;   // query rows of a unit that the streaming kernel holds
cudaError_t launch_kv8_attend_few(const Kv8AttendArgs& a, int sm_count, cudaStream_t st);   // max_new g <= kKv8FewRows
cudaError_t prepare_kv8_attend_tc(int head_dim, bool bf16);
cudaError_t launch_kv8_attend_tc(const Kv8AttendArgs& a, const KvTcPlan& t, cudaStream_t st);

struct KvPlanArgs {
  int32_t* table;
  int64_t table_pages;
  const int32_t* held;
  int32_t* ring;
  const int32_t* state;
  int n_pages, page_size;
  const int32_t* fresh;         // new tokens, or negative: ended
  const int32_t* kv_len;
  int batch, n_tokens, max_new, max_kv_len;
  int32_t* row_start;
  int32_t* kv_len_out;
  int32_t* held_out;
  int32_t* state_out;
  int32_t* positions;
  int32_t* slots;
  ErrWord* err;
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t st);

struct KvVerifyArgs {
  const void* target;
  int64_t target_stride;
  const void* draft;            // nullptr: certain drafts
  int64_t draft_stride;
  int dtype, vocab;
  const int32_t* row_start;
  int batch, n_tokens;
  const int32_t* draft_tokens;
  int max_draft;
  const float* uniforms;
  int32_t* tokens;
  int32_t* accepted;
  const int32_t* kv_len;
  int32_t* kv_len_out;
  ErrWord* err;
};
cudaError_t launch_kv_verify(const KvVerifyArgs& a, int sm_count, cudaStream_t st);

}  // namespace palu
