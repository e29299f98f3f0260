// C ABI of the quantised key/value cache: argument checks, then one launch
// plan per call.  Nothing throws across the ABI.
#include <cstdint>

#include "fp8q.h"
#include "kv_device.cuh"

using namespace fp8q;

static bool kv_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The cache description itself; *s receives its shape.
static int check_cache(const mx_kv_cache* c, KvShape* s) {
  if (!c) return FP8Q_EINVAL;
  if (c->format != FP8Q_E4M3 && c->format != FP8Q_E5M2 && c->format != FP8Q_E2M1) return FP8Q_EDTYPE;
  if (c->kv_heads < 1 || c->kv_heads > MX_KV_MAX_HEADS || c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32 != 0)
    return FP8Q_EINVAL;
  if (c->page_size < 1 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)) != 0) return FP8Q_EINVAL;
  if (c->num_pages < 0 || c->num_pages > 0x7FFFFFFF) return FP8Q_EINVAL;
  if ((int64_t)c->kv_heads * c->page_size > 0x7FFFFFFF) return FP8Q_EINVAL;
  if (c->num_pages > 0 && (!c->k_q || !c->k_e8m0 || !c->v_q || !c->v_e8m0)) return FP8Q_EINVAL;
  if (!kv_aligned16(c->k_q) || !kv_aligned16(c->k_e8m0) || !kv_aligned16(c->v_q) || !kv_aligned16(c->v_e8m0))
    return FP8Q_EALIGN;
  s->page_shift = 0;
  while ((1 << s->page_shift) < c->page_size) ++s->page_shift;
  s->slots = c->num_pages << s->page_shift;
  s->pages = (int32_t)c->num_pages;
  s->page_rows = (uint32_t)(c->kv_heads * c->page_size);
  s->heads = c->kv_heads;
  s->dim = c->head_dim;
  return FP8Q_OK;
}

// Rows of a plain tensor: base and strides a multiple of 16 bytes.  The
// stride of a dimension of one element is not used.
static int check_rows(const void* x, int dtype, int64_t tokens, int64_t heads, int64_t tok, int64_t head) {
  if (!x) return FP8Q_EINVAL;
  const int64_t per = dtype == FP8Q_F32 ? 4 : 8;
  if (!kv_aligned16(x) || (tokens > 1 && tok % per != 0) || (heads > 1 && head % per != 0)) return FP8Q_EALIGN;
  return FP8Q_OK;
}

static int check_copy(const mx_kv_cache* c, const void* k, const void* v, int dtype, int64_t tokens,
                      int64_t k_tok, int64_t k_head, int64_t v_tok, int64_t v_head, const int64_t* slots,
                      KvShape* s) {
  int st = check_cache(c, s);
  if (st != FP8Q_OK) return st;
  if (dtype != FP8Q_F32 && dtype != FP8Q_BF16) return FP8Q_EDTYPE;
  if (tokens < 0 || tokens > 0x7FFFFFFF) return FP8Q_EINVAL;
  if (tokens == 0) return FP8Q_OK;
  if (!slots) return FP8Q_EINVAL;
  st = check_rows(k, dtype, tokens, c->kv_heads, k_tok, k_head);
  if (st != FP8Q_OK) return st;
  return check_rows(v, dtype, tokens, c->kv_heads, v_tok, v_head);
}

static int finish(cudaError_t e, int launches) {
  note_launches(launches);
  return e == cudaSuccess ? FP8Q_OK : record_cuda_error(e);
}

extern "C" {

FP8Q_API int mx_kv_write(const mx_kv_cache* c, const void* k, const void* v, int dtype, int64_t tokens,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                         int64_t v_head_stride, const int64_t* slots, int rule, void* stream) {
  FP8Q_TRACE_CALL();
  KvShape s;
  int st = check_copy(c, k, v, dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, &s);
  if (st != FP8Q_OK) return st;
  if (rule < FP8Q_MX_FLOOR || rule > FP8Q_MX_NEAREST) return FP8Q_EINVAL;
  if (tokens == 0) return FP8Q_OK;
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  int launches = 0;
  const cudaError_t e = launch_kv_write(s, c->format, {c->k_q, c->k_e8m0}, {c->v_q, c->v_e8m0}, k, v, dtype, tokens,
                                        strides, slots, rule, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

FP8Q_API int mx_kv_read(const mx_kv_cache* c, const int64_t* slots, int64_t tokens, void* k, void* v, int dtype,
                        int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                        int64_t v_head_stride, void* stream) {
  FP8Q_TRACE_CALL();
  KvShape s;
  int st = check_copy(c, k, v, dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, &s);
  if (st != FP8Q_OK) return st;
  if (tokens == 0) return FP8Q_OK;
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  int launches = 0;
  const cudaError_t e = launch_kv_read(s, c->format, {c->k_q, c->k_e8m0}, {c->v_q, c->v_e8m0}, k, v, dtype, tokens,
                                       strides, slots, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

// The shape checks that the attention call and its workspace query share.
static int check_attention(const mx_kv_cache* c, int64_t total_q, int q_heads, int batch, int max_q, int table_width,
                           KvShape* s) {
  int st = check_cache(c, s);
  if (st != FP8Q_OK) return st;
  if (c->format != FP8Q_E2M1) return FP8Q_EDTYPE;
  if (c->head_dim != 64 && c->head_dim != 128) return FP8Q_EINVAL;
  if (q_heads < 1 || q_heads > MX_KV_MAX_HEADS || q_heads % c->kv_heads != 0) return FP8Q_EINVAL;
  if (total_q < 0 || total_q > 0x7FFFFFFF / q_heads || batch < 0 || batch > 65535) return FP8Q_EINVAL;
  if (max_q < 1 || table_width < 1) return FP8Q_EINVAL;
  if (((int64_t)table_width << s->page_shift) > 0x7FFFFFFF / 2) return FP8Q_EINVAL;
  return FP8Q_OK;
}

FP8Q_API int64_t mx_kv_attention_workspace(const mx_kv_cache* c, int64_t total_q, int q_heads, int batch, int max_q,
                                           int table_width) {
  FP8Q_TRACE_CALL();
  KvShape s;
  int st = check_attention(c, total_q, q_heads, batch, max_q, table_width, &s);
  if (st != FP8Q_OK) return st;
  if (total_q == 0 || batch == 0) return 0;
  if (max_q > total_q) max_q = (int)total_q;
  int64_t bytes = 0;
  try {                            // the occupancy cache allocates
    const cudaError_t e = kv_attention_workspace(s, q_heads, batch, total_q, max_q, table_width,
                                                 sm_count(device_of_current()), &bytes);
    return e == cudaSuccess ? bytes : record_cuda_error(e);
  } catch (...) {
    return FP8Q_ENOMEM;
  }
}

FP8Q_API int mx_kv_attention(const mx_kv_cache* c, const void* q, int dtype, int64_t total_q, int q_heads,
                             int64_t q_token_stride, int64_t q_head_stride, void* out, int64_t out_token_stride,
                             int64_t out_head_stride, float* lse, const int32_t* cu_q, const int32_t* kv_lens,
                             const int32_t* page_table, int64_t table_stride, int table_width, int batch, int max_q,
                             float scale, int window, void* workspace, int64_t workspace_bytes, void* stream) {
  FP8Q_TRACE_CALL();
  KvAttn a;
  int st = check_attention(c, total_q, q_heads, batch, max_q, table_width, &a.shape);
  if (st != FP8Q_OK) return st;
  if (dtype != FP8Q_BF16) return FP8Q_EDTYPE;
  if (window < 0 || !(scale > 0.0f) || scale > 3.0e38f || (batch > 1 && table_stride < table_width)) return FP8Q_EINVAL;
  if (!cu_q && (total_q != batch || max_q != 1)) return FP8Q_EINVAL;
  if (total_q == 0 || batch == 0) return FP8Q_OK;
  if (!kv_lens || !page_table || workspace_bytes < 0) return FP8Q_EINVAL;
  st = check_rows(q, dtype, total_q, q_heads, q_token_stride, q_head_stride);
  if (st == FP8Q_OK) st = check_rows(out, dtype, total_q, q_heads, out_token_stride, out_head_stride);
  if (st != FP8Q_OK) return st;
  if (max_q > total_q) max_q = (int)total_q;
  a.k = {c->k_q, c->k_e8m0};
  a.v = {c->v_q, c->v_e8m0};
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.table = page_table;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.out_tok = out_token_stride;
  a.out_head = out_head_stride;
  a.table_stride = table_stride;
  a.table_width = table_width;
  a.batch = batch;
  a.total_q = (int32_t)total_q;
  a.max_q = max_q;
  a.q_heads = q_heads;
  a.group = q_heads / c->kv_heads;
  a.by_group = FastDiv((uint32_t)a.group);
  a.window = window > 0x3FFFFFFF ? 0 : window;   // no sequence is that long
  a.scale = scale;
  int launches = 0;
  cudaError_t e;
  try {                            // the occupancy cache allocates
    e = launch_kv_attention(a, {workspace, workspace_bytes}, sm_count(device_of_current()),
                            reinterpret_cast<cudaStream_t>(stream), &st, &launches);
  } catch (...) {
    return FP8Q_ENOMEM;
  }
  if (st != FP8Q_OK) return st;
  return finish(e, launches);
}

}  // extern "C"
