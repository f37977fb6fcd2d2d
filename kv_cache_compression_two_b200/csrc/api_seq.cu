// api_seq.cu -- the extern "C" entry points of the sequence calls: the
// quantised paged cache and attention over it and over packed prompts.
#include <math.h>

#include "kvq.cuh"

using namespace ispa;

namespace {

bool half_type(ispa_dtype d) { return d == ISPA_BF16 || d == ISPA_F16; }

ispa_status check_cache(const ispa_kvq_desc *d) {
  if (!d) return fail(ISPA_ERR_INVALID_ARG, "desc is NULL");
  if (d->H_kv < 1 || d->n_pages < 1) return fail(ISPA_ERR_INVALID_ARG, "H_kv and n_pages must be >= 1");
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(ISPA_ERR_INVALID_ARG, "head_dim must be 64 or 128 (got %d)", d->head_dim);
  if (kvq_log2(d->page_tokens) < 0 || d->page_tokens != 1 << kvq_log2(d->page_tokens))
    return fail(ISPA_ERR_INVALID_ARG, "page_tokens must be 16, 32, 64, 128 or 256 (got %d)", d->page_tokens);
  if (d->fmt != ISPA_KVQ_E4M3 && d->fmt != ISPA_KVQ_INT8 && d->fmt != ISPA_KVQ_INT4)
    return fail(ISPA_ERR_INVALID_ARG, "bad cache format");
  if (d->H_kv > (1 << 16) || (long long)d->n_pages * d->H_kv > (1LL << 32))
    return fail(ISPA_ERR_INVALID_ARG, "cache too large");
  return ISPA_OK;
}

ispa_status check_table(int B, const int *table, int max_pages, int page_tokens) {
  if (B < 1) return fail(ISPA_ERR_INVALID_ARG, "B must be >= 1");
  if (max_pages < 1 || (long long)max_pages * page_tokens > (1LL << 30))
    return fail(ISPA_ERR_INVALID_ARG, "max_pages must be >= 1 and cover at most 2^30 tokens");
  if (!table) return fail(ISPA_ERR_INVALID_ARG, "block_table is required");
  return ISPA_OK;
}

bool int_ptr_ok(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool row_ptr_ok(const void *p) { return p != nullptr && aligned16(p); }

// A row stride in elements: whole 16-byte steps, and rows that do not overlap.
bool stride_ok(long long stride, int heads, int d) {
  return stride >= (long long)heads * d && stride % 8 == 0 && stride <= (1LL << 30);
}

ispa_status check_attn(const ispa_attn_seq_desc *d, float *scale) {
  if (!d) return fail(ISPA_ERR_INVALID_ARG, "desc is NULL");
  if (d->B < 1 || d->H < 1 || d->H_kv < 1) return fail(ISPA_ERR_INVALID_ARG, "B, H and H_kv must be >= 1");
  if (d->H % d->H_kv != 0) return fail(ISPA_ERR_INVALID_ARG, "H (%d) must be a multiple of H_kv (%d)", d->H, d->H_kv);
  if (d->H / d->H_kv > 128) return fail(ISPA_ERR_INVALID_ARG, "H / H_kv must be at most 128");
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(ISPA_ERR_INVALID_ARG, "head_dim must be 64 or 128 (got %d)", d->head_dim);
  if (d->in_dtype == ISPA_F32) return fail(ISPA_ERR_UNSUPPORTED, "the sequence attentions take bf16 or fp16 inputs");
  if (!half_type(d->in_dtype)) return fail(ISPA_ERR_INVALID_ARG, "bad in_dtype");
  if (d->out_dtype != d->in_dtype && d->out_dtype != ISPA_F32)
    return fail(ISPA_ERR_INVALID_ARG, "out_dtype must be in_dtype or ISPA_F32");
  if (d->causal != 0 && d->causal != 1) return fail(ISPA_ERR_INVALID_ARG, "causal must be 0 or 1");
  *scale = d->softmax_scale <= 0.f ? 1.f / sqrtf((float)d->head_dim) : d->softmax_scale;
  if (!isfinite(*scale)) return fail(ISPA_ERR_INVALID_ARG, "softmax_scale must be finite");
  return ISPA_OK;
}

ispa_status check_rows(int T, long long heads, int d) {
  if (T < 0 || (long long)T * heads * d > (1LL << 40) || (long long)T * ((heads + 3) / 4) > (1LL << 33))
    return fail(ISPA_ERR_INVALID_ARG, "the number of rows must be >= 0 (or the tensor is too large)");
  return ISPA_OK;
}

}  // namespace

extern "C" {

size_t ispa_kvq_bytes(const ispa_kvq_desc *desc) {
  if (check_cache(desc) != ISPA_OK) return 0;
  return kvq_layout(*desc).bytes;
}

ispa_status ispa_kvq_write(const ispa_kvq_desc *desc, int B, int T, const int *block_table, int max_pages,
                           const int *seq_lens, const int *cu_new, const void *k, long long k_stride, const void *v,
                           long long v_stride, ispa_dtype in_dtype, void *kvq, ispa_stream_t stream) {
  ispa_status st = check_cache(desc);
  if (st == ISPA_OK) st = check_table(B, block_table, max_pages, desc->page_tokens);
  if (st == ISPA_OK) st = check_rows(T, desc->H_kv, desc->head_dim);
  if (st != ISPA_OK) return st;
  if (!half_type(in_dtype)) return fail(ISPA_ERR_INVALID_ARG, "in_dtype must be ISPA_BF16 or ISPA_F16");
  if (!int_ptr_ok(block_table) || !int_ptr_ok(seq_lens) || !int_ptr_ok(cu_new))
    return fail(ISPA_ERR_INVALID_ARG, "block_table, seq_lens and cu_new must be int32 device arrays");
  if (!stride_ok(k_stride, desc->H_kv, desc->head_dim) || !stride_ok(v_stride, desc->H_kv, desc->head_dim))
    return fail(ISPA_ERR_INVALID_ARG, "k_stride and v_stride must be multiples of 8, at least H_kv * head_dim");
  if (T == 0) return ISPA_OK;
  if (!row_ptr_ok(k) || !row_ptr_ok(v) || !row_ptr_ok(kvq))
    return fail(ISPA_ERR_INVALID_ARG, "k, v and kvq must be 16-byte aligned device pointers");
  return launch_kvq_write(*desc, B, T, block_table, max_pages, seq_lens, cu_new, k, k_stride, v, v_stride, in_dtype,
                          kvq, (cudaStream_t)stream);
}

ispa_status ispa_kvq_read(const ispa_kvq_desc *desc, int B, int T, const int *block_table, int max_pages,
                          const int *seq_begin, const int *cu_out, const void *kvq, void *k_out, void *v_out,
                          ispa_dtype out_dtype, ispa_stream_t stream) {
  ispa_status st = check_cache(desc);
  if (st == ISPA_OK) st = check_table(B, block_table, max_pages, desc->page_tokens);
  if (st == ISPA_OK) st = check_rows(T, desc->H_kv, desc->head_dim);
  if (st != ISPA_OK) return st;
  if (!half_type(out_dtype)) return fail(ISPA_ERR_INVALID_ARG, "out_dtype must be ISPA_BF16 or ISPA_F16");
  if (!int_ptr_ok(block_table) || !int_ptr_ok(cu_out) || (seq_begin && !int_ptr_ok(seq_begin)))
    return fail(ISPA_ERR_INVALID_ARG, "block_table, cu_out and seq_begin must be int32 device arrays");
  if (T == 0) return ISPA_OK;
  if (!row_ptr_ok(k_out) || !row_ptr_ok(v_out) || !row_ptr_ok(kvq))
    return fail(ISPA_ERR_INVALID_ARG, "kvq, k_out and v_out must be 16-byte aligned device pointers");
  return launch_kvq_read(*desc, B, T, block_table, max_pages, seq_begin, cu_out, kvq, k_out, v_out, out_dtype,
                         (cudaStream_t)stream);
}

size_t ispa_attn_kvq_workspace_bytes(const ispa_attn_seq_desc *desc, const ispa_kvq_desc *cache) {
  float scale;
  if (check_attn(desc, &scale) != ISPA_OK || check_cache(cache) != ISPA_OK) return 0;
  return attn_kvq_workspace_bytes(desc->head_dim);
}

ispa_status ispa_attn_kvq(const ispa_attn_seq_desc *desc, const ispa_kvq_desc *cache, int T, const int *cu_q,
                          const int *block_table, int max_pages, const int *seq_lens, const void *q,
                          long long q_stride, const void *kvq, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, ispa_stream_t stream) {
  float scale;
  ispa_status st = check_attn(desc, &scale);
  if (st == ISPA_OK) st = check_cache(cache);
  if (st == ISPA_OK) st = check_table(desc->B, block_table, max_pages, cache->page_tokens);
  if (st == ISPA_OK) st = check_rows(T, desc->H, desc->head_dim);
  if (st != ISPA_OK) return st;
  if (cache->H_kv != desc->H_kv || cache->head_dim != desc->head_dim)
    return fail(ISPA_ERR_INVALID_ARG, "the cache has %d heads of %d, the attention %d of %d", cache->H_kv,
                cache->head_dim, desc->H_kv, desc->head_dim);
  if (!int_ptr_ok(block_table) || !int_ptr_ok(seq_lens) || !int_ptr_ok(cu_q))
    return fail(ISPA_ERR_INVALID_ARG, "block_table, seq_lens and cu_q must be int32 device arrays");
  if (!stride_ok(q_stride, desc->H, desc->head_dim))
    return fail(ISPA_ERR_INVALID_ARG, "q_stride must be a multiple of 8, at least H * head_dim");
  if (T == 0) return ISPA_OK;
  if (!row_ptr_ok(q) || !row_ptr_ok(kvq) || !row_ptr_ok(o) || (lse && !int_ptr_ok(lse)))
    return fail(ISPA_ERR_INVALID_ARG, "q, kvq and o must be 16-byte aligned device pointers");
  const size_t need = attn_kvq_workspace_bytes(desc->head_dim);
  if (!row_ptr_ok(workspace) || workspace_bytes < need)
    return fail(ISPA_ERR_INVALID_ARG, "workspace needs %zu bytes (16-byte aligned)", need);
  return launch_attn_kvq(*desc, *cache, scale, T, cu_q, block_table, max_pages, seq_lens, q, q_stride, kvq, o, lse,
                         workspace, (cudaStream_t)stream);
}

size_t ispa_attn_prompt_workspace_bytes(const ispa_attn_seq_desc *desc) {
  float scale;
  if (check_attn(desc, &scale) != ISPA_OK) return 0;
  return attn_prompt_workspace_bytes(desc->head_dim);
}

ispa_status ispa_attn_prompt(const ispa_attn_seq_desc *desc, int Tq, int Tk, const int *cu_q, const int *cu_k,
                             const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                             long long v_stride, void *o, float *lse, void *workspace, size_t workspace_bytes,
                             ispa_stream_t stream) {
  float scale;
  ispa_status st = check_attn(desc, &scale);
  if (st == ISPA_OK) st = check_rows(Tq, desc->H, desc->head_dim);
  if (st == ISPA_OK) st = check_rows(Tk, desc->H_kv, desc->head_dim);
  if (st != ISPA_OK) return st;
  if (!int_ptr_ok(cu_q) || !int_ptr_ok(cu_k))
    return fail(ISPA_ERR_INVALID_ARG, "cu_q and cu_k must be int32 device arrays");
  if (!stride_ok(q_stride, desc->H, desc->head_dim) || !stride_ok(k_stride, desc->H_kv, desc->head_dim) ||
      !stride_ok(v_stride, desc->H_kv, desc->head_dim))
    return fail(ISPA_ERR_INVALID_ARG, "row strides must be multiples of 8, at least heads * head_dim");
  if (Tq == 0) return ISPA_OK;
  if (!row_ptr_ok(q) || !row_ptr_ok(o) || (lse && !int_ptr_ok(lse)) || (Tk > 0 && (!row_ptr_ok(k) || !row_ptr_ok(v))))
    return fail(ISPA_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned device pointers");
  const size_t need = attn_prompt_workspace_bytes(desc->head_dim);
  if (!row_ptr_ok(workspace) || workspace_bytes < need)
    return fail(ISPA_ERR_INVALID_ARG, "workspace needs %zu bytes (16-byte aligned)", need);
  return launch_attn_prompt(*desc, scale, Tq, Tk, cu_q, cu_k, q, q_stride, k, k_stride, v, v_stride, o, lse, workspace,
                            (cudaStream_t)stream);
}

}  // extern "C"
