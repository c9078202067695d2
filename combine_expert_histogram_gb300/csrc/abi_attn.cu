// C ABI of the paged cache and its attention (declared in include/ep.h): argument
// validation and the launches.  Every host-detectable error returns before anything is
// enqueued.
#include <math.h>

#include "attn.cuh"

namespace ep {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ep_status_t check_head_dim(int32_t D) {
    if (D < 1) return EP_ERR_INVALID_ARG;
    return D == 64 || D == 128 ? EP_OK : EP_ERR_UNSUPPORTED;
}

ep_status_t check_cache(const ep_kv_cache_t *c) {
    if (!c || c->num_pages < 1 || c->page_size < 8 || c->page_size % 8 != 0 ||
        c->page_size > EP_KV_MAX_PAGE || c->num_kv_heads < 1 ||
        c->num_kv_heads > EP_ATTN_MAX_HEADS)
        return EP_ERR_INVALID_ARG;
    const ep_status_t st = check_head_dim(c->head_dim);
    if (st != EP_OK) return st;
    if (c->quant < EP_QUANT_NONE || c->quant > EP_QUANT_FP8_UE8M0_MN) return EP_ERR_INVALID_ARG;
    if (c->quant != EP_QUANT_NONE && c->quant != EP_QUANT_FP8_UE8M0) return EP_ERR_UNSUPPORTED;
    const int64_t unit = c->quant == EP_QUANT_NONE ? 2 : 1;
    for (const int64_t s : {c->page_stride, c->row_stride, c->head_stride})
        if (s <= 0 || s >= ((int64_t)1 << 40) / unit || s * unit % 16 != 0) return EP_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return EP_ERR_INVALID_ARG;
    if (c->quant == EP_QUANT_NONE) return c->k_scales || c->v_scales ? EP_ERR_INVALID_ARG : EP_OK;
    if (!c->k_scales || !c->v_scales || !aligned(c->k_scales, 8) || !aligned(c->v_scales, 8))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

ep_status_t check_seqs(const ep_kv_seqs_t *s, const ep_kv_cache_t *c) {
    if (!s || s->num_seqs < 0 || s->num_tokens < 0 || s->max_pages < 1 ||
        (int64_t)s->max_pages * c->page_size > EP_KV_MAX_LEN)
        return EP_ERR_INVALID_ARG;
    if (!s->q_start && s->num_tokens != s->num_seqs) return EP_ERR_INVALID_ARG;
    if (!s->status || !aligned(s->status, 4)) return EP_ERR_INVALID_ARG;
    if (s->num_seqs > 0 && (!s->block_table || !s->kv_len || !aligned(s->block_table, 4) ||
                            !aligned(s->kv_len, 4) || !aligned(s->q_start, 4)))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// A call without a row to work on.
bool no_rows(const ep_kv_seqs_t *s) { return s->num_seqs == 0 || s->num_tokens == 0; }

// Rows of `heads` heads, `stride` elements apart.
ep_status_t check_rows(const void *p, int64_t stride, int32_t heads, int32_t D) {
    if (!p || !aligned(p, 16) || stride < (int64_t)heads * D || stride % 8 != 0 ||
        stride >= (int64_t)1 << 40)
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

KvArgs kv_args(const ep_kv_cache_t *c) {
    const int64_t unit = c->quant == EP_QUANT_NONE ? 2 : 1;
    return {static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scales, c->v_scales,
            c->page_stride * unit, c->row_stride * unit, c->head_stride * unit,
            c->num_pages, c->page_size, c->num_kv_heads, c->head_dim};
}

SeqArgs seq_args(const ep_kv_seqs_t *s) {
    return {s->block_table, s->kv_len, s->q_start, s->status, s->num_seqs, s->num_tokens, s->max_pages};
}

ep_status_t check_heads(int32_t Hq, int32_t Hkv) {
    return Hq >= 1 && Hq <= EP_ATTN_MAX_HEADS && Hkv >= 1 && Hq % Hkv == 0 ? EP_OK
                                                                           : EP_ERR_INVALID_ARG;
}

// The rules that both forms of the attention share; `a` is filled in.
ep_status_t check_attn(const ep_kv_cache_t *c, const ep_kv_seqs_t *s, const void *q,
                       int64_t q_stride, int32_t Hq, float scale, int32_t window, int32_t sinks,
                       void *out, float *lse, AttnArgs *a) {
    ep_status_t st = check_cache(c);
    if (st != EP_OK) return st;
    st = check_seqs(s, c);
    if (st != EP_OK) return st;
    st = check_heads(Hq, c->num_kv_heads);
    if (st != EP_OK) return st;
    if (!(scale > 0.0f) || isinf(scale) || window < 0 || sinks < 0) return EP_ERR_INVALID_ARG;
    if ((int64_t)s->num_tokens * Hq > EP_ATTN_MAX_ROWS) return EP_ERR_INVALID_ARG;
    if (no_rows(s)) return EP_OK;
    if (check_rows(q, q_stride, Hq, c->head_dim) != EP_OK || !out || !aligned(out, 16) ||
        !aligned(lse, 4))
        return EP_ERR_INVALID_ARG;
    a->kv = kv_args(c);
    a->seq = seq_args(s);
    a->q = static_cast<const uint16_t *>(q);
    a->q_stride = q_stride;
    a->Hq = Hq;
    a->scale = scale;
    a->window = window > EP_KV_MAX_LEN ? 0 : window;  // all keys
    a->sinks = a->window ? (sinks < EP_KV_MAX_LEN ? sinks : EP_KV_MAX_LEN) : 0;
    a->out = static_cast<uint16_t *>(out);
    a->lse = lse;
    return EP_OK;
}

ep_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status_t ep_kv_append(const ep_kv_cache_t *c, const ep_kv_seqs_t *s, const void *q,
                         int64_t q_stride, int32_t Hq, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const float *cos_sin,
                         int32_t rotary_dim, int32_t positions, int32_t interleaved, void *q_out,
                         int64_t q_out_stride, ep_stream_t stream) {
    const TraceRange trace("ep_kv_append");
    ep_status_t st = check_cache(c);
    if (st != EP_OK) return st;
    st = check_seqs(s, c);
    if (st != EP_OK) return st;
    if (Hq < 0 || Hq > EP_ATTN_MAX_HEADS || positions < 0) return EP_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim % 16 != 0 || rotary_dim > c->head_dim) return EP_ERR_INVALID_ARG;
    if ((int64_t)s->num_tokens * (Hq + 2 * c->num_kv_heads) > EP_ATTN_MAX_ROWS) return EP_ERR_INVALID_ARG;
    if (no_rows(s)) return EP_OK;
    if (check_rows(k, k_stride, c->num_kv_heads, c->head_dim) != EP_OK ||
        check_rows(v, v_stride, c->num_kv_heads, c->head_dim) != EP_OK)
        return EP_ERR_INVALID_ARG;
    if (Hq == 0 ? q != nullptr || q_out != nullptr
                : check_rows(q, q_stride, Hq, c->head_dim) != EP_OK ||
                      check_rows(q_out, q_out_stride, Hq, c->head_dim) != EP_OK)
        return EP_ERR_INVALID_ARG;
    if (rotary_dim == 0 ? cos_sin != nullptr : !cos_sin || !aligned(cos_sin, 16))
        return EP_ERR_INVALID_ARG;
    return from_cuda(launch_kv_append(
        kv_args(c), seq_args(s), static_cast<const uint16_t *>(q), q_stride, Hq,
        static_cast<const uint16_t *>(k), k_stride, static_cast<const uint16_t *>(v), v_stride,
        cos_sin, rotary_dim, positions, interleaved != 0, static_cast<uint16_t *>(q_out),
        q_out_stride, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ep_attn_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
    if (B < 0 || check_heads(Hq, Hkv) != EP_OK || check_head_dim(D) != EP_OK) return 0;
    return attn_decode_workspace(B, Hq, Hkv, D);
}

ep_status_t ep_attn_decode(const ep_kv_cache_t *c, const ep_kv_seqs_t *s, const void *q,
                           int64_t q_stride, int32_t Hq, float scale, int32_t window,
                           int32_t sinks, void *out, float *lse, void *workspace,
                           size_t workspace_bytes, ep_stream_t stream) {
    const TraceRange trace("ep_attn_decode");
    AttnArgs a = {};
    const ep_status_t st = check_attn(c, s, q, q_stride, Hq, scale, window, sinks, out, lse, &a);
    if (st != EP_OK) return st;
    if (s->q_start) return EP_ERR_INVALID_ARG;  // one token a sequence
    if (no_rows(s)) return EP_OK;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < attn_decode_workspace(s->num_seqs, Hq, c->num_kv_heads, c->head_dim))
        return EP_ERR_INVALID_ARG;
    return from_cuda(launch_attn_decode(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ep_attn_prefill_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
    if (T < 0 || B < 0 || check_heads(Hq, Hkv) != EP_OK || check_head_dim(D) != EP_OK ||
        (int64_t)T * Hq > EP_ATTN_MAX_ROWS)
        return 0;
    return attn_prefill_workspace(D);
}

ep_status_t ep_attn_prefill(const ep_kv_cache_t *c, const ep_kv_seqs_t *s, const void *q,
                            int64_t q_stride, int32_t Hq, float scale, int32_t window,
                            int32_t sinks, void *out, float *lse, void *workspace,
                            size_t workspace_bytes, ep_stream_t stream) {
    const TraceRange trace("ep_attn_prefill");
    AttnArgs a = {};
    const ep_status_t st = check_attn(c, s, q, q_stride, Hq, scale, window, sinks, out, lse, &a);
    if (st != EP_OK || no_rows(s)) return st;
    if (workspace &&
        (!aligned(workspace, 16) ||
         workspace_bytes < attn_prefill_workspace(c->head_dim)))
        return EP_ERR_INVALID_ARG;
    return from_cuda(launch_attn_prefill(a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
