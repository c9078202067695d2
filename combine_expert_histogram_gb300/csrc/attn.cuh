// What the paged cache's kernels share: their arguments, the visible keys of a
// query, the cache's addresses.
#pragma once

#include "ep_common.cuh"
#include "fp8.cuh"

namespace ep {

// The cache, checked by the C ABI.  Strides in bytes.
struct KvArgs {
    uint8_t *k, *v;              // bf16 or E4M3
    uint8_t *k_scales, *v_scales;  // E8M0 [pages, Hkv, page_size]; nullptr: bf16 rows
    int64_t page_stride, row_stride, head_stride;
    int pages, page_size, Hkv, D;
};

// The sequences.
struct SeqArgs {
    const int32_t *table;    // [B, max_pages]
    const int32_t *kv_len;   // [B]
    const int32_t *q_start;  // [B+1], or nullptr: token b is sequence b's
    int32_t *status;
    int B, T, max_pages;
};

struct AttnArgs {
    KvArgs kv;
    SeqArgs seq;
    const uint16_t *q;  // bf16 [T, Hq, D], tokens q_stride elements apart
    int64_t q_stride;
    int Hq;
    float scale;
    int window, sinks;  // window 0: none
    uint16_t *out;      // bf16 [T, Hq, D]
    float *lse;         // [T, Hq] or nullptr
};

// Tokens of sequence b among the call's rows, and its length, which may be past the table; both
// are whatever the device arrays hold, brought into range.
struct Span {
    int first, n, len;
};
__device__ __forceinline__ Span seq_rows(const SeqArgs &s, int b) {
    Span r;
    r.len = max(ld_dep(s.kv_len + b), 0);
    if (s.q_start) {
        r.first = min(max(ld_dep(s.q_start + b), 0), s.T);
        r.n = min(max(ld_dep(s.q_start + b + 1), r.first), s.T) - r.first;
    } else {
        r.first = b;
        r.n = 1;
    }
    return r;
}
// The same for the attention: a length past the table raises EP_ERR_BAD_PAGE and counts as the table's.
__device__ __forceinline__ Span seq_span(const SeqArgs &s, int page_size, int b) {
    Span r = seq_rows(s, b);
    const int most = s.max_pages * page_size;
    if (r.len > most) {
        raise_status(s.status, EP_ERR_BAD_PAGE);
        r.len = most;
    }
    return r;
}

// Sequence of token t, or -1: the last b with q_start[b] <= t, if t is its.
__device__ __forceinline__ int seq_of(const SeqArgs &s, int t) {
    if (!s.q_start) return t < s.B ? t : -1;
    int lo = 0, hi = s.B;  // q_start[lo] <= t < q_start[hi], if t is any sequence's
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ld_dep(s.q_start + mid) <= t) lo = mid; else hi = mid;
    }
    return s.B > 0 && ld_dep(s.q_start + lo) <= t && t < ld_dep(s.q_start + lo + 1) ? lo : -1;
}

// The page of a table's entry, -1 (and EP_ERR_BAD_PAGE) if the cache has no such page.
__device__ __forceinline__ int page_of(const KvArgs &kv, const SeqArgs &s, int b, int entry) {
    const int p = ld_dep(s.table + (int64_t)b * s.max_pages + entry);
    if ((unsigned)p < (unsigned)kv.pages) return p;
    raise_status(s.status, EP_ERR_BAD_PAGE);
    return -1;
}

// ld_dep_v4 where `there`, else zeros, without a branch: one would wait for each load where
// its two ways meet.
__device__ __forceinline__ uint4 ld_dep_v4_if(bool there, const void *p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)there)
        : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_dep_if(bool there, const void *p) {
    uint32_t v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t@p ld.global.u32 %0, [%1];\n\t}"
        : "=&r"(v)
        : "l"(p), "r"((uint32_t)there)
        : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_byte_if(bool there, const void *p, uint32_t otherwise) {
    uint32_t v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t@p ld.global.u8 %0, [%1];\n\t}"
        : "=&r"(v)
        : "l"(p), "r"((uint32_t)there), "r"(otherwise)
        : "memory");
    return v;
}

// Four E4M3 values -> two pairs of fp16, exactly.
__device__ __forceinline__ void half_pairs(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

cudaError_t launch_kv_append(const KvArgs &kv, const SeqArgs &seq, const uint16_t *q,
                             int64_t q_stride, int Hq, const uint16_t *k, int64_t k_stride,
                             const uint16_t *v, int64_t v_stride, const float *cos_sin, int R,
                             int positions, bool interleaved, uint16_t *q_out,
                             int64_t q_out_stride, cudaStream_t stream);
cudaError_t launch_attn_decode(const AttnArgs &a, void *workspace, cudaStream_t stream);
size_t attn_decode_workspace(int B, int Hq, int Hkv, int D);
// workspace may be nullptr.
cudaError_t launch_attn_prefill(const AttnArgs &a, void *workspace, cudaStream_t stream);
size_t attn_prefill_workspace(int D);

}  // namespace ep
