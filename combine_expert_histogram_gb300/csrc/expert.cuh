// What the expert kernels share: which rows of a layout belong to an expert,
// and the scale of a row's 1x128 group in each quantisation mode.
#pragma once

#include "ep_common.cuh"
#include "fp8.cuh"

namespace ep {

// Arguments of the experts' products, by value into the kernels.
struct ExpertArgs {
    const int32_t *count;   // [E] rows requested per expert
    const int32_t *offset;  // [E+1] first row (contiguous layout)
    int E;
    int cap;                // masked: slots per expert; 0: contiguous layout
    int rows_cap;           // rows of the row space
    const uint8_t *x;       // [rows_cap, K] E4M3
    const void *x_scales;   // by `quant`
    int quant;              // EP_QUANT_FP8_F32, _UE8M0 or _UE8M0_MN
    int K;
    const uint8_t *w;       // [E, N, K] E4M3 (N = 2I with the gated SiLU)
    const float *w_scales;  // [E, ceil(N/128), K/128]
    int N;                  // columns of the output (I with the gated SiLU)
    void *out;              // bf16 or E4M3 [rows_cap, N]
    void *out_scales;
    int out_quant;
    int32_t *status;
};

// Arguments of the few-token layer.
struct MoeArgs {
    const void *x;            // [T, H] bf16, or E4M3 with x_scales
    const void *x_scales;
    int quant;
    const int32_t *topk_idx;  // [T, K]
    const float *topk_w;
    int T, K, E, H, I;
    const uint8_t *w13;       // [E, 2I, H]
    const float *w13_scales;  // [E, 2I/128, H/128]
    const uint8_t *w2;        // [E, H, I]
    const float *w2_scales;   // [E, H/128, I/128]
    void *out;                // bf16 [T, H]
    int32_t *status;
};
// Bytes of scratch for exactly T tokens, and for any number up to T.
size_t moe_workspace_bytes(int T, int K, int E, int H, int I);
size_t moe_workspace_bytes_up_to(int T, int K, int E, int H, int I);
cudaError_t launch_moe_decode(const MoeArgs &a, void *workspace, cudaStream_t stream);
cudaError_t launch_expert(const ExpertArgs &a, bool gated, cudaStream_t stream);

// silu(g) * u = g / (1 + exp(-g)) * u by the fast exponential and division.  The
// first is off by at most 2 + 1.173 |g| units in the last place, the second by 2, so
// the result is within (11 + 2.4 |g|) 2^-24 of the formula: below half a step of
// bf16 and E4M3 for any |g| whose exponential is finite.  Where 1 + exp(-g) is above
// 2^126 (g < -87.3) the division gives 0; there |silu(g)| < 2^-119.  (expf and the
// rounded division, whose slow path is a call across 128 live sums, took the prompt
// case of ep_expert_swiglu from 3.6 to 4.7 ms, the few-token layer from 16.6 to 17.2 us.)
__device__ __forceinline__ float gated_silu(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// Rows of expert e: [first, first + n).  Clamped into the row space, so a
// layout whose arrays were never filled addresses nothing outside it.
__device__ __forceinline__ int expert_first(const ExpertArgs &a, int e) {
    return a.cap ? e * a.cap : min(max(ld_dep(a.offset + e), 0), a.rows_cap);
}
__device__ __forceinline__ int expert_rows(const ExpertArgs &a, int e) {
    const int n = max(ld_dep(a.count + e), 0);
    return a.cap ? min(n, a.cap) : min(n, a.rows_cap - expert_first(a, e));
}

// Scales of groups g .. g+3 of row r (row r belongs to expert e; g a multiple of
// 4; groups past the last one get anything).  The packed forms are one word.
__device__ __forceinline__ float4 row_scales4(const ExpertArgs &a, int r, int e, int g) {
    const int G = a.K >> 7, P = (G + 3) >> 2;
    if (a.quant == EP_QUANT_FP8_F32) {
        const float *p = static_cast<const float *>(a.x_scales) + (size_t)r * G + g;
        if ((G & 3) == 0 && (reinterpret_cast<uintptr_t>(a.x_scales) & 15) == 0) {
            const uint4 v = ld_dep_v4(p);
            return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                               __uint_as_float(v.w));
        }
        const int last = G - 1 - g;
        return make_float4(ld_dep(p), ld_dep(p + min(1, last)), ld_dep(p + min(2, last)),
                           ld_dep(p + min(3, last)));
    }
    size_t word;
    if (a.quant == EP_QUANT_FP8_UE8M0) {
        word = (size_t)r * P + (g >> 2);
    } else if (a.cap) {
        const int stride = (a.cap + 3) / 4 * 4;
        word = ((size_t)e * P + (g >> 2)) * stride + (r - e * a.cap);
    } else {
        word = (size_t)(g >> 2) * ((a.rows_cap + 3ll) / 4 * 4) + r;
    }
    const uint32_t v = (uint32_t)ld_dep(static_cast<const int32_t *>(a.x_scales) + word);
    return make_float4(ue8m0_value(v & 255u), ue8m0_value(v >> 8 & 255u),
                       ue8m0_value(v >> 16 & 255u), ue8m0_value(v >> 24));
}

// Store the scale of group g of output row r: fp32, or the biased exponent e8
// as byte g%4 of word g/4 (the last group also fills its word with 127 = 2^0).
__device__ __forceinline__ void store_out_scale(const ExpertArgs &a, int r, int e, int g, float s,
                                                int e8) {
    const int G = a.N >> 7, P = (G + 3) >> 2;
    if (a.out_quant == EP_QUANT_FP8_F32) {
        static_cast<float *>(a.out_scales)[(size_t)r * G + g] = s;
        return;
    }
    const int last = g == G - 1 ? (g | 3) : g;
    for (int b = g; b <= last; ++b) {
        size_t word;
        if (a.out_quant == EP_QUANT_FP8_UE8M0)
            word = (size_t)r * P + (b >> 2);
        else if (a.cap)
            word = ((size_t)e * P + (b >> 2)) * ((a.cap + 3) / 4 * 4) + (r - e * a.cap);
        else
            word = (size_t)(b >> 2) * ((a.rows_cap + 3ll) / 4 * 4) + r;
        static_cast<uint8_t *>(a.out_scales)[word * 4 + (b & 3)] = (uint8_t)(b == g ? e8 : 127);
    }
}

}  // namespace ep
