// ep_moe_decode: a whole mixture-of-experts layer for a few tokens.
//
//   xq = 1x128 E4M3 of x,  g = W13[e][:I] xq,  u = W13[e][I:] xq,
//   hq = 1x128 E4M3 of silu(g) * u,  out[t] = sum over k of w[t,k] * W2[e] hq
//
// One warp per output: the 128 products of a block are summed by the warp and
// scaled into the running sum.
#include <cuda_bf16.h>

#include "expert.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;

// E4M3 bytes and fp32 scales of 1x128 groups, one warp per group.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    quantise_kernel(const void *src, int groups, uint8_t *q, float *s) {
    const int lane = threadIdx.x & 31;
    const int g = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (g >= groups) return;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t at = (size_t)g * 128 + 4 * lane + i;
        v[i] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(src)[at])
                    : static_cast<const float *>(src)[at];
    }
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
    const float sc = group_scale(amax);
    reinterpret_cast<uint32_t *>(q)[(size_t)g * 32 + lane] =
        fp8x4(__fdiv_rn(v[0], sc), __fdiv_rn(v[1], sc), __fdiv_rn(v[2], sc), __fdiv_rn(v[3], sc));
    if (lane == 0) s[g] = sc;
}

// fp32 scales of G groups a row from packed UE8M0 words.
__global__ void __launch_bounds__(kThreads)
    unpack_scales_kernel(const uint32_t *words, int rows, int G, float *s) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= rows * G) return;
    const int g = i % G;
    s[i] = ue8m0_value(words[(size_t)(i / G) * ((G + 3) / 4) + (g >> 2)] >> (8 * (g & 3)) & 255u);
}

// Block-scaled dot product of two E4M3 rows of K elements, by one warp.
__device__ float block_dot(const uint8_t *x, const float *sx, const uint8_t *w, const float *sw,
                           int K) {
    const int lane = threadIdx.x & 31;
    float acc = 0.0f;
    for (int g = 0; g < K / 128; ++g) {
        const float4 a = e4m3x4_to_float4(reinterpret_cast<const uint32_t *>(x)[g * 32 + lane]);
        const float4 b = e4m3x4_to_float4(reinterpret_cast<const uint32_t *>(w)[g * 32 + lane]);
        const float d = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
        acc = fmaf(d, sx[g] * sw[g], acc);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) acc += __shfl_xor_sync(kFullMask, acc, d);
    return acc;
}

__global__ void __launch_bounds__(kThreads) up_kernel(const MoeArgs a, const uint8_t *xq,
                                                      const float *xs, float *h) {
    const long long o = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int entry = (int)(o / a.I), i = (int)(o % a.I), t = entry / a.K;
    if (entry >= a.T * a.K) return;
    const int e = a.topk_idx[entry];
    float v = 0.0f;
    if (e >= 0 && e < a.E) {
        const int G = a.H >> 7, NB = a.I / 64;
        const float *sw = a.w13_scales + (size_t)e * NB * G;
        const uint8_t *w = a.w13 + (size_t)e * 2 * a.I * a.H;
        const float g = block_dot(xq + (size_t)t * a.H, xs + t * G, w + (size_t)i * a.H,
                                  sw + (size_t)(i / 128) * G, a.H);
        const float u = block_dot(xq + (size_t)t * a.H, xs + t * G, w + (size_t)(a.I + i) * a.H,
                                  sw + (size_t)((a.I + i) / 128) * G, a.H);
        v = g / (1.0f + expf(-g)) * u;
    } else if (e != -1 && i == 0 && (threadIdx.x & 31) == 0) {
        raise_status(a.status, EP_ERR_BAD_EXPERT_ID);
    }
    if ((threadIdx.x & 31) == 0) h[(size_t)entry * a.I + i] = v;
}

__global__ void __launch_bounds__(kThreads) down_kernel(const MoeArgs a, const uint8_t *hq,
                                                        const float *hs) {
    const long long o = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(o / a.H), n = (int)(o % a.H);
    if (t >= a.T) return;
    const int G = a.I >> 7, NB = a.H >> 7;
    float acc = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int entry = t * a.K + k, e = a.topk_idx[entry];
        if (e < 0 || e >= a.E) continue;
        const float y = block_dot(hq + (size_t)entry * a.I, hs + (size_t)entry * G,
                                  a.w2 + ((size_t)e * a.H + n) * a.I,
                                  a.w2_scales + ((size_t)e * NB + n / 128) * G, a.I);
        acc = fmaf(a.topk_w[entry], y, acc);
    }
    if ((threadIdx.x & 31) == 0) static_cast<__nv_bfloat16 *>(a.out)[(size_t)t * a.H + n] = __float2bfloat16_rn(acc);
}

}  // namespace

size_t moe_workspace_bytes(int T, int K, int H, int I) {
    const size_t n = (size_t)T * K;
    return n * I * 4 + n * I + n * (I / 128) * 4 + (size_t)T * H + (size_t)T * (H / 128) * 4;
}

cudaError_t launch_moe_decode(const MoeArgs &a, void *workspace, cudaStream_t stream) {
    const int n = a.T * a.K;
    float *h = static_cast<float *>(workspace);
    float *hs = h + (size_t)n * a.I;
    float *xs = hs + (size_t)n * (a.I / 128);
    uint8_t *hq = reinterpret_cast<uint8_t *>(xs + (size_t)a.T * (a.H / 128));
    uint8_t *xq = hq + (size_t)n * a.I;
    const int per = kThreads / 32;
    cudaError_t err = cudaMemsetAsync(a.status, 0, 4, stream);
    if (err != cudaSuccess) return err;
    const int gx = a.T * (a.H / 128), gh = n * (a.I / 128);
    const uint8_t *q = static_cast<const uint8_t *>(a.x);
    const float *s = static_cast<const float *>(a.x_scales);
    if (a.quant == EP_QUANT_NONE) {
        quantise_kernel<true><<<(gx + per - 1) / per, kThreads, 0, stream>>>(a.x, gx, xq, xs);
        q = xq;
        s = xs;
    } else if (a.quant == EP_QUANT_FP8_UE8M0) {
        unpack_scales_kernel<<<(gx + kThreads - 1) / kThreads, kThreads, 0, stream>>>(
            static_cast<const uint32_t *>(a.x_scales), a.T, a.H / 128, xs);
        s = xs;
    }
    up_kernel<<<(int)(((long long)n * a.I + per - 1) / per), kThreads, 0, stream>>>(a, q, s, h);
    quantise_kernel<false><<<(gh + per - 1) / per, kThreads, 0, stream>>>(h, gh, hq, hs);
    down_kernel<<<(int)(((long long)a.T * a.H + per - 1) / per), kThreads, 0, stream>>>(a, hq, hs);
    return cudaGetLastError();
}

}  // namespace ep
