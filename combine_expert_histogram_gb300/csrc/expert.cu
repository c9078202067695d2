// ep_expert_gemm / ep_expert_swiglu: the experts' products on a layout's E4M3
// rows, with one scale per 1x128 group of a row and one per 128x128 block of a
// weight ([DISC-26563]: 128x128 blockwise FP8 with dynamic activation scaling):
//
//   y[r, n] = sum over blocks b of sx[r, b] * sw[e, n/128, b]
//                                  * sum over k in b of x[r, k] * w[e, n, k]
//
// 32 x 128 tiles on the fp32 pipes: the block sums stay in registers and are
// scaled into the running sums after each 128 of K.
#include <cuda_bf16.h>

#include "expert.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTM = 32, kTN = 128;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, d));
    return v;
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads) expert_kernel(const ExpertArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    float *xs = reinterpret_cast<float *>(smem);             // [128][kTM]: k-major
    uint32_t *ws = reinterpret_cast<uint32_t *>(smem + 128 * kTM * 4);  // [2][kTN][32 + 1]
    int32_t *pre = reinterpret_cast<int32_t *>(ws + 2 * kTN * 33);      // [E+1]
    __shared__ int32_t tmp[kThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    block_exclusive_scan<kThreads>(
        a.E, [&](int e) { return (expert_rows(a, e) + kTM - 1) / kTM; }, pre, tmp);
    const int ntn = (a.N + kTN - 1) / kTN;
    const long long total = (long long)pre[a.E] * ntn;
    const int G = a.K >> 7, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int W = GATED ? 2 * a.N : a.N, NB = (W + 127) / 128;
    for (long long t = blockIdx.x; t < total; t += gridDim.x) {
        const int mt = (int)(t / ntn), n0 = (int)(t % ntn) * kTN;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= mt) lo = mid; else hi = mid;
        }
        const int e = lo, first = expert_first(a, e), rows = expert_rows(a, e);
        const int r0 = (mt - pre[e]) * kTM;
        float acc[GATED ? 2 : 1][4][4] = {};
        for (int g = 0; g < G; ++g) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTM * 32; i += kThreads) {
                const int m = i >> 5, k4 = i & 31;
                float4 f = make_float4(0, 0, 0, 0);
                if (r0 + m < rows)
                    f = e4m3x4_to_float4((uint32_t)ld_dep(reinterpret_cast<const int32_t *>(
                        a.x + (size_t)(first + r0 + m) * a.K + g * 128 + k4 * 4)));
                xs[(4 * k4) * kTM + m] = f.x;
                xs[(4 * k4 + 1) * kTM + m] = f.y;
                xs[(4 * k4 + 2) * kTM + m] = f.z;
                xs[(4 * k4 + 3) * kTM + m] = f.w;
            }
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
                for (int i = threadIdx.x; i < kTN * 32; i += kThreads) {
                    const int n = i >> 5, k4 = i & 31;
                    uint32_t v = 0;
                    if (n0 + n < a.N)
                        v = __ldg(reinterpret_cast<const uint32_t *>(
                            a.w + ((size_t)e * W + h * a.N + n0 + n) * a.K + g * 128 + k4 * 4));
                    ws[(h * kTN + n) * 33 + k4] = v;
                }
            __syncthreads();
            float blk[GATED ? 2 : 1][4][4] = {};
            for (int k4 = 0; k4 < 32; ++k4) {
                float4 xr[4];  // [k][4 rows]
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    xr[q] = *reinterpret_cast<const float4 *>(xs + (4 * k4 + q) * kTM + ty * 4);
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 w = e4m3x4_to_float4(ws[(h * kTN + j * 32 + tx) * 33 + k4]);
                        const float wk[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            blk[h][0][j] = fmaf(xr[q].x, wk[q], blk[h][0][j]);
                            blk[h][1][j] = fmaf(xr[q].y, wk[q], blk[h][1][j]);
                            blk[h][2][j] = fmaf(xr[q].z, wk[q], blk[h][2][j]);
                            blk[h][3][j] = fmaf(xr[q].w, wk[q], blk[h][3][j]);
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h) {
                const float sw = __ldg(a.w_scales + ((size_t)e * NB + (h * a.N + n0) / 128) * G + g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + ty * 4 + i;
                    if (r >= rows) continue;
                    const float s = sw * row_scale(a, first + r, e, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(blk[h][i][j], s, acc[h][i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + ty * 4 + i;
            if (r >= rows) continue;  // the same for the whole warp
            float v[4], amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = acc[0][i][j];
                if (GATED) v[j] = v[j] / (1.0f + expf(-v[j])) * acc[GATED ? 1 : 0][i][j];
                amax = fmaxf(amax, fabsf(v[j]));
            }
            const size_t at = (size_t)(first + r) * a.N + n0;
            if (!GATED || a.out_quant == EP_QUANT_NONE) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + j * 32 + tx < a.N)
                        static_cast<__nv_bfloat16 *>(a.out)[at + j * 32 + tx] = __float2bfloat16_rn(v[j]);
            } else {
                amax = warp_max(amax);
                const float s = group_scale(amax);
                const int e8 = ue8m0_exponent(s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float q = a.out_quant == EP_QUANT_FP8_F32
                                        ? __fdiv_rn(v[j], s)
                                        : __fmul_rn(v[j], exp_reciprocal(e8));
                    static_cast<uint8_t *>(a.out)[at + j * 32 + tx] =
                        __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
                }
                if (tx == 0) store_out_scale(a, first + r, e, n0 / 128, s, e8);
            }
        }
    }
}

}  // namespace

cudaError_t launch_expert(const ExpertArgs &a, bool gated, cudaStream_t stream) {
    const size_t smem = 128 * kTM * 4 + 2 * kTN * 33 * 4 + (a.E + 1) * 4;
    auto k = gated ? expert_kernel<true> : expert_kernel<false>;
    const cudaError_t err = allow_dynamic_smem(k, smem);
    if (err != cudaSuccess) return err;
    return launch_kernel(k, 2 * sm_count(), kThreads, smem, stream, true, a);
}

}  // namespace ep
