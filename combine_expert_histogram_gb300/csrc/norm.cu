// ep_rmsnorm kernel: residual addition, root-mean-square norm and the output
// as bf16 rows and / or E4M3 rows with dynamic scales (the formats of
// ep_dispatch; [PR-35634] "Supported scope": dynamic blockwise FP8).
//
//   s = x + residual,  y = s * (1 / sqrt(mean(s^2) + eps)) * weight
//
// One CTA per row: the row is read once into registers (8 elements per lane
// and vector), squared and summed in fp32 (lane, xor-shuffles, one exchange
// through shared memory), scaled, and written from the same registers; the
// 8-bit output takes the group maxima by xor-shuffles over the 16 lanes that
// hold a 1x128 group (4 lanes for 1x32), so nothing is read twice.  HBM-bound:
// 16384 rows of 7168 with the residual, bf16 and 8-bit rows (1.06 GB) take 154 to
// 155 us, 6.8 TB/s; one such row 2.4 us.
#include "ep_common.cuh"
#include "fp8.cuh"

namespace ep {
namespace {

constexpr int kMaxThreads = 1024;

template <int Q, int V>
__global__ void __launch_bounds__(kMaxThreads)
    rmsnorm_kernel(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps,
                   int H, uint16_t *residual_out, uint16_t *out, uint8_t *rows, uint8_t *scales,
                   int mn_stride) {
    __shared__ float part[kMaxThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int NT = blockDim.x, vecs = H >> 3;
    const size_t row = blockIdx.x;
    // the weight waits too: the kernel before may have written it (read ahead of the
    // wait, it gained one row 0.07 us of 2.1 and cost 1021 rows of 2056 0.1 us of 2.9)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    uint4 xv[V], rv[V], wv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * NT + threadIdx.x;
        xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (j < vecs) {
            xv[i] = ld_stream_coh(x + row * H + 8 * j);
            if (residual) rv[i] = ld_stream_coh(residual + row * H + 8 * j);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * NT + threadIdx.x;
        wv[i] = j < vecs ? ld_dep_v4(weight + 8 * j) : make_uint4(0, 0, 0, 0);
    }
    float v[V][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t a[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
        const uint32_t b[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            v[i][2 * m] = bf16_lo(a[m]);
            v[i][2 * m + 1] = bf16_hi(a[m]);
            if (residual) {
                v[i][2 * m] += bf16_lo(b[m]);
                v[i][2 * m + 1] += bf16_hi(b[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) ss = fmaf(v[i][m], v[i][m], ss);
    }
    if (residual_out) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * NT + threadIdx.x;
            if (j < vecs)
                st_v4(residual_out + row * H + 8 * j,
                      make_uint4(pack_bf16(v[i][0], v[i][1]), pack_bf16(v[i][2], v[i][3]),
                                 pack_bf16(v[i][4], v[i][5]), pack_bf16(v[i][6], v[i][7])));
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lane < NT / 32 ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps)));

#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * NT + threadIdx.x;
        const uint32_t w[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
        float y[8];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            y[2 * m] = v[i][2 * m] * rstd * bf16_lo(w[m]);
            y[2 * m + 1] = v[i][2 * m + 1] * rstd * bf16_hi(w[m]);
        }
        if (out && j < vecs)
            st_v4(out + row * H + 8 * j,
                  make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                             pack_bf16(y[6], y[7])));
        if constexpr (Q != EP_QUANT_NONE) {
            // quantised from the fp32 values, not from the bf16 output: one
            // rounding instead of two, and the bf16 rows need not be written
            float amax = 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m) amax = fmaxf(amax, fabsf(y[m]));
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
            if (Q != EP_QUANT_MXFP8) {
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 4));
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 8));
            }
            if (Q == EP_QUANT_FP8_F32) {
                // 16384 x 7168: 154.3 us; 4 % more with eight divisions a lane, 154.1 with
                // the product by inv alone, which falls to the other side of some ties
                const float s = group_scale(amax), inv = __frcp_rn(s);
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = group_quotient(y[m], s, inv);
                if (j < vecs && (lane & 15) == 0)
                    reinterpret_cast<float *>(scales)[row * (H >> 7) + (j >> 4)] = s;
            } else {
                const int e = Q == EP_QUANT_MXFP8 ? mx_exponent(amax)
                                                  : ue8m0_exponent(group_scale(amax));
                const float inv = exp_reciprocal(e);
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = __fmul_rn(y[m], inv);
                if (Q == EP_QUANT_MXFP8) {
                    if (j < vecs && (lane & 3) == 0) scales[row * (H >> 5) + (j >> 2)] = (uint8_t)e;
                } else if (j < vecs && (lane & 15) == 0) {
                    // byte g%4 of word g/4; the last group also fills the word (127 = 2^0)
                    const int g = j >> 4, G = H >> 7;
                    const int last = g == G - 1 ? (g | 3) : g;
                    for (int b = g; b <= last; ++b) {
                        const size_t word = Q == EP_QUANT_FP8_UE8M0_MN
                                                ? (size_t)(b >> 2) * mn_stride + row
                                                : row * ((G + 3) >> 2) + (b >> 2);
                        scales[word * 4 + (b & 3)] = (uint8_t)(b == g ? e : 127);
                    }
                }
            }
            if (j < vecs)
                *reinterpret_cast<uint2 *>(rows + row * H + 8 * j) =
                    make_uint2(fp8x4(y[0], y[1], y[2], y[3]), fp8x4(y[4], y[5], y[6], y[7]));
        }
    }
}

template <int Q>
cudaError_t launch_q(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps,
                     int T, int H, uint16_t *residual_out, uint16_t *out, uint8_t *rows,
                     uint8_t *scales, cudaStream_t stream) {
    const int vecs = H / 8;
    // Up to two rows an SM: a vector a lane, the shortest way through one row.  Above:
    // blocks of up to 256 threads with up to four, so that more rows share an SM and
    // some load while others reduce.  On the GPU, 8-bit rows of 7168: 1 row 2.3 us
    // (2.8 in blocks of 256), 304 rows 3.8 (4.0); 305 rows 4.8 (5.1 with a vector a
    // lane), 456 rows 5.2 (5.6), 16384 rows 154 (185).  bf16 rows of 2056: 1.7 either
    // way at 304, 2.3 (2.6) at 1021.
    const int want = T > 2 * sm_count() ? 256 : kMaxThreads;
    int V = 1;
    while (V < 4 && vecs > V * want) V *= 2;
    const int threads = ((vecs + V - 1) / V + 31) / 32 * 32;
    auto k = V == 1 ? rmsnorm_kernel<Q, 1> : V == 2 ? rmsnorm_kernel<Q, 2> : rmsnorm_kernel<Q, 4>;
    return launch_kernel(k, T, threads, 0, stream, true, x, residual, weight, eps, H, residual_out,
                         out, rows, scales, (int)((T + 3ll) / 4 * 4));
}

}  // namespace

cudaError_t launch_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                           int T, int H, ep_quant_t quant, void *residual_out, void *out,
                           void *rows, void *scales, cudaStream_t stream) {
    auto go = [&](auto launch) {
        return launch(static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(residual),
                      static_cast<const uint16_t *>(weight), eps, T, H,
                      static_cast<uint16_t *>(residual_out), static_cast<uint16_t *>(out),
                      static_cast<uint8_t *>(rows), static_cast<uint8_t *>(scales), stream);
    };
    switch (quant) {
        case EP_QUANT_FP8_F32: return go(launch_q<EP_QUANT_FP8_F32>);
        case EP_QUANT_FP8_UE8M0: return go(launch_q<EP_QUANT_FP8_UE8M0>);
        case EP_QUANT_MXFP8: return go(launch_q<EP_QUANT_MXFP8>);
        case EP_QUANT_FP8_UE8M0_MN: return go(launch_q<EP_QUANT_FP8_UE8M0_MN>);
        default: return go(launch_q<EP_QUANT_NONE>);
    }
}

}  // namespace ep
