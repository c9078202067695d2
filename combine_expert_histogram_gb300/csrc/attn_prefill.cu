// ep_attn_prefill, plain: one warp for each query head of a token.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  m the largest so far
//
// in one pass over the visible keys: when m grows, the sums are scaled down.
#include "attn.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;

// The N values of this lane of a cache row.
template <int N>
__device__ __forceinline__ void load_row(const KvArgs &kv, const uint8_t *base,
                                         const uint8_t *scales, int page, int row, int h, int lane,
                                         float (&x)[N]) {
    if (page < 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.0f;
        return;
    }
    const uint8_t *p = base + page * kv.page_stride + row * kv.row_stride + h * kv.head_stride;
    if (scales) {
        const float s = scale_value(scales[((int64_t)page * kv.Hkv + h) * kv.page_size + row]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const __half_raw r = __nv_cvt_fp8_to_halfraw(p[N * lane + i], __NV_E4M3);
            x[i] = __half2float(__half(r)) * s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint32_t u = reinterpret_cast<const uint32_t *>(p)[(N * lane + i) / 2];
            x[i] = bf16_lo(u);
            x[i + 1] = bf16_hi(u);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(unit / a.Hq), hq = (int)(unit % a.Hq), h = hq / (a.Hq / a.kv.Hkv);
    constexpr int D = 32 * N;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.seq.T) return;
    const int b = seq_of(a.seq, t);
    if (b < 0) return;
    const Span sp = seq_span(a.seq, a.kv.page_size, b);
    const int i = a.seq.q_start ? sp.len - sp.n + (t - sp.first) : sp.len - 1;
    float q[N], k[N], o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int n = 0; n < N; n += 2) {
        const uint32_t u = reinterpret_cast<const uint32_t *>(a.q + t * a.q_stride + (int64_t)hq * D)[(N * lane + n) / 2];
        q[n] = bf16_lo(u);
        q[n + 1] = bf16_hi(u);
        o[n] = o[n + 1] = 0.0f;
    }
    const int near = a.window ? max(0, i - a.window + 1) : 0;
    int entry = -1, page = -1;
    for (int j = 0; j <= i; ++j) {
        if (j < near && j >= a.sinks) j = near;
        if (j / a.kv.page_size != entry) {
            entry = j / a.kv.page_size;
            page = page_of(a.kv, a.seq, b, entry);
        }
        const int row = j % a.kv.page_size;
        load_row<N>(a.kv, a.kv.k, a.kv.k_scales, page, row, h, lane, k);
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) s = fmaf(q[n], k[n], s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFullMask, s, d);
        s *= a.scale;
        const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.0f : top;
        const float f = m == top ? 1.0f : expf(m - ref), p = expf(s - ref);
        load_row<N>(a.kv, a.kv.v, a.kv.v_scales, page, row, h, lane, k);
        l = l * f + p;
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = o[n] * f + p * k[n];
        m = top;
    }
    const bool none = i < 0;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + ((int64_t)t * a.Hq + hq) * D);
#pragma unroll
    for (int n = 0; n < N; n += 2)
        dst[(N * lane + n) / 2] = none ? 0u : pack_bf16(o[n] / l, o[n + 1] / l);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + hq] = none ? -INFINITY : m + logf(l);
}

cudaError_t launch_rows(const AttnArgs &a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.seq.T * a.Hq;
    const int grid = (int)((units + kWarps - 1) / kWarps);
    return a.kv.D == 64 ? launch_kernel(attn_kernel<2>, grid, kWarps * 32, 0, stream, true, a)
                        : launch_kernel(attn_kernel<4>, grid, kWarps * 32, 0, stream, true, a);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs &a, cudaStream_t stream) {
    return launch_rows(a, stream);
}

}  // namespace ep
