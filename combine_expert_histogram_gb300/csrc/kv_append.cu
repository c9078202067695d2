// ep_kv_append: new tokens' keys and values into a paged cache, with the rotation by
// position of the queries and keys on the way:
//
//   a' = a cos - b sin,  b' = b cos + a sin   for the pairs of the first R channels
//
// A warp takes one token and some of its head rows, D/16 lanes a row, each with the
// eight channels and their pairs' other halves of eight angles, whose cosines and sines serve
// all rows the warp goes through.  HBM-bound: every row is read once and written once: 14000
// tokens of 64 + 2 * 8 heads of 128 into an 8-bit cache, 670 MB, take 109 us (6.1 TB/s); one
// token takes 2.3 us, which is a launch.
#include "attn.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;

struct AppendArgs {
    KvArgs kv;
    SeqArgs seq;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int Hq;  // 0: no queries
    const float *cos_sin;
    int R, positions;
    uint16_t *q_out;
    int rows;  // head rows a warp takes
};

// A pair of channels turned, each product and sum rounded by itself, so that the bits do not
// hang on a choice of fused operations (the assembler fuses packed ones, mul.rn.f32x2 and
// add.rn.f32x2, although their rounding is given).
__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
    const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = u;
}
__device__ __forceinline__ uint4 bf16x8(const float (&y)[8]) {
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}
__device__ __forceinline__ void floats(const uint4 &x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo(w[i]), y[2 * i + 1] = bf16_hi(w[i]);
}

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendArgs a) {
    constexpr int L = D / 16, P = 32 / L, U = 2;  // lanes a row, rows at a time, of which in flight
    const int lane = threadIdx.x & 31, c = lane % L, sub = lane / L;
    const int heads = a.Hq + 2 * a.kv.Hkv, parts = (heads + a.rows - 1) / a.rows;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(unit / parts), h0 = (int)(unit % parts) * a.rows, h1 = min(h0 + a.rows, heads);
    // the lane's two vectors of eight channels
    const bool turned = 16 * c < a.R;
    const int v0 = INTER ? 2 * c : turned ? c : 2 * c, v1 = !INTER && turned ? c + a.R / 16 : v0 + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.seq.T) return;
    // The rows first: where they go is a chain of small loads.
    auto load = [&](int h, uint4 (&x)[U][2]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = h + i * P + sub;
            x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
            if (r >= h1) continue;
            const bool is_q = r < a.Hq, is_k = r < a.Hq + a.kv.Hkv;
            const int kh = r - a.Hq - (is_k ? 0 : a.kv.Hkv);
            const uint16_t *src = is_q   ? a.q + t * a.q_stride + (int64_t)r * D
                                  : is_k ? a.k + t * a.k_stride + (int64_t)kh * D
                                         : a.v + t * a.v_stride + (int64_t)kh * D;
            x[i][0] = ld_dep_stream(src + 8 * v0);
            x[i][1] = ld_dep_stream(src + 8 * v1);
        }
    };
    uint4 now[U][2], next[U][2];
    load(h0, now);

    const int b = seq_of(a.seq, t);
    if (b < 0) return;
    const Span sp = seq_rows(a.seq, b);
    const int pos = sp.len - sp.n + (t - sp.first);
    if (pos < 0) return;
    // past a table there is no place for the token, and none that it may take
    if (pos >= a.seq.max_pages * a.kv.page_size || (a.R && pos >= a.positions)) {
        raise_status(a.seq.status, EP_ERR_BAD_PAGE);
        return;
    }
    const int page = page_of(a.kv, a.seq, b, pos / a.kv.page_size);
    if (page < 0) return;
    const int row = pos % a.kv.page_size;
    const int64_t place = page * a.kv.page_stride + row * a.kv.row_stride;

    float cs[8], sn[8];  // of the angles 8 c .. 8 c + 7
    if (turned) {
        const float *p = a.cos_sin + (int64_t)pos * a.R + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const uint4 u = ld_dep_v4(p + i), w = ld_dep_v4(p + a.R / 2 + i);
            cs[i] = __uint_as_float(u.x), cs[i + 1] = __uint_as_float(u.y);
            cs[i + 2] = __uint_as_float(u.z), cs[i + 3] = __uint_as_float(u.w);
            sn[i] = __uint_as_float(w.x), sn[i + 1] = __uint_as_float(w.y);
            sn[i + 2] = __uint_as_float(w.z), sn[i + 3] = __uint_as_float(w.w);
        }
    }
    for (int h = h0; h < h1; h += U * P) {
        if (h + U * P < h1) load(h + U * P, next);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (h + i * P >= h1) break;
            const int r = h + i * P + sub;
            const bool live = r < h1, is_q = r < a.Hq, is_k = r < a.Hq + a.kv.Hkv;
            const int kh = r - a.Hq - (is_k ? 0 : a.kv.Hkv);
            uint4 w0 = now[i][0], w1 = now[i][1];
            float y0[8], y1[8];
            floats(w0, y0);
            floats(w1, y1);
            if (turned && is_k) {
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    if constexpr (INTER) {
                        float *y = m < 4 ? y0 + 2 * m : y1 + 2 * (m - 4);
                        turn(y[0], y[1], cs[m], sn[m]);
                    } else {
                        turn(y0[m], y1[m], cs[m], sn[m]);
                    }
                }
                w0 = bf16x8(y0);
                w1 = bf16x8(y1);
            }
            if (is_q) {
                uint16_t *dst = a.q_out + t * a.q_out_stride + (int64_t)r * D;
                if (live) {
                    st_v4(dst + 8 * v0, w0);
                    st_v4(dst + 8 * v1, w1);
                }
            }
            uint8_t *dst = (is_k ? a.kv.k : a.kv.v) + place + kh * a.kv.head_stride;
            if constexpr (!FP8) {
                if (live && !is_q) {
                    st_v4(dst + 16 * v0, w0);
                    st_v4(dst + 16 * v1, w1);
                }
            } else if (__any_sync(kFullMask, !is_q)) {
                float amax = 0.0f;
                bool odd = false;  // an infinity or NaN: the row has no scale
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    amax = fmaxf(amax, fmaxf(fabsf(y0[m]), fabsf(y1[m])));
                    odd |= !(fabsf(y0[m]) <= 3.402823466e38f) || !(fabsf(y1[m]) <= 3.402823466e38f);
                }
                if (odd) amax = __uint_as_float(0x7f800000u);
#pragma unroll
                for (int m = 1; m < L; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, m));
                if (live && !is_q) {
                    int e = ue8m0_exponent(group_scale(amax));
                    odd = amax > 3.402823466e38f;
                    if (odd) e = 255;
                    const float inv = odd ? 0.0f : exp_reciprocal(e);
                    auto store = [&](int v, const float (&y)[8]) {
                        uint32_t w[2];
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            w[m] = odd ? 0x7f7f7f7fu
                                       : fp8x4(__fmul_rn(y[4 * m], inv), __fmul_rn(y[4 * m + 1], inv),
                                               __fmul_rn(y[4 * m + 2], inv), __fmul_rn(y[4 * m + 3], inv));
                        *reinterpret_cast<uint2 *>(dst + 8 * v) = make_uint2(w[0], w[1]);
                    };
                    store(v0, y0);
                    store(v1, y1);
                    if (c == 0)
                        (is_k ? a.kv.k_scales : a.kv.v_scales)[((int64_t)page * a.kv.Hkv + kh) *
                                                                   a.kv.page_size + row] = (uint8_t)e;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) now[i][0] = next[i][0], now[i][1] = next[i][1];
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs &kv, const SeqArgs &seq, const uint16_t *q,
                             int64_t q_stride, int Hq, const uint16_t *k, int64_t k_stride,
                             const uint16_t *v, int64_t v_stride, const float *cos_sin, int R,
                             int positions, bool interleaved, uint16_t *q_out,
                             int64_t q_out_stride, cudaStream_t stream) {
    AppendArgs a = {kv, seq, q, k, v, q_stride, k_stride, v_stride, q_out_stride, Hq, cos_sin,
                    R, positions, q_out, 0};
    const int heads = Hq + 2 * kv.Hkv;
    // Whole tokens where that leaves every SM 32 warps and more, else fewer rows a warp, in whole
    // passes.
    const int pass = 512 / kv.D;
    auto passes = [&](int rows) { return (rows + pass - 1) / pass * pass; };
    const int64_t warps = 32ll * sm_count();
    a.rows = passes(heads);
    while (a.rows > pass && (int64_t)seq.T * ((heads + a.rows - 1) / a.rows) < warps) a.rows = passes(a.rows / 2);
    const int64_t units = (int64_t)seq.T * ((heads + a.rows - 1) / a.rows);
    const int grid = (int)((units + kWarps - 1) / kWarps);
    const bool fp8 = kv.k_scales != nullptr;
    auto k0 = kv.D == 64 ? (fp8 ? (interleaved ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                                : (interleaved ? append_kernel<64, false, true> : append_kernel<64, false, false>))
                         : (fp8 ? (interleaved ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                                : (interleaved ? append_kernel<128, false, true> : append_kernel<128, false, false>));
    return launch_kernel(k0, grid, kWarps * 32, 0, stream, true, a);
}

}  // namespace ep
