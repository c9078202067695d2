// ep_kv_append: new tokens' keys and values into a paged cache, with the rotation by
// position of the queries and keys on the way:
//
//   a' = a cos - b sin,  b' = b cos + a sin   for the pairs of the first R channels
//
// A warp takes one token and some of its head rows, D/8 lanes a row with eight
// channels each, so that a lane's eight cosines and sines serve all rows the warp
// goes through.  A pair's other half is another lane's vector (one shuffle) or the
// neighbouring channel.  HBM-bound: every row is read once and written once.
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

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendArgs a) {
    constexpr int L = D / 8, P = 32 / L;  // lanes a row, rows at a time
    const int lane = threadIdx.x & 31, c = lane % L, sub = lane / L;
    const int heads = a.Hq + 2 * a.kv.Hkv, parts = (heads + a.rows - 1) / a.rows;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = (int)(unit / parts), h0 = (int)(unit % parts) * a.rows;
    if (t >= a.seq.T) return;
    const int b = seq_of(a.seq, t);
    if (b < 0) return;
    const Span sp = seq_span(a.seq, a.kv.page_size, b);
    const int pos = sp.len - sp.n + (t - sp.first);
    if (pos < 0) return;
    if (a.R && pos >= a.positions) {
        raise_status(a.seq.status, EP_ERR_BAD_PAGE);
        return;
    }
    const int page = page_of(a.kv, a.seq, b, pos / a.kv.page_size);
    if (page < 0) return;
    const int row = pos % a.kv.page_size;

    float cs[8], sn[8];
    const bool turned = 8 * c < a.R, low = 16 * c < a.R;
    if (turned) {
        // half of a row's angles fall on each lane's eight channels (INTER: four)
        const float *p = a.cos_sin + (int64_t)pos * a.R;
        const int at = INTER ? 4 * c : 8 * c - (low ? 0 : a.R / 2);
#pragma unroll
        for (int i = 0; i < (INTER ? 4 : 8); ++i) {
            cs[i] = ld_dep(p + at + i);
            sn[i] = ld_dep(p + a.R / 2 + at + i);
        }
    }
    for (int h = h0 + sub; h - sub < min(h0 + a.rows, heads); h += P) {
        const bool live = h < min(h0 + a.rows, heads);
        const bool is_q = h < a.Hq, is_k = h < a.Hq + a.kv.Hkv;
        const int kh = h - a.Hq - (is_k ? 0 : a.kv.Hkv);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live) {
            const uint16_t *src = is_q   ? a.q + t * a.q_stride + (int64_t)h * D
                                  : is_k ? a.k + t * a.k_stride + (int64_t)kh * D
                                         : a.v + t * a.v_stride + (int64_t)kh * D;
            x = ld_dep_stream(src + 8 * c);
        }
        float y[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                      bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
        if (a.R) {
            // each product and sum rounded by itself, so that the bits do not hang on
            // the compiler's choice of fused operations
            const bool turn = turned && is_k;
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = y[2 * i], w = y[2 * i + 1];
                    if (turn) {
                        y[2 * i] = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(w, sn[i]));
                        y[2 * i + 1] = __fadd_rn(__fmul_rn(w, cs[i]), __fmul_rn(u, sn[i]));
                    }
                }
            } else {
                const int other = turned ? lane + (low ? a.R / 16 : -(a.R / 16)) : lane;
                uint4 o;
                o.x = __shfl_sync(kFullMask, x.x, other);
                o.y = __shfl_sync(kFullMask, x.y, other);
                o.z = __shfl_sync(kFullMask, x.z, other);
                o.w = __shfl_sync(kFullMask, x.w, other);
                const float z[8] = {bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y),
                                    bf16_lo(o.z), bf16_hi(o.z), bf16_lo(o.w), bf16_hi(o.w)};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = __fmul_rn(y[i], cs[i]), r = __fmul_rn(z[i], sn[i]);
                    if (turn) y[i] = low ? __fsub_rn(p, r) : __fadd_rn(p, r);
                }
            }
        }
        if (is_q) {
            if (live)
                st_v4(a.q_out + t * a.q_out_stride + (int64_t)h * D + 8 * c,
                      make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                 pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])));
        }
        uint8_t *dst = (is_k ? a.kv.k : a.kv.v) + page * a.kv.page_stride +
                       row * a.kv.row_stride + kh * a.kv.head_stride;
        if constexpr (!FP8) {
            if (live && !is_q)
                st_v4(dst + 16 * c, make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                               pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])));
        } else {
            float amax = 0.0f;
            bool odd = false;  // an infinity or NaN: the row has no scale
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(y[i]));
                odd |= !(fabsf(y[i]) <= 3.402823466e38f);
            }
            if (odd) amax = __uint_as_float(0x7f800000u);
#pragma unroll
            for (int d = 1; d < L; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
            if (live && !is_q) {
                int e = ue8m0_exponent(group_scale(amax));
                odd = amax > 3.402823466e38f;
                if (odd) e = 255;
                const float inv = odd ? 0.0f : exp_reciprocal(e);
                uint32_t w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[i] = odd ? 0x7f7f7f7fu
                               : fp8x4(__fmul_rn(y[4 * i], inv), __fmul_rn(y[4 * i + 1], inv),
                                       __fmul_rn(y[4 * i + 2], inv), __fmul_rn(y[4 * i + 3], inv));
                *reinterpret_cast<uint2 *>(dst + 8 * c) = make_uint2(w[0], w[1]);
                if (c == 0)
                    (is_k ? a.kv.k_scales : a.kv.v_scales)[((int64_t)page * a.kv.Hkv + kh) *
                                                               a.kv.page_size + row] = (uint8_t)e;
            }
        }
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
    a.rows = 8;
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
