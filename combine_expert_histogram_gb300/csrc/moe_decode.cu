// ep_moe_decode: a whole mixture-of-experts layer for a few tokens.
//
//   xq = 1x128 E4M3 of x,  g = W13[e][:I] xq,  u = W13[e][I:] xq,
//   hq = 1x128 E4M3 of silu(g) * u,  out[t] = sum over k of w[t,k] * W2[e] hq
//
// Bound by reading the picked experts' weights once.  Two kernels of the same
// body (rows of W13 against the tokens, rows of W2 against the gated results)
// and a small one for the weighted sum; all launched as programmatic
// dependents.  Each CTA groups the T*K entries by expert itself (at most 1024,
// in shared memory) into chunks of one expert and up to 8 or 16 entries; the
// (chunk, 16 weight rows) units are split evenly over one persistent CTA per
// SM, which walks a contiguous run of them:
//   - a loader warp keeps a ring of (16 rows x 1024 bytes) pieces in flight with
//     one bulk copy per row.  It never waits for the previous kernel (weights
//     are not its output), so the second kernel's ring fills while the first
//     one drains;
//   - eight warps multiply, each one 128-wide block of the piece, on the
//     m16n8k32 E4M3 instruction: the weight rows are its 16 rows, the entries
//     its 8 columns.  Sixteen-row units keep the SMs' shares within a few
//     percent of each other for single tokens, which 128-row tcgen05 tiles
//     would not, and the rate of this path is a small part of its peak.  Block
//     sums are scaled into fp32 registers, and the warps' parts meet in shared
//     memory at the end of a unit, in a fixed order.
// The inner order of a product is permuted (each lane takes 16 consecutive
// bytes of its row), the same for weights and entries, so that shared memory
// is read 16 bytes a lane; rows are 64 bytes off a multiple of 128 apart, which
// makes those reads free of bank conflicts.
#include "expert.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;                        // multiplying warps
constexpr int kThreads = 32 * (kWarps + 1);      // + loader
constexpr int kRows = 16;                        // weight rows of a unit
constexpr int kPiece = 128 * kWarps;             // bytes of a row in one piece
constexpr int kRowStride = kPiece + 64;
constexpr int kStageBytes = kRows * kRowStride;
constexpr int kMaxStages = 12;
constexpr int kMaxEntries = EP_MOE_DECODE_MAX_ENTRIES;
constexpr int kSmemMax = 227 * 1024 - 2048;      // less the static part

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int fail;
    int issued;
    int32_t scan[kThreads / 32];
    int32_t chunks;
    uint16_t entry[kMaxEntries];   // entries, grouped by expert
    uint32_t chunk[kMaxEntries];   // expert | first entry << 10 | entries << 20
};

__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

// Group the routed entries by expert.  `tmp` holds 3 * E + 2 ints and n 16-bit
// ids; every thread of the CTA calls it.  Every CTA must put the same entries
// into the same chunk.  Within a chunk their order is free (no entry's result
// depends on which column it takes), so only the entries of an expert with
// several chunks are ranked by counting the same ids before them.
__device__ void group_entries(const MoeArgs &a, int cols, int32_t *tmp, Shared &sh) {
    int32_t *cnt = tmp, *start = cnt + a.E, *first = start + a.E + 1;  // [E], [E+1], [E+1]
    uint16_t *ids = reinterpret_cast<uint16_t *>(first + a.E + 1);     // [n]
    const int n = a.T * a.K;
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    __syncthreads();
    int mine[(kMaxEntries + kThreads - 1) / kThreads];
#pragma unroll
    for (int i = 0; i < (kMaxEntries + kThreads - 1) / kThreads; ++i) {
        const int j = i * kThreads + threadIdx.x;
        mine[i] = -1;
        if (j < n) {
            const int e = ld_dep(a.topk_idx + j);
            ids[j] = (uint16_t)(e >= 0 && e < a.E ? e : a.E);
            if (e >= 0 && e < a.E) {
                mine[i] = e;
                atomicAdd(cnt + e, 1);
            } else if (e != -1 && blockIdx.x == 0) {
                raise_status(a.status, EP_ERR_BAD_EXPERT_ID);
            }
        }
    }
    __syncthreads();
    block_exclusive_scan<kThreads>(a.E, [&](int e) { return cnt[e]; }, start, sh.scan);
    block_exclusive_scan<kThreads>(
        a.E, [&](int e) { return (cnt[e] + cols - 1) / cols; }, first, sh.scan);
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        for (int c = 0, at = 0; at < cnt[e]; ++c, at += cols)
            sh.chunk[first[e] + c] = (uint32_t)e | (uint32_t)(start[e] + at) << 10 |
                                     (uint32_t)min(cols, cnt[e] - at) << 20;
    }
    if (threadIdx.x == 0) sh.chunks = first[a.E];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (kMaxEntries + kThreads - 1) / kThreads; ++i) {
        const int e = mine[i], j = i * kThreads + threadIdx.x;
        if (e < 0) continue;
        int rank = 0;
        if (start[e + 1] - start[e] <= cols)
            rank = atomicAdd(cnt + e, 1);
        else
            for (int k = 0; k < j; ++k) rank += ids[k] == e;
        sh.entry[start[e] + rank] = (uint16_t)j;
    }
    __syncthreads();
}

__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Unit u of the list: its chunk and its first weight row / 16.
struct Unit {
    uint32_t chunk;
    int rows16;
};
struct Units {
    int per_chunk;  // units of one chunk: (2I or H) / 16
    __device__ __forceinline__ Unit at(const Shared &sh, int u) const {
        const int c = u / per_chunk;
        return {sh.chunk[c], u - c * per_chunk};
    }
};

// The chunk's entries as E4M3 columns in shared memory: xq[col][D + 64] and
// xs[group][cols].  UP: the tokens' x in any of its formats; else the gated
// results in fp32.  Half a warp takes a 1x128 group, 8 values a lane.
template <bool UP>
__device__ __forceinline__ void load_columns(const MoeArgs &a, const float *h, uint32_t chunk,
                                             const Shared &sh, int D, int cols, uint8_t *xq,
                                             float *xs) {
    constexpr int kBatch = 4;
    const int first = chunk >> 10 & 1023, n = (int)(chunk >> 20);
    const int G = D >> 7, items = n * G;
    const int half = (threadIdx.x >> 4) & 1, l = threadIdx.x & 15;
    // the bound is the same for both halves of a warp, which shuffle together
    for (int w0 = 2 * (threadIdx.x >> 5); w0 < items; w0 += 2 * kWarps * kBatch) {
        const int i0 = w0 + half;
        float v[kBatch][8];
        uint2 q[kBatch];
        float s[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * 2 * kWarps;
            const int col = i / G, g = i - col * G;
#pragma unroll
            for (int m = 0; m < 8; ++m) v[b][m] = 0.0f;
            q[b] = make_uint2(0, 0);
            s[b] = 0.0f;
            if (i < items) {
                const int entry = sh.entry[first + col], t = UP ? entry / a.K : entry;
                const size_t at = (size_t)t * D + g * 128 + 8 * l;
                if (!UP) {
                    const uint4 lo = ld_dep_v4(h + at), hi = ld_dep_v4(h + at + 4);
                    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int m = 0; m < 8; ++m) v[b][m] = __uint_as_float(w[m]);
                } else if (a.quant == EP_QUANT_NONE) {
                    const uint4 x = ld_dep_v4(static_cast<const uint16_t *>(a.x) + at);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        v[b][2 * m] = bf16_lo(w[m]);
                        v[b][2 * m + 1] = bf16_hi(w[m]);
                    }
                } else {
                    const int32_t *p = reinterpret_cast<const int32_t *>(
                        static_cast<const uint8_t *>(a.x) + at);
                    q[b] = make_uint2((uint32_t)ld_dep(p), (uint32_t)ld_dep(p + 1));
                    if (a.quant == EP_QUANT_FP8_F32) {
                        s[b] = ld_dep(static_cast<const float *>(a.x_scales) + (size_t)t * G + g);
                    } else {
                        const uint32_t word = (uint32_t)ld_dep(
                            static_cast<const int32_t *>(a.x_scales) + (size_t)t * ((G + 3) / 4) +
                            (g >> 2));
                        s[b] = ue8m0_value(word >> (8 * (g & 3)) & 255u);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * 2 * kWarps;
            const int col = i / G, g = i - col * G;
            if (!UP || a.quant == EP_QUANT_NONE) {
                float amax = 0.0f;
#pragma unroll
                for (int m = 0; m < 8; ++m) amax = fmaxf(amax, fabsf(v[b][m]));
#pragma unroll
                for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
                s[b] = group_scale(amax);
#pragma unroll
                for (int m = 0; m < 8; ++m) v[b][m] = __fdiv_rn(v[b][m], s[b]);
                q[b] = make_uint2(fp8x4(v[b][0], v[b][1], v[b][2], v[b][3]),
                                  fp8x4(v[b][4], v[b][5], v[b][6], v[b][7]));
            }
            if (i < items) {
                *reinterpret_cast<uint2 *>(xq + (size_t)col * (D + 64) + g * 128 + 8 * l) = q[b];
                if (l == 0) xs[g * cols + col] = s[b];
            }
        }
    }
}

// UP: dst = h [T*K, I] fp32 from x, gate row i and up row i in one unit (8 of
// each); else dst = y [T*K, H] fp32 from h.  NB: blocks of 8 columns.
template <bool UP, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const MoeArgs a, const float *h, float *dst, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    constexpr int kCols = 8 * NB;
    const int D = UP ? a.H : a.I, G = D >> 7;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem;
    float *red = reinterpret_cast<float *>(ring + stages * kStageBytes);  // [2][kWarps][NB][128]
    float *xs = red + 2 * kWarps * NB * 128;                              // [G][kCols]
    uint8_t *xq = reinterpret_cast<uint8_t *>(xs + G * kCols);            // [kCols][D + 64]
    const volatile int *fail = &sh.fail;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        sh.fail = 0;
        sh.issued = 0;
        mbar_init_fence();
    }
    if (UP) {  // the ids may be the previous kernel's; for the second kernel they are complete
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = EP_OK;
        __syncthreads();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    group_entries(a, kCols, reinterpret_cast<int32_t *>(ring), sh);
    const Units units = {UP ? a.I / 8 : a.H / 16};
    const long long total = (long long)sh.chunks * units.per_chunk;
    const int u0 = (int)(total * blockIdx.x / gridDim.x), u1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
    const int pieces = (D + kPiece - 1) / kPiece;

    if (warp == kWarps) {
        // ---- loads: lane r copies row r of each piece ----
        fence_proxy_async_smem();  // the ring held the grouping's counters
        int it = 0;
        for (int u = u0; u < u1 && !__any_sync(kFullMask, *fail); ++u) {
            const Unit un = units.at(sh, u);
            const size_t e = un.chunk & 1023;
            const uint8_t *src;
            if (UP)  // 8 gate rows, then the same 8 up rows
                src = a.w13 + (e * 2 * a.I + (size_t)un.rows16 * 8 + (lane & 7) + (lane & 8 ? a.I : 0)) * D;
            else
                src = a.w2 + (e * a.H + (size_t)un.rows16 * 16 + (lane & 15)) * D;
            for (int p = 0; p < pieces; ++p, ++it) {
                const int s = it % stages;
                bool ok = it < stages || mbar_wait(&sh.empty[s], (it / stages - 1) & 1, fail);
                if (!__all_sync(kFullMask, ok)) {
                    sh.fail = 1;
                    break;
                }
                const uint32_t bytes = min(kPiece, D - p * kPiece);
                if (lane == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                                     smem_addr(&sh.full[s])),
                                 "r"(bytes * kRows)
                                 : "memory");
                __syncwarp();
                if (lane < kRows)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                        "[%1], %2, [%3];" ::"r"(smem_addr(ring + s * kStageBytes + lane * kRowStride)),
                        "l"(src + (size_t)p * kPiece), "r"(bytes), "r"(smem_addr(&sh.full[s]))
                        : "memory");
            }
        }
        if (lane == 0) sh.issued = it;
    } else {
        // ---- products.  After a wait that ran out the loops go on (every later
        // wait returns at once), so that all warps meet at the barriers ----
        if (!UP) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int g = lane >> 2, t = lane & 3;
        const int gb = UP ? a.I / 128 : 0;  // scale rows from a gate block to its up block
        uint32_t have = 0xffffffffu;  // the chunk whose entries are in xq
        int it = 0;
        for (int u = u0; u < u1; ++u) {
            const Unit un = units.at(sh, u);
            const int e = un.chunk & 1023, first = un.chunk >> 10 & 1023, n = (int)(un.chunk >> 20);
            const int block = un.rows16 / (UP ? 16 : 8);
            const float *sw = UP ? a.w13_scales + ((size_t)e * 2 * gb + block) * G
                                 : a.w2_scales + ((size_t)e * (a.H >> 7) + block) * G;
            float w0 = 0.0f, w1 = 0.0f;
            if (warp < G) {
                w0 = __ldg(sw + warp);
                w1 = UP ? __ldg(sw + (size_t)gb * G + warp) : w0;
            }
            if (un.chunk != have) {
                load_columns<UP>(a, h, un.chunk, sh, D, kCols, xq, xs);
                have = un.chunk;
                consumer_sync();
            }
            float acc[NB][4] = {};
            for (int p = 0; p < pieces; ++p, ++it) {
                const int s = it % stages, kb = p * kWarps + warp;
                const float s0 = w0, s1 = w1;
                if (kb + kWarps < G) {
                    w0 = __ldg(sw + kb + kWarps);
                    w1 = UP ? __ldg(sw + (size_t)gb * G + kb + kWarps) : w0;
                }
                if (!mbar_wait(&sh.full[s], (it / stages) & 1, fail)) sh.fail = 1;
                if (kb < G) {
                    const uint8_t *ap = ring + s * kStageBytes + g * kRowStride + warp * 128 + t * 16;
                    uint4 lo[2], hi[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        lo[i] = *reinterpret_cast<const uint4 *>(ap + 64 * i);
                        hi[i] = *reinterpret_cast<const uint4 *>(ap + 64 * i + 8 * kRowStride);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if (nb && n <= 8 * nb) break;
                        const uint8_t *bp = xq + (size_t)(8 * nb + g) * (D + 64) + kb * 128 + t * 16;
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 b = *reinterpret_cast<const uint4 *>(bp + 64 * i);
                            mma_16x8x32(d, lo[i].x, hi[i].x, lo[i].y, hi[i].y, b.x, b.y);
                            mma_16x8x32(d, lo[i].z, hi[i].z, lo[i].w, hi[i].w, b.z, b.w);
                        }
                        const float2 x = *reinterpret_cast<const float2 *>(xs + kb * kCols + 8 * nb + 2 * t);
                        acc[nb][0] = fmaf(d[0], s0 * x.x, acc[nb][0]);
                        acc[nb][1] = fmaf(d[1], s0 * x.y, acc[nb][1]);
                        acc[nb][2] = fmaf(d[2], s1 * x.x, acc[nb][2]);
                        acc[nb][3] = fmaf(d[3], s1 * x.y, acc[nb][3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.empty[s]);
            }
            // the warps' parts, [row][col] of each block of columns; the buffer of
            // the unit before last is free, all its readers have met at a barrier since
            float *mine = red + ((u & 1) * kWarps + warp) * NB * 128;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                *reinterpret_cast<float2 *>(mine + nb * 128 + g * 8 + 2 * t) = make_float2(acc[nb][0], acc[nb][1]);
                *reinterpret_cast<float2 *>(mine + nb * 128 + (g + 8) * 8 + 2 * t) = make_float2(acc[nb][2], acc[nb][3]);
            }
            consumer_sync();
            const float *part = red + (u & 1) * kWarps * NB * 128;
            // thread -> (row, column), rows fastest: an entry's outputs are consecutive
            if (UP) {
                const int r = threadIdx.x & 7, c = threadIdx.x >> 3;
                if (c < kCols && c < n) {
                    const float *q = part + (c >> 3) * 128 + r * 8 + (c & 7);
                    float gate = 0.0f, up = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        gate += q[w * NB * 128];
                        up += q[w * NB * 128 + 64];
                    }
                    dst[(size_t)sh.entry[first + c] * a.I + un.rows16 * 8 + r] =
                        __fdividef(gate, 1.0f + __expf(-gate)) * up;
                }
            } else {
                const int r = threadIdx.x & 15, c = threadIdx.x >> 4;
                if (c < kCols && c < n) {
                    const float *q = part + (c >> 3) * 128 + r * 8 + (c & 7);
                    float y = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) y += q[w * NB * 128];
                    dst[(size_t)sh.entry[first + c] * a.H + un.rows16 * 16 + r] = y;
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (sh.fail) {
        if (threadIdx.x == 0) raise_status(a.status, EP_ERR_TIMEOUT);
        // let the copies in flight land before the shared memory goes
        if ((int)threadIdx.x < stages) {
            const int last = sh.issued - 1 - (int)threadIdx.x;
            if (last >= 0) mbar_wait(&sh.full[last % stages], (last / stages) & 1, nullptr);
        }
        __syncthreads();
    }
}

// out[t] = sum over k of w[t,k] * y[t*K + k], 8 columns a thread.
__global__ void __launch_bounds__(128) sum_kernel(const MoeArgs a, const float *y) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int per = a.H / 8, i = blockIdx.x * 128 + threadIdx.x;
    const int t = i / per, c = i - t * per;
    if (t >= a.T) return;
    float acc[8] = {};
    for (int k = 0; k < a.K; ++k) {
        const int entry = t * a.K + k, e = ld_dep(a.topk_idx + entry);
        if (e < 0 || e >= a.E) continue;
        const float w = ld_dep(a.topk_w + entry);
        const float *p = y + (size_t)entry * a.H + 8 * c;
        const uint4 lo = ld_dep_v4(p), hi = ld_dep_v4(p + 4);
        const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int m = 0; m < 8; ++m) acc[m] = fmaf(w, __uint_as_float(v[m]), acc[m]);
    }
    st_v4(static_cast<uint16_t *>(a.out) + (size_t)t * a.H + 8 * c,
          make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                     pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7])));
}

template <bool UP, int NB>
cudaError_t launch_rows(const MoeArgs &a, const float *h, float *dst, cudaStream_t stream) {
    const int D = UP ? a.H : a.I;
    const size_t fixed = 2 * kWarps * NB * 128 * 4 + (size_t)(D / 128) * 8 * NB * 4 +
                         (size_t)8 * NB * (D + 64);
    const int fit = (int)((kSmemMax - sizeof(Shared) - fixed) / kStageBytes);
    const int stages = fit < kMaxStages ? fit : kMaxStages;
    const size_t smem = fixed + (size_t)stages * kStageBytes;
    auto k = rows_kernel<UP, NB>;
    const cudaError_t err = allow_dynamic_smem(k, smem);
    if (err != cudaSuccess) return err;
    return launch_kernel(k, sm_count(), kThreads, smem, stream, true, a, h, dst, stages);
}

}  // namespace

size_t moe_workspace_bytes(int T, int K, int H, int I) {
    return (size_t)T * K * ((size_t)I + H) * 4;
}

cudaError_t launch_moe_decode(const MoeArgs &a, void *workspace, cudaStream_t stream) {
    float *h = static_cast<float *>(workspace), *y = h + (size_t)a.T * a.K * a.I;
    // 16 columns hold an expert's entries in one chunk where experts have more
    // than a few on average; 8 leave more shared memory to the ring, and are all
    // that fits beside it for long rows
    const bool wide = a.T * a.K > 4 * a.E;
    cudaError_t err = wide && a.H <= 8192 ? launch_rows<true, 2>(a, nullptr, h, stream)
                                          : launch_rows<true, 1>(a, nullptr, h, stream);
    if (err != cudaSuccess) return err;
    err = wide && a.I <= 8192 ? launch_rows<false, 2>(a, h, y, stream)
                              : launch_rows<false, 1>(a, h, y, stream);
    if (err != cudaSuccess) return err;
    const long long threads = (long long)a.T * (a.H / 8);
    return launch_kernel(sum_kernel, (int)((threads + 127) / 128), 128, 0, stream, true, a,
                         (const float *)y);
}

}  // namespace ep
