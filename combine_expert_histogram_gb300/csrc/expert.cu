// ep_expert_gemm / ep_expert_swiglu: the experts' products on a layout's E4M3
// rows, with one scale per 1x128 group of a row and one per 128x128 block of a
// weight ([DISC-26563]: 128x128 blockwise FP8 with dynamic activation scaling):
//
//   y[r, n] = sum over blocks b of sx[r, b] * sw[e, n/128, b]
//                                  * sum over k in b of x[r, k] * w[e, n, k]
//
// Persistent CTAs, one per SM, take 128 x 256 tiles of (expert, 128 rows,
// 256 weight rows); the gated form's tile is 128 gate and the same 128 up
// columns, so that one CTA holds both factors of 128 outputs, which are one
// scale group of the result.  Four roles:
//   - one thread keeps a ring of 128-deep K blocks (rows and weights, 48 KB) in
//     flight by tiled TMA loads with 128-byte swizzle;
//   - one thread issues the tensor core's E4M3 products of a block, four
//     instructions of K = 32, into one of two tensor-memory tiles;
//   - two warps multiply the block's row and weight scales, four blocks ahead;
//   - eight warps take each block's sums out of tensor memory and add them,
//     times sx * sw, to running sums in registers (128 a thread), while the
//     tensor core fills the other tile.  The scales change every 128 of K, so
//     the running sum cannot stay in tensor memory.
// Few rows an expert are bound by reading the weights (16384 entries of 256 experts,
// K = 7168, I = 2048: 1.13 ms, 6.8 TB/s; 256 tokens in slabs, K = 2048, I = 768: 72 us,
// 768 tiles in 6 rounds).  Many (131072 entries of the 256 experts: 3.1 ms the first
// pass after a pause, 3.66 ms or 2.1 PFLOP/s repeated) by the power cap when repeated
// (1370 W, SM at 1.5 to 1.8 GHz), else by the chain of a block's product and its
// scaling over two tensor-memory tiles, about 850 clocks a block where the product
// alone takes 512.  Every expert's rows are rounded up to 128, which is about 12 % more
// products at 512 rows an expert, 25 % at 256.  Clusters of two with the weights by
// multicast, which spare a third of the reads from L2, took the same time.
// Rows past an expert's segment that share 32 of a tile with its last ones are
// loaded (whatever they hold, products of other rows do not see it) and never
// stored.
#include "expert.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kEpiWarps = 8;                     // warps that scale and store
constexpr int kThreads = 32 * (kEpiWarps + 4);   // + loader, + products, + two for the scales
// Registers a thread: 168 at launch (384 threads); the last warpgroup gives up
// what the first two, with 128 sums a thread, take: 2 * 216 + 72 = 3 * 168.
constexpr int kEpiRegs = 216, kOtherRegs = 72;
constexpr int kTM = 128, kTN = 256;              // tile: rows, weight rows
constexpr int kPart = 32;                        // rows of a part of a tile that is not full
constexpr int kABytes = kTM * 128, kBBytes = kTN * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kMaxStages = 4;
constexpr int kOutStride = 256 + 16;             // staged bf16 half row; the pad spreads the banks
constexpr int kOutBytes = kEpiWarps * 32 * kOutStride;
// The plain product stages its output rows in place of a fourth K block.
template <bool GATED>
constexpr int stages() { return GATED ? 4 : 3; }
template <bool GATED>
constexpr int ring_bytes() { return stages<GATED>() * kStageBytes + (GATED ? 0 : kOutBytes); }
constexpr int kSlots = 4;                        // K blocks of scales ahead of their sums

struct Tile {
    int e, row, rows, n0;  // expert, first row of the tile, valid rows in it, first weight row
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];  // ring of K blocks
    uint64_t tfull[2], tempty[2];            // tensor-memory tiles
    uint64_t sfull[kSlots], sempty[kSlots];  // scales
    uint64_t xchg;                           // the column halves' group maxima
    uint64_t drain;
    uint32_t tmem;
    int fail;
    int issued;                              // K blocks requested, for the drain
    int32_t scan[kThreads / 32];
    // The adding warps read a tile's place here once its sums are done; its entry is
    // written again eight tiles later, after their sums of the fourth.
    Tile tile[8];
    float scale[kSlots][2][kTM];             // sx * sw of each row, for the two weight blocks
    float amax[2][2][kTM];                   // [tile parity][column half][row]
};

__device__ __forceinline__ int row_tiles(const ExpertArgs &a, int e) {
    return (expert_rows(a, e) + kTM - 1) / kTM;
}

// Tile t of the list: experts in order; within one, row tiles run fastest, so
// that CTAs working at the same time share weights.  Where the counts are no
// layout's and their tiles' sum wrapped, a tile that is none has no rows.
__device__ __forceinline__ Tile find_tile(const ExpertArgs &a, const int32_t *pre, int t, int cols,
                                          int ntn) {
    int lo = 0, hi = a.E;  // pre[lo] <= t < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= t) lo = mid; else hi = mid;
    }
    const int mt = row_tiles(a, lo), local = t - pre[lo];
    const int n = local / max(mt, 1), i = local - n * mt;
    Tile r;
    r.e = lo;
    if (local < 0 || n >= ntn || mt == 0) {
        r.row = r.rows = r.n0 = 0;
        return r;
    }
    r.n0 = n * cols;
    r.row = expert_first(a, lo) + i * kTM;
    r.rows = min(expert_rows(a, lo) - i * kTM, kTM);
    return r;
}

// acc[2i], acc[2i+1] += v[2i] * s, v[2i+1] * s, two to an instruction.
__device__ __forceinline__ void fma_scaled(float *acc, const uint32_t (&v)[32], float s) {
    uint64_t ss;
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint64_t p, c;
        asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(acc[2 * i]), "f"(acc[2 * i + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(p), "l"(ss));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[2 * i]), "=f"(acc[2 * i + 1]) : "l"(c));
    }
}

__device__ __forceinline__ uint4 bf16x8(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void bulk_store_row(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap pmap,
                  const __grid_constant__ CUtensorMap wmap, const ExpertArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    // K blocks (the swizzle wants 1024-byte alignment), output rows, [E+1] tile prefix
    uint8_t *smem = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    __shared__ Shared sh;
    constexpr int kStages = stages<GATED>();
    int32_t *pre = reinterpret_cast<int32_t *>(smem + ring_bytes<GATED>());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const volatile int *fail = &sh.fail;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.tfull[i], 1);
            mbar_init(&sh.tempty[i], kEpiWarps);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.sfull[i], 2);
            mbar_init(&sh.sempty[i], kEpiWarps);
        }
        mbar_init(&sh.xchg, kEpiWarps);
        mbar_init(&sh.drain, 1);
        sh.fail = 0;
        sh.issued = 0;
        mbar_init_fence();
        tma_prefetch_map(&xmap);
        tma_prefetch_map(&wmap);
    }
    // after the wait: a predecessor's blocks that still have to allocate tensor
    // memory must find it free
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == kEpiWarps + 1) tmem_alloc<512>(&sh.tmem);
    tc_fence_before();
    const int cols = GATED ? 128 : kTN;  // output columns of a tile
    const int ntn = (a.N + cols - 1) / cols;
    block_exclusive_scan<kThreads>(
        a.E, [&](int e) { return row_tiles(a, e) * ntn; }, pre, sh.scan);
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // at most this many tiles where the experts' rows are disjoint: more are no layout's
    const int64_t most = ((int64_t)a.rows_cap / kTM + a.E) * ntn;
    const int total = pre[a.E] <= most ? min(pre[a.E], 0x7fffffff - (int)gridDim.x) : 0;
    const int G = a.K >> 7;

    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kEpiWarps) {
            // ---- loads ----
            int it = 0;
            for (int t = blockIdx.x; t < total && !__any_sync(kFullMask, *fail); t += gridDim.x) {
                const Tile q = find_tile(a, pre, t, cols, ntn);
                for (int g = 0; g < G; ++g, ++it) {
                    const int s = it % kStages;
                    const bool ok = it < kStages || mbar_wait_fast(&sh.empty[s], (it / kStages - 1) & 1, fail);
                    if (!__all_sync(kFullMask, ok)) {
                        sh.fail = 1;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *st = smem + s * kStageBytes;
                        expect_bytes(&sh.full[s], kStageBytes);
                        if (q.rows > kTM - kPart) {
                            tma_load_2d(st, &xmap, g * 128, q.row, &sh.full[s]);
                        } else {
                            // parts without a row start past the row space: zeros, and no
                            // reads (a decode batch of 16 rows an expert: 73.7 us, 76.2
                            // with whole tiles)
#pragma unroll
                            for (int i = 0; i < kTM; i += kPart)
                                tma_load_2d(st + i * 128, &pmap, g * 128,
                                            i < q.rows ? q.row + i : a.rows_cap, &sh.full[s]);
                        }
                        tma_load_3d(st + kABytes, &wmap, g * 128, q.n0, q.e, &sh.full[s]);
                        tma_load_3d(st + kABytes + kBBytes / 2, &wmap, g * 128,
                                    q.n0 + (GATED ? a.N : 128), q.e, &sh.full[s]);
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) sh.issued = it;
        } else if (warp == kEpiWarps + 1) {
            // ---- products ----
            constexpr uint32_t instr = e4m3_instr(kTM, kTN);
            int it = 0;
            for (int t = blockIdx.x; t < total && !__any_sync(kFullMask, *fail); t += gridDim.x) {
                for (int g = 0; g < G; ++g, ++it) {
                    const int s = it % kStages, b = it & 1;
                    const bool ok = (it < 2 || mbar_wait_fast(&sh.tempty[b], (it / 2 - 1) & 1, fail)) &&
                                    mbar_wait_fast(&sh.full[s], (it / kStages) & 1, fail);
                    if (!__all_sync(kFullMask, ok)) {
                        sh.fail = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = tile_desc(smem_addr(smem + s * kStageBytes));
                    const uint64_t db = tile_desc(smem_addr(smem + s * kStageBytes + kABytes));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 bytes of each row further
                            mma_e4m3(tmem + b * kTN, da + 2 * k, db + 2 * k, instr, k > 0);
                        mma_commit(&sh.empty[s]);
                        mma_commit(&sh.tfull[b]);
                    }
                    __syncwarp();
                }
            }
            // tensor memory and the barriers outlive the last product
            if (elect_one()) mma_commit(&sh.drain);
            __syncwarp();
            if (!mbar_wait(&sh.drain, 0, nullptr)) sh.fail = 1;
        } else {
            // ---- scales: rows r and r + 64, four K blocks at a time, the next four
            // in flight.  (Loaded by the adding warps, each from its own row, they cost
            // a third of the time: 32 lines a load, beside 64 KB of tensor memory.) ----
            const int r = (warp - kEpiWarps - 2) * 32 + lane;
            const int NB = GATED ? a.N / 64 : (a.N + 127) / 128;
            int it = 0, tiles = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total && !__any_sync(kFullMask, *fail); t += gridDim.x, ++tiles) {
                const Tile q = find_tile(a, pre, t, cols, ntn);
                if (warp == kEpiWarps + 2 && lane == 0) sh.tile[tiles & 7] = q;
                const int b0 = q.n0 / 128, b1 = GATED ? b0 + a.N / 128 : min(b0 + 1, NB - 1);
                const float *sw0 = a.w_scales + ((size_t)q.e * NB + b0) * G;
                const float *sw1 = a.w_scales + ((size_t)q.e * NB + b1) * G;
                const bool v0 = r < q.rows, v1 = r + 64 < q.rows;
                const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float4 n0 = v0 ? row_scales4(a, q.row + r, q.e, 0) : none;
                float4 n1 = v1 ? row_scales4(a, q.row + r + 64, q.e, 0) : none;
                for (int g4 = 0; ok && g4 < G; g4 += 4) {
                    const float x0[4] = {n0.x, n0.y, n0.z, n0.w}, x1[4] = {n1.x, n1.y, n1.z, n1.w};
                    if (g4 + 4 < G) {
                        if (v0) n0 = row_scales4(a, q.row + r, q.e, g4 + 4);
                        if (v1) n1 = row_scales4(a, q.row + r + 64, q.e, g4 + 4);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (g4 + i >= G) break;
                        const int s = it % kSlots;
                        const float w0 = __ldg(sw0 + g4 + i), w1 = __ldg(sw1 + g4 + i);
                        ok = it < kSlots || mbar_wait_fast(&sh.sempty[s], (it / kSlots - 1) & 1, fail);
                        ok = __all_sync(kFullMask, ok);
                        if (!ok) {
                            sh.fail = 1;
                            break;
                        }
                        sh.scale[s][0][r] = x0[i] * w0;
                        sh.scale[s][0][r + 64] = x1[i] * w0;
                        sh.scale[s][1][r] = x0[i] * w1;
                        sh.scale[s][1][r + 64] = x1[i] * w1;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.sfull[s]);
                        ++it;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // ---- scales, running sums, outputs ----
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;  // column half, row of the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        // the gated tile: this half's 64 gate columns, then the same 64 up columns
        const uint32_t col0 = half * (GATED ? 64 : 128), col1 = GATED ? 128 + half * 64 : col0 + 64;
        int it = 0, tiles = 0;
        for (int t = blockIdx.x; t < total && !__any_sync(kFullMask, *fail); t += gridDim.x, ++tiles) {
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
            bool ok = true;
            for (int g = 0; g < G; ++g, ++it) {
                const int b = it & 1, s = it % kSlots;
                ok = mbar_wait_fast(&sh.sfull[s], (it / kSlots) & 1, fail);
                const float s0 = sh.scale[s][GATED ? 0 : half][r], s1 = GATED ? sh.scale[s][1][r] : s0;
                ok = mbar_wait_fast(&sh.tfull[b], (it / 2) & 1, fail) && ok;
                if (!__all_sync(kFullMask, ok)) {
                    sh.fail = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = tmem + lanes + b * kTN;
                uint32_t v[2][32];
                tmem_ld(base + col0, v[0]);
                tmem_ld_wait(v[0]);
                tmem_ld(base + col0 + 32, v[1]);
                fma_scaled(acc, v[0], s0);
                tmem_ld_wait(v[1]);
                tmem_ld(base + col1, v[0]);
                fma_scaled(acc + 32, v[1], s0);
                tmem_ld_wait(v[0]);
                tmem_ld(base + col1 + 32, v[1]);
                fma_scaled(acc + 64, v[0], s1);
                tmem_ld_wait(v[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.tempty[b]);
                    mbar_arrive(&sh.sempty[s]);
                }
                fma_scaled(acc + 96, v[1], s1);
            }
            if (!ok) break;
            const Tile q = sh.tile[tiles & 7];
            const bool valid = r < q.rows;
            if constexpr (!GATED) {
                // Each thread's 256 bytes of its row go through shared memory to one
                // bulk copy: stored from registers, 32 rows an instruction, a tile took
                // 4300 clocks.
                const int c0 = q.n0 + half * 128;
                uint8_t *row = smem + kStages * kStageBytes + threadIdx.x * kOutStride;
                bulk_wait_read<0>();  // the last tile's copy has read them
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<uint4 *>(row + 16 * j) = bf16x8(acc + 8 * j);
                fence_proxy_async_smem();
                if (valid && c0 < a.N) {
                    bulk_store_row(static_cast<uint16_t *>(a.out) + (size_t)(q.row + r) * a.N + c0,
                                   row, 2u * (uint32_t)min(128, a.N - c0));
                    bulk_commit();
                }
                __syncwarp();
            } else {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    acc[i] = gated_silu(acc[i], acc[64 + i]);
                    amax = fmaxf(amax, fabsf(acc[i]));
                }
                const size_t at = (size_t)(q.row + r) * a.N + q.n0 + half * 64;
                if (a.out_quant == EP_QUANT_NONE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (valid) st_v4(static_cast<uint16_t *>(a.out) + at + 8 * j, bf16x8(acc + 8 * j));
                    continue;
                }
                // the row's other 64 columns are with the other half's warp
                sh.amax[tiles & 1][half][r] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.xchg);
                ok = mbar_wait_fast(&sh.xchg, tiles & 1, fail);
                if (!__all_sync(kFullMask, ok)) {
                    sh.fail = 1;
                    break;
                }
                amax = fmaxf(amax, sh.amax[tiles & 1][half ^ 1][r]);
                const float s = group_scale(amax);
                const int e8 = ue8m0_exponent(s);
                // The quotient by the fp32 scale or by the power of two (which the product
                // by inv gives already; its error is 0).  With divisions, whose slow path
                // is a call across 128 live sums, the prompt case took 4.7 ms, not 3.6.
                const bool f32 = a.out_quant == EP_QUANT_FP8_F32;
                const float by = f32 ? s : ue8m0_value(e8);
                const float inv = f32 ? __frcp_rn(s) : exp_reciprocal(e8);
                uint8_t *dst = static_cast<uint8_t *>(a.out) + at;
                if (valid) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                v[m] = group_quotient(acc[16 * j + 4 * i + m], by, inv);
                            p[i] = fp8x4(v[0], v[1], v[2], v[3]);
                        }
                        st_v4(dst + 16 * j, make_uint4(p[0], p[1], p[2], p[3]));
                    }
                    if (half == 0) store_out_scale(a, q.row + r, q.e, q.n0 / 128, s, e8);
                }
            }
        }
    }
    bulk_wait_read<0>();  // shared memory outlives the copies out of it
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sh.fail) {
        if (threadIdx.x == 0) raise_status(a.status, EP_ERR_TIMEOUT);
        // let the loads in flight land before the shared memory goes
        if ((int)threadIdx.x < kStages) {
            const int last = sh.issued - 1 - (int)threadIdx.x;
            if (last >= 0) mbar_wait(&sh.full[last % kStages], (last / kStages) & 1, nullptr);
        }
        __syncthreads();
    }
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        tmem_free<512>(tmem);
    }
}

// The driver's encoder, looked up once (the library links no libcuda).
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

}  // namespace

bool encode_bytes(CUtensorMap *map, const void *p, int rank, const int64_t *dims,
                  const int64_t *strides, const int *box, CUtensorMapSwizzle swizzle) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], ones[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = (cuuint64_t)dims[i];
        b[i] = (cuuint32_t)box[i];
        ones[i] = 1;
        if (i + 1 < rank) s[i] = (cuuint64_t)strides[i];
    }
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(p), d, s, b,
              ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_expert(const ExpertArgs &a, bool gated, cudaStream_t stream) {
    CUtensorMap xmap, pmap, wmap;
    const int64_t xdims[2] = {a.K, a.rows_cap}, xstride[1] = {a.K};
    const int64_t W = gated ? 2 * a.N : a.N;
    const int64_t wdims[3] = {a.K, W, a.E}, wstride[2] = {a.K, W * a.K};
    const int xbox[2] = {128, kTM}, pbox[2] = {128, kPart}, wbox[3] = {128, kTN / 2, 1};
    if (!encode_bytes(&xmap, a.x, 2, xdims, xstride, xbox) ||
        !encode_bytes(&pmap, a.x, 2, xdims, xstride, pbox) ||
        !encode_bytes(&wmap, a.w, 3, wdims, wstride, wbox))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + (gated ? ring_bytes<true>() : ring_bytes<false>()) + (a.E + 1) * 4;
    return gated ? launch_large<expert_kernel<true>>(sm_count(), kThreads, smem, stream, xmap, pmap,
                                                     wmap, a)
                 : launch_large<expert_kernel<false>>(sm_count(), kThreads, smem, stream, xmap, pmap,
                                                      wmap, a);
}

}  // namespace ep
