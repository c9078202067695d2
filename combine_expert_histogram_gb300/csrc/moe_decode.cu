// ep_moe_decode: a whole mixture-of-experts layer for a few tokens.
//
//   xq = 1x128 E4M3 of x,  g = W13[e][:I] xq,  u = W13[e][I:] xq,
//   hq = 1x128 E4M3 of silu(g) * u,  out[t] = sum over k of w[t,k] * W2[e] hq
//
// Bound by reading the picked experts' weights, once for each chunk of an expert's
// entries: once in all where experts get few.  Two kernels of the same
// body (rows of W13 against the tokens, rows of W2 against the gated results)
// and a small one for the weighted sum; all launched as programmatic
// dependents.  Each CTA groups the T*K entries by expert itself (at most 1024,
// in shared memory) into chunks of one expert and up to `cols` entries.  The
// units of work, (chunk, 128 weight rows, a part of their length), are split
// evenly over one persistent CTA per SM, which walks a contiguous run of them:
//   - a loader thread keeps a ring of 16 KB stages (128 rows x 128 bytes of the
//     weights) in flight, one tiled TMA copy each.  It never waits for the
//     previous kernel (weights are not its output), so the second kernel's ring
//     fills while the first one drains;
//   - eight warps quantise a chunk's entries into shared memory when the run
//     comes to the next expert;
//   - one thread issues the tensor core's E4M3 products: the weight rows are the
//     128 rows of A, the entries the columns of B (at least 16; those past the
//     chunk are whatever follows in shared memory, and are never read).  With
//     the entries as A and 64 weight rows as columns, twice as many instructions
//     of about 165 clocks each held the kernel to 3.6 TB/s; the m16n8k32 E4M3
//     instruction, which converts its operands on the vector pipes, to 2.8;
//   - four of these warps take each 128-deep block sum out of tensor memory, one
//     weight row a thread, and add it, scaled, to fp32 registers.
// 64 tokens to 8 of 256 experts, H = 7168, I = 2048 (9.76 GB): 1.48 ms, 6.6 TB/s; 8
// tokens (2.5 GB): 0.37 ms in a graph, 0.385 call by call, 6.5 to 6.7 TB/s.  One
// token to 8 experts, H = 2048, I = 768 (38 MB): 16 us, of which 2 pass before the
// first weights are asked for and 1 at each of the two waits between the kernels.
// Partial sums over parts of a row's length are added where they are read, in
// the order of the parts.
#include "expert.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;                        // quantise; the first four also scale and store
constexpr int kThreads = 32 * (kWarps + 2);      // + loader, + products
constexpr int kRows = 128;                       // weight rows of a unit
constexpr int kStageBytes = kRows * 128;
constexpr int kMaxStages = 12;
constexpr int kMaxCols = 32;                     // entries of a chunk
constexpr int kGroup = 4;                        // blocks of 128 taken together
constexpr int kMaxTiles = 4;                     // tensor-memory tiles of kGroup block sums
constexpr int kMaxEntries = EP_MOE_DECODE_MAX_ENTRIES;
constexpr int kSmemMax = 227 * 1024;
constexpr int kSmemHalf = 113 * 1024;            // two blocks an SM (1 KB of each is reserved)

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[kMaxTiles], tempty[kMaxTiles];
    uint64_t columns;              // a chunk's entries are in shared memory
    uint64_t drain;
    uint32_t tmem;
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

// Group up to 32 entries, one a lane, by one warp.
__device__ void group_few(const MoeArgs &a, int cols, Shared &sh) {
    const int n = a.T * a.K, lane = threadIdx.x & 31;
    int e = lane < n ? ld_dep(a.topk_idx + lane) : -1;
    if (e < -1 || e >= a.E) {
        if (blockIdx.x == 0) raise_status(a.status, EP_ERR_BAD_EXPERT_ID);
        e = -1;
    }
    const int key = e < 0 ? EP_MAX_EXPERTS : e;
    int before = 0, same = 0, count = 0;  // lower ids; the same id on lower lanes, on all
    for (int i = 0; i < n; ++i) {
        const int k = __shfl_sync(kFullMask, key, i);
        before += k < key;
        same += k == key && i < lane;
        count += k == key;
    }
    const bool head = e >= 0 && same % cols == 0;  // the first entry of a chunk
    int chunk = 0;
    for (int i = 0; i < n; ++i) {
        const int k = __shfl_sync(kFullMask, key, i), s = __shfl_sync(kFullMask, same, i);
        chunk += __shfl_sync(kFullMask, (int)head, i) && (k < key || (k == key && s < same));
    }
    if (e >= 0) sh.entry[before + same] = (uint16_t)lane;
    if (head)
        sh.chunk[chunk] = (uint32_t)e | (uint32_t)(before + same) << 10 |
                          (uint32_t)min(cols, count - same) << 20;
    const unsigned heads = __ballot_sync(kFullMask, head);
    if (lane == 0) sh.chunks = __popc(heads);
}

// Group the routed entries by expert.  `tmp` holds 2 * E + 1 ints and n 16-bit
// ids; every thread of the CTA calls it.  Every CTA must put the same entries
// into the same chunk.  Within a chunk their order is free (no entry's result
// depends on which column it takes), so only the entries of an expert with
// several chunks are ranked by counting the same ids before them.
__device__ void group_entries(const MoeArgs &a, int cols, int32_t *tmp, Shared &sh) {
    constexpr int kEach = (kMaxEntries + kThreads - 1) / kThreads;
    int32_t *cnt = tmp, *at = cnt + a.E;  // [E]; [E+1] first entry | first chunk << 16
    uint16_t *ids = reinterpret_cast<uint16_t *>(at + a.E + 1);  // [n]
    const int n = a.T * a.K;
    int mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int j = i * kThreads + threadIdx.x;
        mine[i] = j < n ? ld_dep(a.topk_idx + j) : -1;
    }
    for (int e = threadIdx.x; e < a.E; e += kThreads) cnt[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int j = i * kThreads + threadIdx.x;
        if (mine[i] < -1 || mine[i] >= a.E) {
            if (blockIdx.x == 0) raise_status(a.status, EP_ERR_BAD_EXPERT_ID);
            mine[i] = -1;
        }
        if (j < n) ids[j] = (uint16_t)(mine[i] >= 0 ? mine[i] : a.E);
        if (mine[i] >= 0) atomicAdd(cnt + mine[i], 1);
    }
    __syncthreads();
    // both counts in one scan: neither total is above 1024
    block_exclusive_scan<kThreads>(
        a.E, [&](int e) { return cnt[e] | (cnt[e] + cols - 1) / cols << 16; }, at, sh.scan);
    if (threadIdx.x == 0) sh.chunks = at[a.E] >> 16;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const int first = at[e] & 0xffff, end = at[e + 1] & 0xffff;
        for (int c = at[e] >> 16, f = first; f < end; ++c, f += cols)
            sh.chunk[c] = (uint32_t)e | (uint32_t)f << 10 | (uint32_t)min(cols, end - f) << 20;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = mine[i], j = i * kThreads + threadIdx.x;
        if (e < 0) continue;
        const int first = at[e] & 0xffff;
        int rank = 0;
        if ((at[e + 1] & 0xffff) - first <= cols)
            rank = atomicSub(cnt + e, 1) - 1;
        else
            for (int k = 0; k < j; ++k) rank += ids[k] == e;
        sh.entry[first + rank] = (uint16_t)j;
    }
    __syncthreads();
}

// a / b for a below 2^28 and a quotient below 2^21: the fp32 quotient is off by
// less than one, which the remainder tells.  A third of the latency of an integer
// division, of which a block's first unit takes six in a row.
__device__ __forceinline__ int quotient(uint32_t a, uint32_t b) {
    int q = (int)__fdividef((float)a, (float)b);
    const int r = (int)a - q * (int)b;
    if (r < 0) --q;
    else if (r >= (int)b) ++q;
    return q;
}

// A unit of the list: its chunk, first weight row, and 128-wide blocks [g0, g1).
struct Unit {
    uint32_t chunk;
    int c, row, part, g0, g1;
};
struct Units {
    int row_units, parts, G;
    __device__ __forceinline__ void blocks(Unit &u) const {
        u.g0 = parts == 1 ? 0 : quotient(G * u.part, parts);
        u.g1 = parts == 1 ? G : quotient(G * (u.part + 1), parts);
    }
    // Unit number i (i below their number).
    __device__ __forceinline__ Unit at(const Shared &sh, int i) const {
        Unit u;
        u.c = quotient(i, row_units * parts);
        const int v = i - u.c * row_units * parts, r = quotient(v, parts);
        u.part = v - r * parts;
        u.row = r * kRows;
        u.chunk = sh.chunk[u.c];
        blocks(u);
        return u;
    }
    // The one after u (there has to be one).
    __device__ __forceinline__ void next(const Shared &sh, Unit &u) const {
        if (++u.part == parts) {
            u.part = 0;
            u.row += kRows;
            if (u.row == row_units * kRows) {
                u.row = 0;
                u.chunk = sh.chunk[++u.c];
            }
        }
        blocks(u);
    }
};

// Eight values of group g of the chunk's entry `col`, for lane l of the half warp
// that takes the group: E4M3 bytes (q) and scale (s) where x is in 8 bits, else
// fp32 (v).  UP: the token's x; else silu(gate) * up of the first kernel's sums
// gu[part][T*K][2D].
struct Piece {
    uint4 raw[4];
    float s;
};
template <bool UP>
__device__ __forceinline__ Piece load_piece(const MoeArgs &a, const float *gu, int entry, int D,
                                            int g, int l) {
    Piece r;
    r.s = 0.0f;
    const int t = UP ? quotient(entry, a.K) : entry, G = D >> 7;
    const size_t at = (size_t)t * D + g * 128 + 8 * l;
    if (!UP) {
        const float *p = gu + (size_t)t * 2 * D + g * 128 + 8 * l;
        r.raw[0] = ld_dep_v4(p);
        r.raw[1] = ld_dep_v4(p + 4);
        r.raw[2] = ld_dep_v4(p + D);
        r.raw[3] = ld_dep_v4(p + D + 4);
    } else if (a.quant == EP_QUANT_NONE) {
        r.raw[0] = ld_dep_v4(static_cast<const uint16_t *>(a.x) + at);
    } else {
        const int32_t *p = reinterpret_cast<const int32_t *>(static_cast<const uint8_t *>(a.x) + at);
        r.raw[0].x = (uint32_t)ld_dep(p);
        r.raw[0].y = (uint32_t)ld_dep(p + 1);
        if (a.quant == EP_QUANT_FP8_F32) {
            r.s = ld_dep(static_cast<const float *>(a.x_scales) + (size_t)t * G + g);
        } else {
            const uint32_t word = (uint32_t)ld_dep(static_cast<const int32_t *>(a.x_scales) +
                                                   (size_t)t * ((G + 3) / 4) + (g >> 2));
            r.s = ue8m0_value(word >> (8 * (g & 3)) & 255u);
        }
    }
    return r;
}
__device__ __forceinline__ void add4(uint4 &s, uint4 v) {
    s.x = __float_as_uint(__uint_as_float(s.x) + __uint_as_float(v.x));
    s.y = __float_as_uint(__uint_as_float(s.y) + __uint_as_float(v.y));
    s.z = __float_as_uint(__uint_as_float(s.z) + __uint_as_float(v.z));
    s.w = __float_as_uint(__uint_as_float(s.w) + __uint_as_float(v.w));
}
__device__ __forceinline__ float gate_up(uint32_t g, uint32_t u) {
    return gated_silu(__uint_as_float(g), __uint_as_float(u));
}

// The chunk's entries as E4M3 rows in shared memory: xq[group][cols / 8] atoms of
// 8 rows x 128 bytes in 128-byte swizzle (16-byte piece j of row r lies at piece
// j ^ r), and xs[group][cols].  Half a warp takes a 1x128 group, 8 values a lane,
// with the next group's loads in flight.
template <bool UP>
__device__ __forceinline__ void load_columns(const MoeArgs &a, const float *gu, int gu_parts,
                                             uint32_t chunk, const Shared &sh, int D, int cols,
                                             uint8_t *xq, float *xs) {
    const int first = chunk >> 10 & 1023, n = (int)(chunk >> 20);
    const int G = D >> 7, items = n * G;
    const int l = threadIdx.x & 15, step = 2 * kWarps;
    // items w, w + step, ... of this warp's two halves; the bound is the same for
    // both, which shuffle together
    int i = threadIdx.x >> 4;
    int col = quotient(min(i, items - 1), G), g = min(i, items - 1) - col * G;
    Piece next = load_piece<UP>(a, gu, sh.entry[first + col], D, g, l);
#pragma unroll 1
    for (int w0 = i & ~1; w0 < items; w0 += step, i += step) {
        Piece p = next;
        const int c = col, gc = g, entry = sh.entry[first + col];
        if (w0 + step < items) {
            const int j = min(i + step, items - 1);
            col = quotient(j, G);
            g = j - col * G;
            next = load_piece<UP>(a, gu, sh.entry[first + col], D, g, l);
        }
        uint2 q = make_uint2(p.raw[0].x, p.raw[0].y);
        float s = p.s;
        if (!UP || a.quant == EP_QUANT_NONE) {
            float v[8];
            if (UP) {
                const uint32_t w[4] = {p.raw[0].x, p.raw[0].y, p.raw[0].z, p.raw[0].w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    v[2 * m] = bf16_lo(w[m]);
                    v[2 * m + 1] = bf16_hi(w[m]);
                }
            } else {
                // the sums' other parts, in order, all their loads in flight
                if (gu_parts > 1) {
                    const size_t step_k = (size_t)a.T * a.K * 2 * D;
                    Piece o[3];
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        o[k] = load_piece<UP>(a, gu + min(k + 1, gu_parts - 1) * step_k, entry, D, gc, l);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        if (k + 1 >= gu_parts) break;
#pragma unroll
                        for (int m = 0; m < 4; ++m) add4(p.raw[m], o[k].raw[m]);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint4 x = p.raw[m], y = p.raw[2 + m];
                    v[4 * m] = gate_up(x.x, y.x);
                    v[4 * m + 1] = gate_up(x.y, y.y);
                    v[4 * m + 2] = gate_up(x.z, y.z);
                    v[4 * m + 3] = gate_up(x.w, y.w);
                }
            }
            float amax = 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m) amax = fmaxf(amax, fabsf(v[m]));
#pragma unroll
            for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
            s = group_scale(amax);
#pragma unroll
            for (int m = 0; m < 8; ++m) v[m] = __fdiv_rn(v[m], s);
            q = make_uint2(fp8x4(v[0], v[1], v[2], v[3]), fp8x4(v[4], v[5], v[6], v[7]));
        }
        if (i < items) {
            *reinterpret_cast<uint2 *>(xq + (gc * cols + c) * 128 + (((l >> 1) ^ (c & 7)) << 4) +
                                       8 * (l & 1)) = q;
            if (l == 0) xs[gc * cols + c] = s;
        }
        __syncwarp();
    }
}

// dst[part][T*K][R] = rows of W13 (UP: R = 2I, D = H) or of W2 (R = H, D = I)
// against the entries, fp32.
template <bool UP, int COLS>
__global__ void __launch_bounds__(kThreads, 2)
    rows_kernel(const __grid_constant__ CUtensorMap wmap, const MoeArgs a, const float *gu,
                int gu_parts, float *dst, int parts, int stages) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Shared sh;
    constexpr int cols = COLS;                       // entries of a chunk
    constexpr int kN = COLS < 16 ? 16 : COLS;        // columns of a product
    constexpr int kTileCols = kGroup * kN, kTiles = COLS < 32 ? 4 : 2;
    const int D = UP ? a.H : a.I, R = UP ? 2 * a.I : a.H, G = D >> 7;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // entries first: the products' unused columns read on into the ring
    uint8_t *xq = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    uint8_t *ring = xq + G * cols * 128;
    float *xs = reinterpret_cast<float *>(ring + stages * kStageBytes);  // [G][cols]
    const volatile int *fail = &sh.fail;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&sh.tfull[i], 1);
            mbar_init(&sh.tempty[i], 4);
        }
        mbar_init(&sh.columns, kWarps);
        mbar_init(&sh.drain, 1);
        sh.fail = 0;
        sh.issued = 0;
        mbar_init_fence();
        tma_prefetch_map(&wmap);
    }
    if (UP) {  // the ids may be the previous kernel's; for the second kernel they are complete
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = EP_OK;
        __syncwarp();  // before this warp's group_few may raise a code
    }
    // the first kernel lets the second start only once it holds its tensor memory
    if (warp == kWarps + 1) tmem_alloc<kTiles * kTileCols>(&sh.tmem);
    const bool few = a.T * a.K <= 32;
    if (few && warp == 0) group_few(a, cols, sh);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = sh.tmem;
    if (!few) group_entries(a, cols, reinterpret_cast<int32_t *>(ring), sh);
    const int row_units = R / kRows;
    const Units units = {row_units, parts, G};
    // at most 1024 chunks of 256 row units in 4 parts, 2^20; the grid is the SMs
    const uint32_t total = (uint32_t)sh.chunks * row_units * parts;
    const int u0 = quotient(total * blockIdx.x, gridDim.x);
    const int u1 = quotient(total * (blockIdx.x + 1), gridDim.x);

    if (warp == kWarps) {
        // ---- loads ----
        fence_proxy_async_smem();  // the ring held the grouping's counters
        int it = 0, s = 0;
        uint32_t lap = 0;
        Unit un;
        for (int u = u0; u < u1 && !__any_sync(kFullMask, *fail); ++u) {
            if (u == u0) un = units.at(sh, u);
            else units.next(sh, un);
            for (int g = un.g0; g < un.g1; ++g, ++it) {
                const bool ok = lap == 0 || mbar_wait_fast(&sh.empty[s], (lap - 1) & 1, fail);
                if (!__all_sync(kFullMask, ok)) {
                    sh.fail = 1;
                    break;
                }
                if (elect_one()) {
                    expect_bytes(&sh.full[s], kStageBytes);
                    tma_load_3d_once(ring + s * kStageBytes, &wmap, g * 128, un.row,
                                     un.chunk & 1023, &sh.full[s]);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ++lap;
                }
            }
        }
        if (lane == 0) sh.issued = it;
    } else if (warp == kWarps + 1) {
        // ---- products ----
        constexpr uint32_t instr = e4m3_instr(kRows, kN);
        int tile = 0, s = 0, loaded = 0;
        uint32_t lap = 0;
        uint32_t have = 0xffffffffu;
        bool ok = true;
        Unit un;
        for (int u = u0; ok && u < u1; ++u) {
            if (u == u0) un = units.at(sh, u);
            else units.next(sh, un);
            if (un.chunk != have) {
                have = un.chunk;
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.columns, loaded & 1, fail));
                ++loaded;
            }
            for (int g0 = un.g0; ok && g0 < un.g1; g0 += kGroup, ++tile) {
                const int b = tile % kTiles, n = min(kGroup, un.g1 - g0);
                ok = tile < kTiles || mbar_wait_fast(&sh.tempty[b], (tile / kTiles - 1) & 1, fail);
                for (int k = 0; k < n; ++k) {
                    ok = mbar_wait_fast(&sh.full[s], lap & 1, fail) && ok;
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = tile_desc(smem_addr(ring + s * kStageBytes));
                    const uint64_t db = tile_desc(smem_addr(xq + (g0 + k) * cols * 128));
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_e4m3(tmem + b * kTileCols + k * kN, da + 2 * j, db + 2 * j,
                                     instr, j > 0);
                        mma_commit(&sh.empty[s]);
                        if (k == n - 1) mma_commit(&sh.tfull[b]);
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ++lap;
                    }
                }
            }
        }
        if (!ok) sh.fail = 1;
        // tensor memory and the barriers outlive the last product
        if (elect_one()) mma_commit(&sh.drain);
        __syncwarp();
        if (!mbar_wait(&sh.drain, 0, nullptr)) sh.fail = 1;
    } else {
        // ---- entries, scales, sums.  After a wait that ran out the loops go on
        // (every later wait returns at once), so that all warps meet at the barriers ----
        const bool adds = warp < 4;  // one for each 32 lanes of tensor memory
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float *scales = UP ? a.w13_scales : a.w2_scales;
        // the weight scales of up to 32 blocks, one a lane; those of the next blocks
        // or of the next unit are in flight meanwhile
        auto fetch = [&](const Unit &un, int g0) {
            return g0 + lane < un.g1
                       ? __ldg(scales + ((size_t)(un.chunk & 1023) * row_units + (un.row >> 7)) * G + g0 + lane)
                       : 0.0f;
        };
        uint32_t have = 0xffffffffu;  // the chunk whose entries are in xq
        int tile = 0;
        Unit un = {};
        float wnext = 0.0f;
        if (u0 < u1) {
            un = units.at(sh, u0);
            if (adds) wnext = fetch(un, un.g0);
        }
        if (!UP) asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's sums
        for (int u = u0; u < u1; ++u) {
            const int first = un.chunk >> 10 & 1023, n = (int)(un.chunk >> 20);
            if (un.chunk != have) {
                consumer_sync();  // every warp is done with the old entries
                load_columns<UP>(a, gu, gu_parts, un.chunk, sh, D, cols, xq, xs);
                fence_proxy_async_smem();
                consumer_sync();
                if (lane == 0) mbar_arrive(&sh.columns);
                have = un.chunk;
            }
            const Unit now = un;
            if (u + 1 < u1) units.next(sh, un);
            if (!adds) continue;
            float acc[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
            for (int g32 = now.g0; g32 < now.g1; g32 += 32) {
                const float w = wnext;
                if (g32 + 32 < now.g1) wnext = fetch(now, g32 + 32);
                else if (u + 1 < u1) wnext = fetch(un, un.g0);
                for (int g0 = g32; g0 < min(g32 + 32, now.g1); g0 += kGroup, ++tile) {
                    const int b = tile % kTiles, m = min(kGroup, now.g1 - g0);
                    const bool ok = mbar_wait_fast(&sh.tfull[b], (tile / kTiles) & 1, fail);
                    if (!__all_sync(kFullMask, ok)) sh.fail = 1;
                    tc_fence_after();
                    // eight entries of all the tile's blocks at a time (what lies past
                    // the last block is read and not used)
                    float s[kGroup];
#pragma unroll
                    for (int k = 0; k < kGroup; ++k) s[k] = __shfl_sync(kFullMask, w, g0 - g32 + k);
#pragma unroll
                    for (int c = 0; c < COLS; c += 8) {
                        if (c >= n) break;
                        uint32_t v[kGroup][8];
#pragma unroll
                        for (int k = 0; k < kGroup; ++k)
                            tmem_ld(tmem + lanes + b * kTileCols + k * kN + c, v[k]);
#pragma unroll
                        for (int k = 0; k < kGroup; ++k) tmem_ld_wait(v[k]);
#pragma unroll
                        for (int k = 0; k < kGroup; ++k) {
                            if (k >= m) break;
                            const float4 x0 = *reinterpret_cast<const float4 *>(xs + (g0 + k) * cols + c);
                            const float4 x1 = *reinterpret_cast<const float4 *>(xs + (g0 + k) * cols + c + 4);
                            const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[c + i] = fmaf(__uint_as_float(v[k][i]), s[k] * x[i], acc[c + i]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.tempty[b]);
                }
            }
            float *out = dst + (size_t)now.part * a.T * a.K * R + now.row + threadIdx.x;
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                if (i >= n) break;
                out[(size_t)sh.entry[first + i] * R] = acc[i];
            }
        }
    }
    __syncwarp();
    tc_fence_before();
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
    if (warp == kWarps + 1) {
        tc_fence_after();
        tmem_free<kTiles * kTileCols>(tmem);
    }
}

// out[t] = sum over k of w[t,k] * (sum over parts of y[part][t*K + k]), 4 columns
// a thread.  The loads of 8 entries are in flight together.
__global__ void __launch_bounds__(128) sum_kernel(const MoeArgs a, const float *y, int parts) {
    constexpr int kBatch = 8;
    const int per = a.H / 4, i = blockIdx.x * 128 + threadIdx.x;
    const int t = i / per, c = i - t * per;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.T) return;
    float acc[4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
        int e[kBatch];
        float w[kBatch];
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int entry = t * a.K + min(k0 + k, a.K - 1);
            e[k] = ld_dep(a.topk_idx + entry);
            w[k] = ld_dep(a.topk_w + entry);
            // what an entry that is not routed holds is loaded too, and not used
            v[k] = ld_dep_v4(y + (size_t)entry * a.H + 4 * c);
        }
        float s[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            s[k][0] = __uint_as_float(v[k].x);
            s[k][1] = __uint_as_float(v[k].y);
            s[k][2] = __uint_as_float(v[k].z);
            s[k][3] = __uint_as_float(v[k].w);
        }
        for (int p = 1; p < parts; ++p) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                v[k] = ld_dep_v4(y + ((size_t)p * a.T * a.K + t * a.K + min(k0 + k, a.K - 1)) * a.H + 4 * c);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                s[k][0] += __uint_as_float(v[k].x);
                s[k][1] += __uint_as_float(v[k].y);
                s[k][2] += __uint_as_float(v[k].z);
                s[k][3] += __uint_as_float(v[k].w);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k0 + k >= a.K || e[k] < 0 || e[k] >= a.E) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[m] = fmaf(w[k], s[k][m], acc[m]);
        }
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + (size_t)t * a.H + 4 * c) =
        make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
}

// Entries of a chunk: what experts get on average, with room for twice that, as
// long as the entries leave most of the shared memory to the ring.
int chunk_cols(const MoeArgs &a, int D) {
    int cols = 8;
    while (cols < kMaxCols && cols * a.E < 2 * a.T * a.K && 2 * cols * D <= 128 * 1024) cols *= 2;
    return cols;
}

// Parts a row's length is cut into: with few entries there are few 128-row units,
// and the SM with one more than the others sets the time.  1 from 24 units an SM
// on, 2 from 8 on (how many there will be is not known to a few percent), below
// that the best share-out of 1 to 4.
int row_parts(int entries, int E, int R, int D) {
    const int sms = sm_count(), G = D / 128;
    const int64_t units = (int64_t)(entries < E ? entries : E) * (R / kRows);
    if (units >= 24 * sms) return 1;
    if (units >= 8 * sms) return G >= 4 ? 2 : 1;
    int best = 1;
    double most = 0.0;
    for (int p = 1; p <= 4 && G >= 2 * p; ++p) {
        const int64_t u = units * p;
        const double even = (double)u / ((u + sms - 1) / sms * sms);
        if (even > most + 0.03) {
            most = even;
            best = p;
        }
    }
    return best;
}

template <bool UP, int COLS>
cudaError_t launch_cols(const MoeArgs &a, const float *gu, int gu_parts, float *dst, int parts,
                        cudaStream_t stream) {
    const int D = UP ? a.H : a.I, G = D / 128;
    const int64_t R = UP ? 2 * a.I : a.H;
    const int64_t dims[3] = {D, R, a.E}, strides[2] = {D, R * D};
    const int box[3] = {128, kRows, 1};
    CUtensorMap wmap;
    if (!encode_bytes(&wmap, UP ? a.w13 : a.w2, 3, dims, strides, box)) return cudaErrorInvalidValue;
    const int fixed = 1024 + G * COLS * (128 + 4) + (int)sizeof(Shared);
    // Half of an SM's shared memory where that leaves a ring of five stages: the next
    // kernel's blocks then start beside this one's and load their weights.  H = 7168,
    // I = 2048, E = 256 (the second kernel's; the first has room for two stages): 64
    // tokens 1.49 ms (1.54 with all of the memory), 8 tokens 371 us (375), 1 token
    // 65.6 (64.5).  H = 2048, I = 768, E = 128: 1, 2, 4, 16, 64 tokens 15.7, 26.0,
    // 36.8, 77.4, 119 us (16.4, 25.1, 38.5, 78.0, 121).  13 tokens of 20 experts, H =
    // 1152, I = 640: 21.1 us either way.
    const int half = (kSmemHalf - fixed) / kStageBytes, fit = (kSmemMax - fixed) / kStageBytes;
    const int stages = half >= 5 ? half : fit < kMaxStages ? fit : kMaxStages;
    const size_t smem = 1024 + (size_t)G * COLS * (128 + 4) + (size_t)stages * kStageBytes;
    return launch_large<rows_kernel<UP, COLS>>(sm_count(), kThreads, smem, stream, wmap, a, gu,
                                               gu_parts, dst, parts, stages);
}

template <bool UP>
cudaError_t launch_rows(const MoeArgs &a, const float *gu, int gu_parts, float *dst, int parts,
                        cudaStream_t stream) {
    switch (chunk_cols(a, UP ? a.H : a.I)) {
        case 8: return launch_cols<UP, 8>(a, gu, gu_parts, dst, parts, stream);
        case 16: return launch_cols<UP, 16>(a, gu, gu_parts, dst, parts, stream);
        default: return launch_cols<UP, 32>(a, gu, gu_parts, dst, parts, stream);
    }
}

}  // namespace

size_t moe_workspace_bytes(int T, int K, int E, int H, int I) {
    const int n = T * K;
    return (size_t)n * 4 * ((size_t)row_parts(n, E, 2 * I, H) * 2 * I + (size_t)row_parts(n, E, H, I) * H);
}

size_t moe_workspace_bytes_up_to(int T, int K, int E, int H, int I) {
    size_t most = 0;  // fewer tokens may be cut into more parts
    for (int t = 1; t <= T; ++t) {
        const size_t b = moe_workspace_bytes(t, K, E, H, I);
        if (b > most) most = b;
    }
    return most;
}

cudaError_t launch_moe_decode(const MoeArgs &a, void *workspace, cudaStream_t stream) {
    const int n = a.T * a.K;
    const int p1 = row_parts(n, a.E, 2 * a.I, a.H), p2 = row_parts(n, a.E, a.H, a.I);
    float *gu = static_cast<float *>(workspace), *y = gu + (size_t)p1 * n * 2 * a.I;
    cudaError_t err = launch_rows<true>(a, nullptr, 0, gu, p1, stream);
    if (err != cudaSuccess) return err;
    err = launch_rows<false>(a, gu, p1, y, p2, stream);
    if (err != cudaSuccess) return err;
    const long long threads = (long long)a.T * (a.H / 4);
    return launch_kernel(sum_kernel, (int)((threads + 127) / 128), 128, 0, stream, true, a,
                         (const float *)y, p2);
}

}  // namespace ep
