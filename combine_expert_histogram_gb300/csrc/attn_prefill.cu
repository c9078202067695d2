// ep_attn_prefill: causal attention of prompts and of their chunks over the paged cache.
//
//   S = Q K^T,  P = exp(scale S - m),  O = sum P V,  l = sum P,  out = O / l
//
// with the running maximum m of a row.  A block has 256 rows, the tokens of one sequence times
// the query heads that share a key head, in two tiles of 128, and goes once over the 128-key
// tiles that its rows see.  Roles:
//   - a loader keeps a ring of key and value tiles in flight by tiled TMA loads, page by
//     page;
//   - one thread issues the products on tcgen05: S of a tile into tensor memory, and P V
//     with P read from tensor memory, where it takes the place of S.  The two row tiles
//     alternate, so that one tile's exponentials run under the other's products;
//   - two warpgroups, a thread a row, take S out of tensor memory, and put P back as bf16.
//     m is let lag behind the true maximum by up to 2^8 (P and l stay far inside fp32, and
//     P's relative rounding is the same), so that O is rescaled only in the rare tiles where
//     a row's maximum jumps;
//   - 8-bit caches: a warpgroup turns the E4M3 tiles into bf16, row by row, which is exact
//     (a power of two times three bits).  bf16 caches: two warps look for values that are
//     not finite in tiles that not all rows see: 0 * NaN would reach the other rows.
#include "attn.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTile = 128;   // rows of a tile, keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 8.0f;  // log2 of how far m may be behind

template <int D, bool FP8>
struct Cfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // registers a thread: 128 or 168 at launch
    static constexpr int kSoftRegs = FP8 ? 176 : 208, kOtherRegs = FP8 ? 80 : 88;
    static constexpr int kPanels = D / 64;               // 128-byte columns of a tile
    static constexpr int kPanel = kTile * 128;
    static constexpr int kStage = kPanels * kPanel;      // a bf16 tile
    static constexpr int kStages = FP8 ? 4 : 5;
    static constexpr int kRaw = FP8 ? kTile * D : 0, kRaws = 2;
    static constexpr int kSmem = 1024 + (2 + kStages) * kStage + kRaws * kRaw;
};

struct PrefillArgs {
    AttnArgs a;
    int G, box;  // query heads a key head; cache rows of a TMA box
};

struct Shared {
    uint64_t full[5], empty[5], raw_full[2], raw_empty[2];
    uint64_t q_full, s_full[2], p_ready[2], o_full[2], v_check, v_ok, drain;
    int64_t sums[16];
    int64_t before;
    uint32_t tmem;
    int fail, fix, issued;
    int b, block;
};

// bf16 x bf16 -> fp32; the second factor's rows may be along K (values) instead of N.
constexpr uint32_t bf16_instr(int n, bool b_rows_k) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)b_rows_k << 16 | (uint32_t)(n / 8) << 17 |
           (uint32_t)(kTile / 16) << 24;
}
// Descriptor of a value tile: 64 channels a 128-byte row, the rows along K, in 128-byte
// swizzle: 8 rows 1024 bytes apart, the next 64 channels a panel further.
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3ffffu) >> 4) | (uint64_t)(kTile * 128 >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"((uint32_t)accumulate)
        : "memory");
}
// The first factor in tensor memory.
__device__ __forceinline__ void mma_bf16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(instr), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// In the upper bit of each half: whether that bf16 is an infinity or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// w with the halves that are not finite as 0.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
    const uint32_t n = not_finite(w);
    return w & ~((n >> 15) * 0xffffu);
}

// What a block works on, the same for all its threads.
struct Block {
    int b, h;            // sequence, key head
    int row0, rows;      // first row (token * G + head) in the sequence, rows of the block
    int first, pos0;     // token of q that is the sequence's first, its position
    int minpos, maxpos;  // of the block's rows
    int lo, S;           // keys [lo, maxpos] and [0, S), S <= lo, are seen by some row
    int tile0, ns, nt;   // tiles 0 .. ns-1, then from tile0 on, nt in all
    int window, sinks;
    __device__ __forceinline__ int key(int i) const { return (i < ns ? i : tile0 + i - ns) * kTile; }
    // Not all rows see all of the tile's keys.
    __device__ __forceinline__ bool edge(int key) const {
        return !(key + kTile - 1 <= minpos &&
                 (!window || key > maxpos - window || key + kTile <= sinks));
    }
    // Some row may see one of the keys [key, key + n).
    __device__ __forceinline__ bool wanted(int key, int n) const {
        return key <= maxpos && (key + n > lo || key < S);
    }
};

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ PrefillArgs d) {
    using C = Cfg<D, FP8>;
    constexpr int kStages = C::kStages;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    uint8_t *smem = raw_smem + (1024 - (smem_addr(raw_smem) & 1023)) % 1024;
    __shared__ Shared sh;
    uint8_t *ring = smem + 2 * C::kStage, *raws = ring + kStages * C::kStage;
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const volatile int *fail = &sh.fail;
    constexpr int kMmaWarp = FP8 ? 12 : 9;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], FP8 ? 4 : 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.q_full, 8);
        mbar_init(&sh.v_check, 1);
        mbar_init(&sh.v_ok, 2);
        mbar_init(&sh.drain, 1);
        sh.fail = sh.fix = sh.issued = 0;
        sh.b = -1;
        mbar_init_fence();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the block's rows: blocks of 256 rows, a sequence's last ones (with the most keys)
    // first ----
    Block k;
    k.h = blockIdx.x % a.kv.Hkv;
    const int64_t index = blockIdx.x / a.kv.Hkv;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.seq.B; b0 += C::kThreads) {
        const int b = b0 + threadIdx.x;
        int64_t n = 0;
        if (b < a.seq.B) n = ((int64_t)seq_span(a.seq, a.kv.page_size, b).n * d.G + 2 * kTile - 1) / (2 * kTile);
        int64_t incl = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, incl, s);
            if (lane >= s) incl += o;
        }
        __syncthreads();
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        int64_t all = 0, below = 0;
#pragma unroll
        for (int i = 0; i < C::kThreads / 32; ++i) {
            if (i == warp) below = all;
            all += sh.sums[i];
        }
        incl += before + below;
        if (index >= incl - n && index < incl) {
            sh.b = b;
            sh.block = (int)(incl - 1 - index);
        }
        before += all;
        if (before > index) break;
    }
    __syncthreads();
    if (sh.b < 0) return;
    k.b = sh.b;
    {
        const Span sp = seq_span(a.seq, a.kv.page_size, k.b);
        k.first = sp.first;
        k.pos0 = sp.len - sp.n;
        k.row0 = sh.block * 2 * kTile;
        k.rows = min(sp.n * d.G - k.row0, 2 * kTile);
        k.minpos = k.pos0 + k.row0 / d.G;
        k.maxpos = k.pos0 + (k.row0 + k.rows - 1) / d.G;
        k.window = a.window;
        k.sinks = k.S = a.sinks;
        k.lo = a.window && k.minpos >= a.window ? k.minpos - a.window + 1 : 0;
        if (k.S >= k.lo) k.lo = k.S = 0;
        k.tile0 = k.lo / kTile;
        k.ns = min((k.S + kTile - 1) / kTile, k.tile0);
        k.nt = k.maxpos < 0 ? 0 : k.ns + k.maxpos / kTile + 1 - k.tile0;
    }
    const int tiles = k.rows > kTile ? 2 : 1;  // row tiles
    if (warp == kMmaWarp) tmem_alloc<512>(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;  // S (and P) of both tiles, then O of both

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        // ---- a thread's row ----
        const int t = warp >> 2, local = t * kTile + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + t * kTile + lanes, o_at = tmem + 2 * kTile + t * D + lanes;
        const bool valid = local < k.rows;
        const int row = k.row0 + local, token = row / d.G;
        const int pos = valid ? k.pos0 + token : -1;
        const int64_t head = (int64_t)k.h * d.G + (row - token * d.G);
        const int64_t q_off = valid ? (k.first + token) * a.q_stride + head * D : -1;
        const int64_t o_off = valid ? ((int64_t)(k.first + token) * a.Hq + head) * D : -1;
        constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte chunks a row, rows an instruction
        const uint32_t mine = smem_addr(smem) + t * C::kStage;
        const int wrow = (warp & 3) * 32;
        {
            uint4 x[32 / RP];
#pragma unroll
            for (int i = 0; i < 32 / RP; ++i) {
                const int64_t off = __shfl_sync(kFullMask, q_off, i * RP + lane / CH);
                x[i] = off >= 0 ? ld_dep_v4(a.q + off + 8 * (lane % CH)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 32 / RP; ++i) {
                const int r = wrow + i * RP + lane / CH, ch = lane % CH;
                sts16(mine + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7)), x[i]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        }
        const float sl2 = a.scale * kLog2e;
        float m = -INFINITY, l = 0.0f;  // m in S's units
        bool ok = true;
        if (t < tiles) {
            int wmin = pos, wmax = pos;  // of the warp's rows; rows that are none see nothing
#pragma unroll
            for (int x = 16; x; x >>= 1) {
                wmin = min(wmin, __shfl_xor_sync(kFullMask, wmin, x));
                wmax = max(wmax, __shfl_xor_sync(kFullMask, wmax, x));
            }
            for (int i = 0; i < k.nt; ++i) {
                const int key = k.key(i);
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.s_full[t], i & 1, fail));
                if (!ok) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld(s_at + 32 * x, v[x]);
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld_wait(v[x]);
                if (!(key + kTile - 1 <= wmin && (!a.window || key > wmax - a.window || key + kTile <= a.sinks))) {
                    const int hi = pos - key, lo = a.window && hi >= a.window ? hi - a.window + 1 : 0, s = a.sinks - key;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int n = 32 * x + j;
                            if (!(n <= hi && (n >= lo || n < s))) v[x][j] = 0xff800000u;  // -infinity
                        }
                }
                float top = m;
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(v[x][j]));
                const bool grown = top > m && !((top - m) * sl2 <= kLag);
                if (__any_sync(kFullMask, grown)) {
                    const float next = grown ? top : m;
                    const float f = grown ? exp2_fast((m - next) * sl2) : 1.0f;
                    l *= f;
                    m = next;
                    if (i > 0) {
#pragma unroll 1
                        for (int x = 0; x < D / 32; ++x) {
                            uint32_t o[32];
                            tmem_ld(o_at + 32 * x, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st(o_at + 32 * x, o);
                        }
                    }
                }
                // a row that has seen no key yet subtracts 0 from its -infinities
                const float base = m == -INFINITY ? 0.0f : -m * sl2;
                const uint64_t sl = pair(sl2, sl2), bb = pair(base, base);
                uint64_t acc0 = pair(l, 0.0f), acc1 = pair(0.0f, 0.0f);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        uint64_t e = pair(__uint_as_float(v[x][2 * j]), __uint_as_float(v[x][2 * j + 1]));
                        asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(e) : "l"(sl), "l"(bb));
                        float e0, e1;
                        unpair(e, e0, e1);
                        e0 = exp2_fast(e0);
                        e1 = exp2_fast(e1);
                        p[j] = pack_bf16(e0, e1);
                        e = pair(e0, e1);
                        if (j & 1)
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc1) : "l"(e));
                        else
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc0) : "l"(e));
                    }
                    tmem_st(s_at + 16 * x, p);
                }
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc0) : "l"(acc1));
                float l0, l1;
                unpair(acc0, l0, l1);
                l = l0 + l1;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[t]);
            }
            if (ok && k.nt > 0) ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_full[t], 0, fail));
            if (!ok) sh.fail = 1;
            if (ok) {
                tc_fence_after();
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const bool fix = sh.fix != 0 && k.nt > 0;
                const int64_t o_here = o_off;
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t o[32];
                    if (k.nt > 0) {
                        tmem_ld(o_at + 32 * x, o);
                        tmem_ld_wait(o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0;
                    }
                    if (l == 0.0f) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0;  // sees no key
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    if (fix) {
                        // values that the products were spared, added where a row sees them
                        for (int i = 0; i < k.nt; ++i) {
                            const int key = k.key(i);
                            if (!k.edge(key)) continue;
                            for (int j = key; j <= min(pos, key + kTile - 1); ++j) {
                                if (a.window && j <= pos - a.window && j >= a.sinks) continue;
                                const int page = page_of(a.kv, a.seq, k.b, j / a.kv.page_size);
                                if (page < 0) continue;
                                const int r = j % a.kv.page_size;
                                const uint8_t *src = a.kv.v + page * a.kv.page_stride + r * a.kv.row_stride + k.h * a.kv.head_stride;
                                const bool none = FP8 && a.kv.v_scales[((int64_t)page * a.kv.Hkv + k.h) * a.kv.page_size + r] == 255;
#pragma unroll
                                for (int n = 0; n < 16; ++n) {
                                    uint32_t w;
                                    if constexpr (FP8) {
                                        const uint32_t e = reinterpret_cast<const uint16_t *>(src)[16 * x + n];
                                        w = (none || (e & 0x7f) == 0x7f ? 0x7fffu : 0u) |
                                            (none || (e & 0x7f00) == 0x7f00 ? 0x7fff0000u : 0u);
                                    } else {
                                        w = reinterpret_cast<const uint32_t *>(src)[16 * x + n];
                                        w &= (not_finite(w) >> 15) * 0xffffu;
                                    }
                                    if (w) o[n] = pack_bf16(bf16_lo(o[n]) + bf16_lo(w), bf16_hi(o[n]) + bf16_hi(w));
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int ch = 4 * x + j;
                        sts16(mine + (ch >> 3) * C::kPanel + (wrow + lane) * 128 + 16 * ((ch & 7) ^ (lane & 7)),
                              make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32 / RP; ++i) {
                    const int64_t off = __shfl_sync(kFullMask, o_here, i * RP + lane / CH);
                    const int r = wrow + i * RP + lane / CH, ch = lane % CH;
                    if (off >= 0)
                        st_v4(a.out + off + 8 * ch, lds16(mine + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7))));
                }
                if (a.lse && valid)
                    a.lse[o_off / D] = l == 0.0f ? -INFINITY : (m * sl2 + log2f(l)) / kLog2e;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        const int role = warp - 8;
        if (role == (FP8 ? 5 : 0)) {
            // ---- loads: tile 0's keys, its values, tile 1's keys, ... ----
            const int box = d.box, boxes = kTile / box;
            constexpr int bytes = FP8 ? C::kRaw : C::kStage, slots = FP8 ? C::kRaws : kStages;
            uint64_t *fulls = FP8 ? sh.raw_full : sh.full, *empties = FP8 ? sh.raw_empty : sh.empty;
            uint8_t *to = FP8 ? raws : ring;
            int it = 0, page = 0, r = 0;
            bool ok = true;
            for (int i = 0; ok && i < k.nt; ++i) {
                const int key = k.key(i) + lane * box;
                page = a.kv.pages;  // outside: zeros, and no reads
                r = 0;
                if (lane < boxes && k.wanted(key, box)) {
                    const int entry = key / a.kv.page_size;
                    const int p = page_of(a.kv, a.seq, k.b, entry);
                    if (p >= 0) page = p;
                    r = key - entry * a.kv.page_size;
                }
                for (int v = 0; ok && v < 2; ++v, ++it) {
                    const int s = it % slots;
                    ok = __all_sync(kFullMask, it < slots || mbar_wait_fast(&empties[s], (it / slots - 1) & 1, fail));
                    if (!ok) {
                        sh.fail = 1;
                        break;
                    }
                    if (elect_one()) expect_bytes(&fulls[s], bytes);
                    __syncwarp();
                    for (int x = 0; x < boxes; ++x) {
                        const int px = __shfl_sync(kFullMask, page, x), rx = __shfl_sync(kFullMask, r, x);
                        if (elect_one()) {
                            uint8_t *dst = to + s * bytes;
                            const CUtensorMap *map = v ? &vmap : &kmap;
                            if constexpr (FP8) {
                                tma_load_4d(dst + x * box * D, map, 0, k.h, rx, px, &fulls[s]);
                            } else {
#pragma unroll
                                for (int n = 0; n < C::kPanels; ++n)
                                    tma_load_4d(dst + n * C::kPanel + x * box * 128, map, 128 * n, k.h, rx, px, &fulls[s]);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (lane == 0) sh.issued = it;
        } else if (warp == kMmaWarp) {
            // ---- products ----
            constexpr uint32_t qk = bf16_instr(kTile, false), pv = bf16_instr(D, true);
            int edges = 0;
            bool ok = k.nt == 0 || mbar_wait_fast(&sh.q_full, 0, fail);
            auto full = [&](int it) { return mbar_wait_fast(&sh.full[it % kStages], (it / kStages) & 1, fail); };
            auto logits = [&](int t, int it) {
                const uint64_t da = tile_desc(smem_addr(smem + t * C::kStage));
                const uint64_t db = tile_desc(smem_addr(ring + (it % kStages) * C::kStage));
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t at = (x / 4) * (C::kPanel / 16) + 2 * (x % 4);
                    mma_bf16(tmem + t * kTile, da + at, db + at, qk, x > 0);
                }
                mma_commit(&sh.s_full[t]);
            };
            ok = __all_sync(kFullMask, ok && (k.nt == 0 || full(0)));
            if (ok && k.nt > 0) {
                tc_fence_after();
                if (elect_one()) {
                    for (int t = 0; t < tiles; ++t) logits(t, 0);
                    mma_commit(&sh.empty[0]);
                }
                __syncwarp();
            }
            for (int i = 0; ok && i < k.nt; ++i) {
                const int kt = 2 * i + 2, vt = 2 * i + 1;
                const bool more = i + 1 < k.nt;
                const bool check = !FP8 && k.edge(k.key(i));
                ok = __all_sync(kFullMask, full(vt));
                if (check && ok && elect_one()) mbar_arrive(&sh.v_check);
                __syncwarp();
                const uint64_t db = value_desc(smem_addr(ring + (vt % kStages) * C::kStage));
                for (int t = 0; t < tiles; ++t) {
                    ok = ok && mbar_wait_fast(&sh.p_ready[t], i & 1, fail);
                    if (t == 0 && check) ok = ok && mbar_wait_fast(&sh.v_ok, edges++ & 1, fail);
                    if (t == 0 && more) ok = ok && full(kt);
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < kTile / 16; ++x)
                            mma_bf16_tmem(tmem + 2 * kTile + t * D, tmem + t * kTile + 8 * x, db + x * (2048 / 16), pv, i > 0 || x > 0);
                        if (more)
                            logits(t, kt);
                        else
                            mma_commit(&sh.o_full[t]);
                        if (t == tiles - 1) {
                            mma_commit(&sh.empty[vt % kStages]);
                            if (more) mma_commit(&sh.empty[kt % kStages]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok) sh.fail = 1;
            // tensor memory and the barriers outlive the last product
            if (elect_one()) mma_commit(&sh.drain);
            __syncwarp();
            if (!mbar_wait(&sh.drain, 0, nullptr)) sh.fail = 1;
        } else if (!FP8 && role >= 2) {
            // ---- values that are not finite, in tiles that not all rows see ----
            bool ok = true;
            int edges = 0;
            for (int i = 0; ok && i < k.nt; ++i) {
                const int key = k.key(i), vt = 2 * i + 1;
                if (!k.edge(key)) continue;
                ok = mbar_wait_fast(&sh.v_check, edges++ & 1, fail) &&
                     mbar_wait_fast(&sh.full[vt % kStages], (vt / kStages) & 1, fail);
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                const uint32_t st = smem_addr(ring + (vt % kStages) * C::kStage);
#pragma unroll 4
                for (int x = (role - 2) * 32 + lane; x < C::kStage / 16; x += 64) {
                    uint4 w = lds16(st + 16 * x);
                    if (not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w)) {
                        const int j = key + (x * 16 % C::kPanel) / 128;
                        if (k.wanted(j, 1)) sh.fix = 1;
                        sts16(st + 16 * x, make_uint4(finite_part(w.x), finite_part(w.y), finite_part(w.z), finite_part(w.w)));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_ok);
            }
            if (!ok) sh.fail = 1;
        } else if (FP8 && role < 4) {
            // ---- E4M3 rows to bf16, a thread a row ----
            const int r = role * 32 + lane;
            bool ok = true;
            // scale bytes of the row's key and value; 0 where there are none
            auto scales = [&](int i, uint32_t &sk, uint32_t &sv) {
                sk = sv = 0;
                const int j = k.key(i) + r;
                if (i < k.nt && k.wanted(j, 1)) {
                    const int entry = j / a.kv.page_size;
                    const int page = page_of(a.kv, a.seq, k.b, entry);
                    if (page >= 0) {
                        const int64_t at = ((int64_t)page * a.kv.Hkv + k.h) * a.kv.page_size + (j - entry * a.kv.page_size);
                        sk = a.kv.k_scales[at];
                        sv = a.kv.v_scales[at];
                    }
                }
            };
            uint32_t sk, sv;
            scales(0, sk, sv);
            for (int i = 0; ok && i < k.nt; ++i) {
                const int key = k.key(i);
                const bool edge = k.edge(key), wanted = k.wanted(key + r, 1);
                const uint32_t e[2] = {sk, sv};
                scales(i + 1, sk, sv);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int it = 2 * i + v, rs = it % C::kRaws, s = it % kStages;
                    ok = ok && mbar_wait_fast(&sh.raw_full[rs], (it / C::kRaws) & 1, fail) &&
                         (it < kStages || mbar_wait_fast(&sh.empty[s], (it / kStages - 1) & 1, fail));
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    const float f = scale_value(e[v]);
                    const uint32_t src = smem_addr(raws + rs * C::kRaw), dst = smem_addr(ring + s * C::kStage);
                    uint32_t bad = 0;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t at = src + r * D + 16 * c;
                        at ^= (at >> 3) & (D == 128 ? 0x70 : 0x30);  // the TMA's swizzle, by the address
                        const uint4 x = lds16(at);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        uint32_t y[8];
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            uint32_t hp;
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hp) : "h"((uint16_t)(n & 1 ? w[n / 2] >> 16 : w[n / 2])));
                            const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&hp));
                            y[n] = wanted ? pack_bf16(g.x * f, g.y * f) : 0u;
                            if (v && edge) {
                                bad |= not_finite(y[n]);
                                y[n] = finite_part(y[n]);
                            }
                        }
                        const uint32_t to = dst + (c >> 2) * C::kPanel + r * 128;
                        sts16(to + 16 * ((2 * c & 7) ^ (r & 7)), make_uint4(y[0], y[1], y[2], y[3]));
                        sts16(to + 16 * ((2 * c + 1 & 7) ^ (r & 7)), make_uint4(y[4], y[5], y[6], y[7]));
                    }
                    if (bad) sh.fix = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.full[s]);
                        mbar_arrive(&sh.raw_empty[rs]);
                    }
                }
            }
            if (!ok) sh.fail = 1;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sh.fail) {
        if (threadIdx.x == 0) raise_status(a.seq.status, EP_ERR_TIMEOUT);
        // let the loads in flight land before the shared memory goes
        constexpr int slots = FP8 ? C::kRaws : kStages;
        if ((int)threadIdx.x < slots) {
            const int last = sh.issued - 1 - (int)threadIdx.x;
            if (last >= 0) mbar_wait(FP8 ? &sh.raw_full[last % slots] : &sh.full[last % slots], (last / slots) & 1, nullptr);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free<512>(tmem);
    }
}

template <int D, bool FP8>
cudaError_t launch(const PrefillArgs &d, cudaStream_t stream) {
    const KvArgs &kv = d.a.kv;
    CUtensorMap kmap, vmap;
    const int row = FP8 ? D : 2 * D;
    const int64_t dims[4] = {row, kv.Hkv, kv.page_size, kv.pages};
    const int64_t strides[3] = {kv.head_stride, kv.row_stride, kv.page_stride};
    const int box[4] = {row < 128 ? row : 128, 1, d.box, 1};
    const auto swizzle = row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!encode_bytes(&kmap, kv.k, 4, dims, strides, box, swizzle) ||
        !encode_bytes(&vmap, kv.v, 4, dims, strides, box, swizzle))
        return cudaErrorInvalidValue;
    // at most this many blocks of 256 rows, a sequence's last one not being full
    const int64_t T = d.a.seq.T, blocks = (T * d.G) / (2 * kTile) + (T < d.a.seq.B ? T : d.a.seq.B);
    return launch_large<prefill_kernel<D, FP8>>((int)(blocks * kv.Hkv), Cfg<D, FP8>::kThreads,
                                                Cfg<D, FP8>::kSmem, stream, kmap, vmap, d);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs &a, cudaStream_t stream) {
    PrefillArgs d = {};
    d.a = a;
    d.G = a.Hq / a.kv.Hkv;
    d.box = a.kv.page_size & -a.kv.page_size;  // a box lies within a page
    if (d.box > kTile) d.box = kTile;
    const bool fp8 = a.kv.k_scales != nullptr;
    if (a.kv.D == 64) return fp8 ? launch<64, true>(d, stream) : launch<64, false>(d, stream);
    return fp8 ? launch<128, true>(d, stream) : launch<128, false>(d, stream);
}

}  // namespace ep
