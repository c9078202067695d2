// ep_attn_prefill: causal attention of prompts and of their chunks over the paged cache.
//
//   S = Q K^T,  P = exp(scale S - m),  O = sum P V,  l = sum P,  out = O / l
//
// with the running maximum m of a row.  A block has up to 256 rows, the tokens of one sequence
// times the query heads that share a key head, and goes once over the 128-key tiles that its
// rows see.  Roles:
//   - a loader keeps a ring of key and value tiles in flight by tiled TMA loads, page by
//     page;
//   - one thread for each of two row tiles of 128 issues the products on tcgen05: S of a tile
//     into tensor memory, and P V with P read from tensor memory, where it takes the place of
//     S.  One tile's exponentials run under the other's products; a block of at most
//     128 rows has the even key tiles in one and the odd ones in the other.  (With one thread
//     for both, its waits for one tile left the other's products undone: 3700 clocks for two
//     row tiles and 128 keys, where the products take 2270.);
//   - two warpgroups, a thread a row, take S out of tensor memory, and put P back as bf16, in
//     two halves, so that the first one's products run under the second's exponentials.
//     m is let lag behind the true maximum by up to 2^8 (P and l stay far inside fp32, and
//     P's relative rounding is the same), so that O is rescaled only in the rare tiles where
//     a row's maximum jumps;
//   - 8-bit caches: two warpgroups turn the E4M3 tiles into bf16, a thread half a row, which is
//     exact (a power of two times three bits).  bf16 caches: a warp looks for values that are not
//     finite in tiles that not all rows see: 0 * NaN would reach the other rows.
// Few blocks are multiplied by sharing their key tiles out among several, whose sums a second
// kernel adds.
#include "attn.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTile = 128;   // rows of a tile, keys of a tile
constexpr int kRows = 2 * kTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 8.0f;  // log2 of how far m may be behind

struct Shared {
    uint64_t full[5], empty[5], raw_full[5], raw_empty[5];
    uint64_t q_full[2], s_full[2], p_ready[2][2], o_full[2], turn[2], v_ok[4], drain;
    int64_t sums[20];
    uint32_t tmem;
    int fail, fix, issued;
    int b, block;
};

template <int D, bool FP8>
struct Cfg {
    static constexpr int kThreads = FP8 ? 640 : 384;
    // registers a thread: 96 or 168 at launch
    static constexpr int kSoftRegs = FP8 ? 168 : 208, kOtherRegs = FP8 ? 48 : 88;
    static constexpr int kPanels = D / 64;               // 128-byte columns of a tile
    static constexpr int kPanel = kTile * 128;
    static constexpr int kStage = kPanels * kPanel;      // a bf16 tile
    static constexpr int kStages = FP8 && D == 128 ? 3 : 5;
    // 8-bit tiles: memory answers after about 1.5 us, in which four are wanted
    static constexpr int kRaw = FP8 ? kTile * D : 0, kRaws = D == 128 ? 4 : 5;
    static constexpr int kSmem = (2 + kStages) * kStage + kRaws * kRaw + (int)sizeof(Shared);
};

struct PrefillArgs {
    AttnArgs a;
    int G, box;  // query heads a key head; cache rows of a TMA box
    int shares;  // blocks that may share one's key tiles
    float *ws;   // [block][share][row]: m (log2), l; then [block][share][row][D]
    int64_t blocks;
};
__host__ __device__ constexpr size_t ws_floats(int64_t blocks, int shares, int D) {
    return (size_t)blocks * shares * kRows * (D + 2);
}

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
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
// Bits 0 .. n-1, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
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
__device__ __forceinline__ uint32_t finite_part(uint32_t w) { return w & ~((not_finite(w) >> 15) * 0xffffu); }

// What a block works on, the same for all its threads.
struct Block {
    int b, h;            // sequence, key head
    int row0, rows;      // first row (token * G + head) in the sequence, rows of the block
    int first, pos0;     // token of q that is the sequence's first, its position
    int minpos, maxpos;  // of the block's rows
    int lo, S;           // keys [lo, maxpos] and [0, S), S <= lo, are seen by some row
    int tile0, ns;       // tiles 0 .. ns-1, then from tile0 on
    int nt, i0;          // this share's tiles, of which the first
    int shares;          // blocks that share the rows
    int window, sinks;
    __device__ __forceinline__ int key(int i) const {
        i += i0;
        return (i < ns ? i : tile0 + i - ns) * kTile;
    }
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

// Block `index` of a key head: blocks of 256 rows, a sequence's last ones (with the most keys)
// first.  False if there are not so many.  All threads of the block call it.
template <int NT>
__device__ __forceinline__ bool find_block(const PrefillArgs &d, int64_t index, int h, int share, Shared &sh, Block &k) {
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.seq.B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        int64_t n = 0;
        if (b < a.seq.B) n = ((int64_t)seq_span(a.seq, a.kv.page_size, b).n * d.G + kRows - 1) / kRows;
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
        for (int i = 0; i < NT / 32; ++i) {
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
    if (before <= index) return false;
    k.b = sh.b;
    k.h = h;
    const Span sp = seq_span(a.seq, a.kv.page_size, k.b);
    k.first = sp.first;
    k.pos0 = sp.len - sp.n;
    k.row0 = sh.block * kRows;
    k.rows = min(sp.n * d.G - k.row0, kRows);
    k.minpos = k.pos0 + k.row0 / d.G;
    k.maxpos = k.pos0 + (k.row0 + k.rows - 1) / d.G;
    k.window = a.window;
    k.sinks = k.S = a.sinks;
    k.lo = a.window && k.minpos >= a.window ? k.minpos - a.window + 1 : 0;
    if (k.S >= k.lo) k.lo = k.S = 0;
    k.tile0 = k.lo / kTile;
    k.ns = min((k.S + kTile - 1) / kTile, k.tile0);
    const int nt = k.maxpos < 0 ? 0 : k.ns + k.maxpos / kTile + 1 - k.tile0;
    // two tiles a share at least
    k.shares = min(d.shares, max(nt / 2, 1));
    k.i0 = (int)((int64_t)nt * share / k.shares);
    k.nt = (int)((int64_t)nt * (share + 1) / k.shares) - k.i0;
    return share < k.shares;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ PrefillArgs d) {
    using C = Cfg<D, FP8>;
    constexpr int kStages = C::kStages;
    // all of the block's shared memory: queries, the ring (the swizzle wants 1024-byte
    // alignment; static arrays would push it off), 8-bit tiles
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem + 2 * C::kStage, *raws = ring + kStages * C::kStage;
    Shared &sh = *reinterpret_cast<Shared *>(raws + C::kRaws * C::kRaw);
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const volatile int *fail = &sh.fail;
    constexpr int kMmaWarp = FP8 ? 12 : 9;  // and the next one

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], FP8 ? 8 : 1);
            mbar_init(&sh.empty[i], FP8 ? 2 : 3);
        }
        for (int i = 0; i < C::kRaws; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i][0], 4);
            mbar_init(&sh.p_ready[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.turn[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sh.v_ok[i], 1);
        mbar_init(&sh.drain, 2);
        sh.fail = sh.fix = sh.issued = 0;
        mbar_init_fence();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    Block k;
    const int share = blockIdx.x % d.shares;
    const int64_t block = blockIdx.x / d.shares;
    if (!find_block<C::kThreads>(d, block / a.kv.Hkv, (int)(block % a.kv.Hkv), share, sh, k)) return;
    // one row tile: its even key tiles here, its odd ones there
    const bool halves = k.rows <= kTile;
    const int stride = halves ? 2 : 1;
    if (warp == kMmaWarp) tmem_alloc<512>(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;  // S (and P) of both tiles, then O of both

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        // ---- a thread's row ----
        const int t = warp >> 2, local = (halves ? 0 : t * kTile) + (warp & 3) * 32 + lane;
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
        const float sl2 = a.scale * kLog2e;
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
            if (lane == 0) mbar_arrive(&sh.q_full[t]);
        }
        float m = -INFINITY, l = 0.0f;  // m in S's units
        bool ok = true;
        int wmin = valid ? pos : 0x7fffffff, wmax = pos;  // of the warp's rows
#pragma unroll
        for (int x = 16; x; x >>= 1) {
            wmin = min(wmin, __shfl_xor_sync(kFullMask, wmin, x));
            wmax = max(wmax, __shfl_xor_sync(kFullMask, wmax, x));
        }
        const int i_first = halves ? t : 0;
        int n = 0;
        for (int i = i_first; i < k.nt; i += stride, ++n) {
            const int key = k.key(i);
            ok = __all_sync(kFullMask, mbar_wait_fast(&sh.s_full[t], n & 1, fail));
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
                for (int x = 0; x < 4; ++x) {
                    const uint32_t seen = low_bits(hi + 1 - 32 * x) & (~low_bits(lo - 32 * x) | low_bits(s - 32 * x));
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[x][j] = seen >> j & 1 ? v[x][j] : 0xff800000u;  // -infinity
                }
            }
            float top = m;
            {
                float part[4] = {m, m, m, m};
#pragma unroll
                for (int j = 0; j < 32; j += 2)
#pragma unroll
                    for (int x = 0; x < 4; ++x) part[x] = max3(part[x], __uint_as_float(v[x][j]), __uint_as_float(v[x][j + 1]));
                top = fmaxf(max3(part[0], part[1], part[2]), part[3]);
            }
            const bool grown = top > m && !((top - m) * sl2 <= kLag);
            if (__any_sync(kFullMask, grown)) {
                const float next = grown ? top : m;
                const float f = grown ? exp2_fast((m - next) * sl2) : 1.0f;
                l *= f;
                m = next;
                if (n > 0) {
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
                    const uint64_t y = fma2(pair(__uint_as_float(v[x][2 * j]), __uint_as_float(v[x][2 * j + 1])), sl, bb);
                    float e0, e1;
                    unpair(y, e0, e1);
                    e0 = exp2_fast(e0);
                    e1 = exp2_fast(e1);
                    p[j] = pack_bf16(e0, e1);
                    if (j & 1)
                        acc1 = add2(acc1, pair(e0, e1));
                    else
                        acc0 = add2(acc0, pair(e0, e1));
                }
                tmem_st(s_at + 16 * x, p);
                if (x & 1) {  // half of the keys
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_ready[t][x >> 1]);
                }
            }
            acc0 = add2(acc0, acc1);
            float l0, l1;
            unpair(acc0, l0, l1);
            l = l0 + l1;
        }
        if (ok && n > 0) ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_full[t], 0, fail));
        float m2 = m == -INFINITY ? m : m * sl2;  // in log2 units
        float f0 = 1.0f, f1 = 0.0f;  // of this warpgroup's sums, of the other's
        const uint32_t other = smem_addr(ring);  // [128][D] fp32, then [128] m2, l
        if (halves) {
            // the products of both are done, and nothing loads: the ring is free
            if (ok && k.nt > 1) ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_full[t ^ 1], 0, fail));
            if (!ok) sh.fail = 1;
            if (t == 1) {
                if (ok && n > 0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < D / 32; ++x) {
                        uint32_t o[32];
                        tmem_ld(o_at + 32 * x, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sts16(other + (wrow + lane) * D * 4 + 16 * ((8 * x + j) ^ (lane & 7)),
                                  make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                    }
                    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(other + kTile * D * 4 + (wrow + lane) * 8), "f"(m2), "f"(l) : "memory");
                }
                __syncwarp();
                asm volatile("bar.sync 1, 256;" ::: "memory");
            } else {
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (ok && k.nt > 1) {
                    float om, ol;
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(om), "=f"(ol) : "r"(other + kTile * D * 4 + (wrow + lane) * 8) : "memory");
                    const float both = fmaxf(m2, om), ref = both == -INFINITY ? 0.0f : both;
                    f0 = exp2_fast(m2 - ref);
                    f1 = exp2_fast(om - ref);
                    l = l * f0 + ol * f1;
                    m2 = both;
                }
            }
        }
        if (!ok) sh.fail = 1;
        if (ok && !(halves && t == 1)) {
            tc_fence_after();
            const bool fix = sh.fix != 0 && k.nt > 0, direct = k.shares == 1;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int64_t o_here = o_off;
            const int64_t part = (int64_t)blockIdx.x * kRows + local;  // of the workspace
            float *sums = d.ws + d.blocks * d.shares * kRows * 2 + part * D;
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld(o_at + 32 * x, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;
                }
                if (halves && k.nt > 1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 w = lds16(other + (wrow + lane) * D * 4 + 16 * ((8 * x + j) ^ (lane & 7)));
                        o[4 * j] = __float_as_uint(__uint_as_float(o[4 * j]) * f0 + __uint_as_float(w.x) * f1);
                        o[4 * j + 1] = __float_as_uint(__uint_as_float(o[4 * j + 1]) * f0 + __uint_as_float(w.y) * f1);
                        o[4 * j + 2] = __float_as_uint(__uint_as_float(o[4 * j + 2]) * f0 + __uint_as_float(w.z) * f1);
                        o[4 * j + 3] = __float_as_uint(__uint_as_float(o[4 * j + 3]) * f0 + __uint_as_float(w.w) * f1);
                    }
                }
                if (l == 0.0f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;  // sees no key
                }
                if (fix) {
                    // values that the products were spared, added where a row sees them (an
                    // infinity or NaN, so any probability will do)
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
                            for (int w = 0; w < 16; ++w) {
                                uint32_t y;
                                if constexpr (FP8) {
                                    const uint32_t e = reinterpret_cast<const uint16_t *>(src)[16 * x + w];
                                    y = (none || (e & 0x7f) == 0x7f ? 0x7fffu : 0u) |
                                        (none || (e & 0x7f00) == 0x7f00 ? 0x7fff0000u : 0u);
                                } else {
                                    y = reinterpret_cast<const uint32_t *>(src)[16 * x + w];
                                    y &= (not_finite(y) >> 15) * 0xffffu;
                                }
                                if (y) {
                                    o[2 * w] = __float_as_uint(__uint_as_float(o[2 * w]) + bf16_lo(y));
                                    o[2 * w + 1] = __float_as_uint(__uint_as_float(o[2 * w + 1]) + bf16_hi(y));
                                }
                            }
                        }
                    }
                }
                if (!direct) {
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_v4(sums + 32 * x + 4 * j, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                    }
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ch = 4 * x + j;
                    sts16(mine + (ch >> 3) * C::kPanel + (wrow + lane) * 128 + 16 * ((ch & 7) ^ (lane & 7)),
                          make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                }
            }
            __syncwarp();
            if (direct) {
#pragma unroll
                for (int i = 0; i < 32 / RP; ++i) {
                    const int64_t off = __shfl_sync(kFullMask, o_here, i * RP + lane / CH);
                    const int r = wrow + i * RP + lane / CH, ch = lane % CH;
                    if (off >= 0)
                        st_v4(a.out + off + 8 * ch, lds16(mine + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7))));
                }
                if (a.lse && valid) a.lse[o_off / D] = l == 0.0f ? -INFINITY : (m2 + log2f(l)) / kLog2e;
            } else if (valid) {
                *reinterpret_cast<float2 *>(d.ws + 2 * part) = make_float2(m2, l);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        const int role = warp - 8;
        if (role == (FP8 ? 6 : 0)) {
            // ---- loads: tile 0's keys, its values, tile 1's keys, ...; a lane a box ----
            const int box = d.box, boxes = kTile / box;
            constexpr int bytes = FP8 ? C::kRaw : C::kStage, slots = FP8 ? C::kRaws : kStages;
            uint64_t *fulls = FP8 ? sh.raw_full : sh.full, *empties = FP8 ? sh.raw_empty : sh.empty;
            uint8_t *to = (FP8 ? raws : ring) + lane * box * (FP8 ? D : 128);
            int it = 0;
            bool ok = true;
            for (int i = 0; ok && i < k.nt; ++i) {
                const int key = k.key(i) + lane * box;
                int page = a.kv.pages, r = 0;  // outside: zeros, and no reads
                if (lane < boxes && k.wanted(key, box)) {
                    const int entry = key / a.kv.page_size;
                    const int p = page_of(a.kv, a.seq, k.b, entry);
                    if (p >= 0) page = p;
                    r = key - entry * a.kv.page_size;
                }
                for (int v = 0; v < 2; ++v, ++it) {
                    const int s = it % slots;
                    ok = __all_sync(kFullMask, it < slots || mbar_wait_fast(&empties[s], (it / slots - 1) & 1, fail));
                    if (!ok) {
                        sh.fail = 1;
                        break;
                    }
                    if (elect_one()) expect_bytes(&fulls[s], bytes);
                    __syncwarp();
                    if (lane < boxes) {
                        const CUtensorMap *map = v ? &vmap : &kmap;
#pragma unroll
                        for (int n = 0; n < (FP8 ? 1 : C::kPanels); ++n)
                            tma_load_4d(to + s * bytes + n * C::kPanel, map, 128 * n, k.h, r, page, &fulls[s]);
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) sh.issued = it;
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---- products of row tile t ----
            constexpr uint32_t qk = bf16_instr(kTile, false), pv = bf16_instr(D, true);
            const int t = warp - kMmaWarp;
            const uint64_t da = tile_desc(smem_addr(smem + t * C::kStage));
            const uint32_t s_at = tmem + t * kTile, o_at = tmem + 2 * kTile + t * D;
            auto full = [&](int it) { return mbar_wait_fast(&sh.full[it % kStages], (it / kStages) & 1, fail); };
            auto logits = [&](int it) {
                const uint64_t db = tile_desc(smem_addr(ring + (it % kStages) * C::kStage));
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t at = (x / 4) * (C::kPanel / 16) + 2 * (x % 4);
                    mma_bf16(s_at, da + at, db + at, qk, x > 0);
                }
                mma_commit(&sh.s_full[t]);
            };
            // a tile is free when both rows' products have read it
            auto release = [&](int it) {
                mma_commit(&sh.empty[it % kStages]);
                if (halves) mma_commit(&sh.empty[it % kStages]);
            };
            int i = halves ? t : 0, n = 0;
            bool ok = true;
            if (i < k.nt) {
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.q_full[t], 0, fail) && full(2 * i));
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) {
                        logits(2 * i);
                        release(2 * i);
                    }
                    __syncwarp();
                }
            }
            for (; ok && i < k.nt; i += stride, ++n) {
                const int kt = 2 * (i + stride), vt = 2 * i + 1;
                const bool more = i + stride < k.nt;
                ok = full(vt) && (FP8 || !k.edge(k.key(i)) || mbar_wait_fast(&sh.v_ok[i & 3], (i >> 2) & 1, fail));
                const uint64_t db = value_desc(smem_addr(ring + (vt % kStages) * C::kStage));
                ok = __all_sync(kFullMask, ok && mbar_wait_fast(&sh.p_ready[t][0], n & 1, fail));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) mma_bf16_tmem(o_at, s_at + 8 * x, db + x * (2048 / 16), pv, n > 0 || x > 0);
                }
                __syncwarp();
                // The tiles take turns, so that one's exponentials run under the other's products:
                // left alone they fall into step, and each waits for the other in both.
                ok = mbar_wait_fast(&sh.p_ready[t][1], n & 1, fail);
                ok = __all_sync(kFullMask, ok && (t + n == 0 || mbar_wait_fast(&sh.turn[t], (n + t - 1) & 1, fail)));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int x = 4; x < 8; ++x) mma_bf16_tmem(o_at, s_at + 8 * x, db + x * (2048 / 16), pv, true);
                    release(vt);
                    if (!more) {
                        mma_commit(&sh.o_full[t]);
                        mbar_arrive(&sh.turn[t ^ 1]);
                    }
                }
                __syncwarp();
                if (!more) break;
                // only now: these keys may be waiting for the values' place
                ok = __all_sync(kFullMask, full(kt));
                if (!ok) break;
                if (elect_one()) {
                    logits(kt);
                    mbar_arrive(&sh.turn[t ^ 1]);
                    release(kt);
                }
                __syncwarp();
            }
            if (!ok) sh.fail = 1;
            // tensor memory and the barriers outlive the last product
            if (elect_one()) mma_commit(&sh.drain);
            __syncwarp();
            if (!mbar_wait(&sh.drain, 0, nullptr)) sh.fail = 1;
        } else if (!FP8 && role == 3) {
            // ---- values that are not finite, in tiles that not all rows see.  It passes every
            // tile, so that the barriers' phases are never two ahead of it. ----
            bool ok = true;
            for (int it = 0; ok && it < 2 * k.nt; ++it) {
                const int s = it % kStages, i = it >> 1, key = k.key(i);
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.full[s], (it / kStages) & 1, fail));
                if (!ok) break;
                if ((it & 1) && k.edge(key)) {
                    const uint32_t st = smem_addr(ring + s * C::kStage);
#pragma unroll 8
                    for (int x = lane; x < C::kStage / 16; x += 32) {
                        uint4 w = lds16(st + 16 * x);
                        if (not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w)) {
                            const int j = key + (x * 16 % C::kPanel) / 128;
                            if (k.wanted(j, 1)) sh.fix = 1;
                            sts16(st + 16 * x, make_uint4(finite_part(w.x), finite_part(w.y), finite_part(w.z), finite_part(w.w)));
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (it & 1) mbar_arrive(&sh.v_ok[i & 3]);
                    mbar_arrive(&sh.empty[s]);
                }
            }
            if (!ok) sh.fail = 1;
        } else if (FP8 && (role < 4 || role >= 8)) {
            // ---- E4M3 rows to bf16, a thread half a row ----
            const int r = (role & 3) * 32 + lane, c0 = role < 4 ? 0 : D / 32;
            bool ok = true;
            // scale bytes of the row's key and value; 2^0 where there are none
            auto bytes = [&](int i, uint32_t &sk, uint32_t &sv) {
                sk = sv = 127;
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
            bytes(0, sk, sv);
            for (int i = 0; ok && i < k.nt; ++i) {
                const int key = k.key(i);
                const bool edge = k.edge(key), wanted = k.wanted(key + r, 1);
                const float f[2] = {scale_value(sk), scale_value(sv)};
                bytes(i + 1, sk, sv);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int it = 2 * i + v, rs = it % C::kRaws, s = it % kStages;
                    ok = ok && mbar_wait_fast(&sh.raw_full[rs], (it / C::kRaws) & 1, fail) &&
                         (it < kStages || mbar_wait_fast(&sh.empty[s], (it / kStages - 1) & 1, fail));
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    const uint32_t src = smem_addr(raws + rs * C::kRaw) + r * D, dst = smem_addr(ring + s * C::kStage) + r * 128;
                    uint32_t bad = 0;
                    uint4 x[D / 32];  // all of it first: it takes its time
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t at = src + 16 * (c0 + c);
                        at ^= (at >> 3) & (D == 128 ? 0x70 : 0x30);  // the TMA's swizzle, by the address
                        x[c] = lds16(at);
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                        uint32_t y[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t p[2];
                            asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
                                "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
                                : "=r"(p[0]), "=r"(p[1])
                                : "r"(w[j]));
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&p[z]));
                                y[2 * j + z] = pack_bf16(g.x * f[v], g.y * f[v]);
                            }
                        }
                        if (v && edge) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                bad |= not_finite(y[j]);
                                y[j] = finite_part(y[j]);
                            }
                        }
                        const int ch = 2 * (c0 + c);
                        const uint32_t to = dst + (ch >> 3) * C::kPanel;
                        sts16(to + 16 * ((ch & 7) ^ (r & 7)), make_uint4(y[0], y[1], y[2], y[3]));
                        sts16(to + 16 * ((ch + 1 & 7) ^ (r & 7)), make_uint4(y[4], y[5], y[6], y[7]));
                    }
                    if (bad && wanted) sh.fix = 1;
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

// The shares' sums of a block's rows, a warp a row.
template <int D>
__global__ void __launch_bounds__(kRows) join_kernel(const __grid_constant__ PrefillArgs d) {
    constexpr int N = D / 32;
    __shared__ Shared sh;
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t block = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Block k;
    if (!find_block<kRows>(d, block / a.kv.Hkv, (int)(block % a.kv.Hkv), 0, sh, k) || k.shares == 1) return;
    const float *ml = d.ws + block * d.shares * kRows * 2;
    const float *sums = d.ws + d.blocks * d.shares * kRows * 2 + block * d.shares * kRows * D + N * lane;
    for (int r = warp; r < k.rows; r += kRows / 32) {
        float m = -INFINITY, l = 0.0f;
        if (lane < k.shares) {
            m = ld_dep(ml + 2 * (lane * kRows + r));
            l = ld_dep(ml + 2 * (lane * kRows + r) + 1);
        }
        float top = m;
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
        const float f = exp2_fast(m - (top == -INFINITY ? 0.0f : top));
        float sum = l * f, acc[N];
#pragma unroll
        for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(kFullMask, sum, x);
#pragma unroll
        for (int x = 0; x < N; ++x) acc[x] = 0.0f;
#pragma unroll 8
        for (int i = 0; i < k.shares; ++i) {
            const float g = __shfl_sync(kFullMask, f, i);
            const float *src = sums + (int64_t)(i * kRows + r) * D;
#pragma unroll
            for (int x = 0; x < N; ++x) acc[x] += ld_dep(src + x) * g;
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int token = (k.row0 + r) / d.G;
        const int64_t to = (int64_t)(k.first + token) * a.Hq + (int64_t)k.h * d.G + (k.row0 + r - token * d.G);
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + to * D + N * lane);
#pragma unroll
        for (int x = 0; x < N; x += 2) dst[x / 2] = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
        if (a.lse && lane == 0) a.lse[to] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
    }
}

// At most this many blocks of 256 rows, a sequence's last one not being full.
int64_t most_blocks(int64_t T, int64_t B, int G, int Hkv) {
    return ((T * G) / kRows + (T < B ? T : B)) * Hkv;
}
// Blocks that share one's keys: as many as two for each SM allow.
int most_shares(int64_t blocks) {
    const int64_t n = 2 * sm_count() / (blocks > 0 ? blocks : 1);
    return n < 1 ? 1 : n > 32 ? 32 : (int)n;
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
    const cudaError_t err = launch_large<prefill_kernel<D, FP8>>((int)(d.blocks * d.shares), Cfg<D, FP8>::kThreads,
                                                                 Cfg<D, FP8>::kSmem, stream, kmap, vmap, d);
    if (err != cudaSuccess || d.shares == 1) return err;
    return launch_kernel(join_kernel<D>, (int)d.blocks, kRows, 0, stream, true, d);
}

}  // namespace

size_t attn_prefill_workspace(int T, int B, int Hq, int Hkv, int D) {
    const int64_t blocks = most_blocks(T, B, Hq / Hkv, Hkv);
    const int shares = most_shares(blocks);
    return shares == 1 ? 0 : ws_floats(blocks, shares, D) * 4;
}

cudaError_t launch_attn_prefill(const AttnArgs &a, void *workspace, cudaStream_t stream) {
    PrefillArgs d = {};
    d.a = a;
    d.G = a.Hq / a.kv.Hkv;
    d.box = a.kv.page_size & -a.kv.page_size;  // a box lies within a page
    if (d.box > kTile) d.box = kTile;
    d.blocks = most_blocks(a.seq.T, a.seq.B, d.G, a.kv.Hkv);
    d.shares = workspace ? most_shares(d.blocks) : 1;
    d.ws = static_cast<float *>(workspace);
    const bool fp8 = a.kv.k_scales != nullptr;
    if (a.kv.D == 64) return fp8 ? launch<64, true>(d, stream) : launch<64, false>(d, stream);
    return fp8 ? launch<128, true>(d, stream) : launch<128, false>(d, stream);
}

}  // namespace ep
