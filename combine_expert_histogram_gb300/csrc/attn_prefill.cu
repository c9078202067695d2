// ep_attn_prefill: causal attention of prompts and of their chunks over the paged cache.
//
//   S = Q K^T,  P = exp(scale S - m),  O = sum P V,  l = sum P,  out = O / l
//
// with the running maximum m of a row.  A block has up to 256 rows, the tokens of one sequence
// times the query heads that share a key head, and goes once over the 128-key tiles that its
// rows see.  Roles:
//   - a loader (two, where pages are short) keeps a ring of key and value tiles in flight by
//     tiled TMA loads, page by page;
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
//   - 8-bit caches: a warpgroup turns the E4M3 tiles into bf16, a thread a row, which is exact (a
//     power of two times four bits; 2^128 and more, which a scale of 2^120 can make, is an infinity), in
//     loops of few instructions: beside the other roles' code long unrolled ones wait for their
//     instructions (570 us for the prompts that take 460 now).  Two such warpgroups would leave the
//     exponentials too few registers for a row of S (540 us, with S taken twice).  bf16 caches: a warp
//     looks for values that are not finite in tiles that not all rows see: 0 * NaN would reach the
//     other rows.
// The work, a step being one tile of keys (two, for a block of at most 128 rows), is one list
// over sequences, key heads and row blocks, of which every SM takes an equal run, wherever row
// blocks begin and end; a row block that several SMs share leaves its sums in the workspace, and
// a second kernel adds them.  The loader walks the run and tells the other roles its pieces.
//
// Bound by the chain S -> exponentials -> P V of a row tile, which takes 3300 clocks for the 2270
// of both tiles' products (tensor pipe 65 % active): S and P share their tensor memory, which
// O fills otherwise, so that a tile's next S waits for its P V.  A prompt of 8192, 32 heads on 4,
// takes 386 us (1.42 PFLOP/s; in long runs about 405); 5 prompts' chunks of 350 - 700 tokens after 3000 -
// 6000, 64 heads on 8, 370 us in bf16 (1.30 PFLOP/s) and 460 in 8 bits, where the conversion competes for
// issue slots and shared memory.  Heads of 64 wait in the same chain, whose products are half as long: no
// unit is over 40 % busy there (a prompt of 8192: 318 us, exponentials 39 %, tensor pipe 38 %).  Two
// threads a row of S would halve its part of the chain, but their 64 columns and 104 registers spill (452 us then
// for 392).
#include "attn.cuh"
#include "attn_ring.h"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTile = 128;   // rows of a tile, keys of a tile
constexpr int kRows = 2 * kTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 8.0f;  // log2 of how far m may be behind

// Steps of time that a row block costs beside its own, and one of at most 128 rows (a prompt of
// 8192: 448 / 402 / 384 / 378 / 388 us with 2 to 6; few tokens a sequence: 68 / 68 / 72 with 2 to 4).
constexpr int kItem = 5, kItemFew = 3;
constexpr int kLeast = 3;   // steps an SM takes at least (few tokens a sequence: the same with 1 to 6)
constexpr int kPieces = 4;  // pieces ahead

// A piece of the list: some of a row block's tiles.
struct Piece {
    int b, h;            // sequence, key head
    int row0, rows;      // first row (token * G + head) in the sequence, rows of the block
    int first, pos0;     // token of q that is the sequence's first, its position
    int minpos, maxpos;  // of the block's rows
    int lo, S;           // keys [lo, maxpos] and [0, S), S <= lo, are seen by some row
    int tile0, ns;       // tiles 0 .. ns-1, then from tile0 on
    int i0, nt;          // the piece's tiles, the first of them; nt < 0: there is no piece more
    int part;            // where its sums go in the workspace, -1: it is a whole block
    __device__ __forceinline__ int key(int i) const {
        i += i0;
        return (i < ns ? i : tile0 + i - ns) * kTile;
    }
    // Not all rows see all of the tile's keys.
    __device__ __forceinline__ bool edge(int key, int window, int sinks) const {
        return !(key + kTile - 1 <= minpos &&
                 (!window || key > maxpos - window || key + kTile <= sinks));
    }
    // Some row may see one of the keys [key, key + n).
    __device__ __forceinline__ bool wanted(int key, int n) const {
        return key <= maxpos && (key + n > lo || key < S);
    }
    // One row tile: its even key tiles are in one half, its odd ones in the other.
    __device__ __forceinline__ bool halves() const { return rows <= kTile; }
    __device__ __forceinline__ int steps() const { return halves() ? (nt + 1) / 2 : nt; }
    __device__ __forceinline__ int beside() const { return halves() ? kItemFew : kItem; }
    // Of row tile t, or half t.
    __device__ __forceinline__ int tiles(int t) const { return ring_tiles(halves(), t, nt); }
};

struct Shared {
    uint64_t full[5], empty[5], raw_full[5], raw_empty[5];
    uint64_t q_full[2], s_full[2], s_free[2], p_ready[2][2], o_full[2], turn[2], v_ok[4], ml_ready, o_read, drain;
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    int64_t sums[20], found_at;
    float2 ml[kTile];  // of the odd tiles' half
    Piece pieces[kPieces];
    uint32_t tmem;
    int fail, fix, issued[2], found_b;
};

// TWO: a warp loads the keys, another the values.
template <int D, bool FP8, bool TWO>
struct Cfg {
    static constexpr int kThreads = FP8 || TWO ? 512 : 384, kMmaWarp = FP8 || TWO ? 12 : 9;  // and the next warp
    // registers a thread: 128 or 168 at launch
    static constexpr int kSoftRegs = FP8 ? 184 : TWO ? 176 : 200, kOtherRegs = FP8 ? 72 : TWO ? 80 : 104;
    static constexpr int kPanels = D / 64;               // 128-byte columns of a tile
    // Tensor memory (512 columns): S of both tiles, then O.  Heads of 64 leave room for P apart from S, so
    // that the next tile's S is there when its exponentials begin.
    static constexpr bool kApart = D == 64;
    static constexpr int kP = kApart ? 2 * kTile : 0, kPStep = kApart ? kTile / 2 : kTile;
    static constexpr int kO = kApart ? 3 * kTile : 2 * kTile;
    static constexpr int kPanel = kTile * 128;
    static constexpr int kStage = kPanels * kPanel;      // a bf16 tile
    static constexpr int kStages = 5;
    // 8-bit tiles: of heads of 128, where there is no room beside the stages, in their stage's second panel,
    // whose rows are as long as theirs
    static constexpr bool kInside = FP8 && D == 128;
    static constexpr int kRawPitch = kInside ? kStage : kTile * D;
    static constexpr int kRawAt = 2 * kStage + (kInside ? kPanel : kStages * kStage);
    static constexpr int kBarriers = (2 + kStages) * kStage + (FP8 && !kInside ? kStages * kRawPitch : 0);
    static constexpr int kSmem = kBarriers + (int)sizeof(Shared);
};

struct PrefillArgs {
    AttnArgs a;
    int G, box;   // query heads a key head; cache rows of a TMA box
    uint8_t *ws;  // on 32 bytes; nullptr: row blocks stay whole
    bool wide;    // the output is on 32 bytes
};
// The workspace: for each SM the shared row block that begins in its run (sequence, head, block,
// SMs after it); m (log2) and l of its first and last piece's rows; their sums, which are stored 32
// bytes at a time.
__host__ __device__ constexpr size_t ws_ml(int blocks) { return ((size_t)blocks * 16 + 31) / 32 * 32; }
__host__ __device__ constexpr size_t ws_sums(int blocks) { return ws_ml(blocks) + (size_t)blocks * 2 * kRows * 8; }
__host__ __device__ constexpr size_t ws_bytes(int blocks, int D) {
    return ws_sums(blocks) + (size_t)blocks * 2 * kRows * D * 4;
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
// 32 bytes, which p may be a multiple of (wide) or of 16 alone.
__device__ __forceinline__ void st_32(bool wide, void *p, const uint32_t *v) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        st_v4(p, make_uint4(v[0], v[1], v[2], v[3]));
        st_v4(static_cast<uint8_t *>(p) + 16, make_uint4(v[4], v[5], v[6], v[7]));
    }
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
// 2^(e - 127), NaN for 255, twice in bf16.
__device__ __forceinline__ uint32_t scale_bf16(uint32_t e) {
    return (e == 255 ? 0x7fffu : e == 0 ? 0x40u : e << 7) * 0x10001u;
}
__device__ __forceinline__ uint32_t mul_bf16(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
// A pair of E4M3 values as fp16 -> bf16, exactly.
__device__ __forceinline__ uint32_t bf16_pair(uint32_t h) {
    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16(g.x, g.y);
}
// In the upper bit of each half: whether that bf16 is an infinity or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// w with the halves that are not finite as 0.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) { return w & ~((not_finite(w) >> 15) * 0xffffu); }

__device__ __forceinline__ int row_blocks(const PrefillArgs &d, const Span &sp) { return (sp.n * d.G + kRows - 1) / kRows; }

// Row block j of a sequence and any head, whole: those with the last rows come first.
__device__ __forceinline__ Piece row_block(const PrefillArgs &d, const Span &sp, int j) {
    Piece k;
    k.first = sp.first;
    k.pos0 = sp.len - sp.n;
    k.row0 = (row_blocks(d, sp) - 1 - j) * kRows;
    k.rows = min(sp.n * d.G - k.row0, kRows);
    k.minpos = k.pos0 + k.row0 / d.G;
    k.maxpos = k.pos0 + (k.row0 + k.rows - 1) / d.G;
    k.S = d.a.sinks;
    k.lo = d.a.window && k.minpos >= d.a.window ? k.minpos - d.a.window + 1 : 0;
    if (k.S >= k.lo) k.lo = k.S = 0;
    k.tile0 = k.lo / kTile;
    k.ns = min((k.S + kTile - 1) / kTile, k.tile0);
    k.i0 = 0;
    k.nt = k.maxpos < 0 ? 0 : k.ns + k.maxpos / kTile + 1 - k.tile0;
    k.part = -1;
    return k;
}
// Its places in the list.
__device__ __forceinline__ int places(const PrefillArgs &d, const Piece &k) { return d.ws ? k.steps() + k.beside() : 1; }
// The places of all of a sequence's blocks of one head, by one warp.
__device__ __forceinline__ int64_t all_places(const PrefillArgs &d, const Span &sp, int lane) {
    int64_t n = 0;
    for (int j = lane; j < row_blocks(d, sp); j += 32) n += places(d, row_block(d, sp, j));
#pragma unroll
    for (int x = 16; x; x >>= 1) n += __shfl_xor_sync(kFullMask, n, x);
    return n;
}

template <int D, bool FP8, bool TWO>
__global__ void __launch_bounds__(Cfg<D, FP8, TWO>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ PrefillArgs d) {
    using C = Cfg<D, FP8, TWO>;
    constexpr int kStages = C::kStages;
    // all of the block's shared memory: queries, the ring (the swizzle wants 1024-byte
    // alignment; static arrays would push it off), 8-bit tiles
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem + 2 * C::kStage;
    Shared &sh = *reinterpret_cast<Shared *>(smem + C::kBarriers);
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const volatile int *fail = &sh.fail;
    constexpr int kMmaWarp = C::kMmaWarp;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], FP8 ? 4 : 1 + TWO);
            mbar_init(&sh.empty[i], FP8 ? 2 : 3);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
            mbar_init(&sh.p_ready[i][0], 4);
            mbar_init(&sh.p_ready[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.turn[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sh.v_ok[i], 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], FP8 ? 14 : 11 + TWO);  // warps that read it
        }
        mbar_init(&sh.ml_ready, 4);
        mbar_init(&sh.o_read, 4);
        mbar_init(&sh.drain, 2);
        sh.fail = sh.fix = sh.issued[0] = sh.issued[1] = 0;
        mbar_init_fence();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the block's run of the list, and its first sequence ----
    int64_t total = 0, n0 = 0, excl0 = 0;
    auto scan = [&](int b0, int64_t &n, int64_t &excl) {
        const int b = b0 + threadIdx.x;
        Span sp = {0, 0, 0};
        if (b < a.seq.B) sp = seq_span(a.seq, a.kv.page_size, b);
        const int nb = row_blocks(d, sp);
        n = 0;
        if (nb <= 4)
            for (int j = 0; j < nb; ++j) n += places(d, row_block(d, sp, j));
        for (uint32_t many = __ballot_sync(kFullMask, nb > 4); many; many &= many - 1) {
            const int src = __ffs(many) - 1;
            const Span one = {__shfl_sync(kFullMask, sp.first, src), __shfl_sync(kFullMask, sp.n, src),
                              __shfl_sync(kFullMask, sp.len, src)};
            const int64_t m = all_places(d, one, lane);
            if (lane == src) n = m;
        }
        n *= a.kv.Hkv;
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
        excl = incl - n + below;
        return all;
    };
    for (int b0 = 0; b0 < a.seq.B; b0 += C::kThreads) {
        int64_t n, excl;
        total += scan(b0, n, excl);
        if (b0 == 0) n0 = n, excl0 = excl;
    }
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)(d.ws ? kLeast : 1));
    const int64_t x0 = blockIdx.x * per, x1 = min(x0 + per, total);
    if (d.ws && threadIdx.x == 0) reinterpret_cast<int4 *>(d.ws)[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (x0 >= x1) return;
    int64_t before = 0;
    for (int b0 = 0;; b0 += C::kThreads) {
        int64_t n = n0, excl = excl0, all = total;
        if (a.seq.B > C::kThreads) all = scan(b0, n, excl);
        if (x0 >= before + excl && x0 < before + excl + n) {
            sh.found_b = b0 + threadIdx.x;
            sh.found_at = before + excl;
        }
        before += all;
        if (before > x0 || b0 + C::kThreads >= a.seq.B) break;
    }
    if (warp == kMmaWarp) tmem_alloc<512>(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // The next piece of the run, for a warp that goes through them.
    auto next_piece = [&](int p, Piece &k) {
        const bool ok = __all_sync(kFullMask, mbar_wait_fast(&sh.piece_full[p % kPieces], (p / kPieces) & 1, fail));
        if (!ok) {
            sh.fail = 1;
            return false;
        }
        k = sh.pieces[p % kPieces];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[p % kPieces]);
        return k.nt >= 0;
    };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        const int t = warp >> 2, wrow = (warp & 3) * 32;
        const uint32_t lanes = (uint32_t)wrow << 16;
        const uint32_t s_at = tmem + t * kTile + lanes, p_at = tmem + C::kP + t * C::kPStep + lanes;
        const uint32_t o_at = tmem + C::kO + t * D + lanes;
        constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte chunks a row, rows an instruction
        const uint32_t mine = smem_addr(smem) + t * C::kStage;
        const float sl2 = a.scale * kLog2e;
        int done = 0, o_done = 0, merged = 0;  // tiles, pieces with tiles, pieces in halves so far
        // The queries of a piece, asynchronously into their tile; zeros where there is no row.
        auto copy_queries = [&](const Piece &k) {
            const int local = (k.halves() ? 0 : t * kTile) + wrow + lane, row = k.row0 + local, token = row / d.G;
            const int64_t off = local < k.rows ? (k.first + token) * a.q_stride + ((int64_t)k.h * d.G + (row - token * d.G)) * D : -1;
#pragma unroll 4
            for (int i = 0; i < 32 / RP; ++i) {
                const int64_t o = __shfl_sync(kFullMask, off, i * RP + lane / CH);
                const int r = wrow + i * RP + lane / CH, ch = lane % CH;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 mine + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7))),
                             "l"(a.q + (o >= 0 ? o + 8 * ch : 0)), "r"(o >= 0 ? 16 : 0)
                             : "memory");
            }
        };
        auto queries_there = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[t]);
        };
        // Pieces stay in shared memory: registers are short here.
        auto piece = [&](int p) -> const Piece & { return sh.pieces[p % kPieces]; };
        auto piece_there = [&](int p) {
            const bool ok = __all_sync(kFullMask, mbar_wait_fast(&sh.piece_full[p % kPieces], (p / kPieces) & 1, fail));
            if (!ok) sh.fail = 1;
            return ok && piece(p).nt >= 0;
        };
        bool have = piece_there(0);
        if (have && piece(0).tiles(t) > 0) {
            copy_queries(piece(0));
            queries_there();
        }
        for (int p = 1; have; ++p) {
        const Piece &k = piece(p - 1), &next = piece(p);
        // ---- a thread's row ----
        const bool halves = k.halves();
        const int local = (halves ? 0 : t * kTile) + wrow + lane;
        const bool valid = local < k.rows;
        const int row = k.row0 + local, token = row / d.G;
        const int pos = valid ? k.pos0 + token : -1;
        const int mine_of = k.tiles(t);
        float m = -INFINITY, l = 0.0f;  // m in S's units
        bool ok = true;
        int wmin = valid ? pos : 0x7fffffff, wmax = pos;  // of the warp's rows
#pragma unroll
        for (int x = 16; x; x >>= 1) {
            wmin = min(wmin, __shfl_xor_sync(kFullMask, wmin, x));
            wmax = max(wmax, __shfl_xor_sync(kFullMask, wmax, x));
        }
        for (int n = 0; n < mine_of; ++n, ++done) {
            const int key = k.key(halves ? 2 * n + t : n);
            ok = __all_sync(kFullMask, mbar_wait_fast(&sh.s_full[t], done & 1, fail));
            if (!ok) break;
            tc_fence_after();
            uint32_t u[4][32];  // the row's S
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld(s_at + 32 * x, u[x]);
            const bool masked = !(key + kTile - 1 <= wmin && (!a.window || key > wmax - a.window || key + kTile <= a.sinks));
            const int hi = pos - key + 1, lo = a.window && hi > a.window ? hi - a.window : 0, first = a.sinks - key;
            auto s_read = [&]() {  // S is in registers
                if (!C::kApart) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_free[t]);
            };
            auto mask = [&](uint32_t (&v)[32], int at) {
                const uint32_t seen = low_bits(hi - at) & (~low_bits(lo - at) | low_bits(first - at));
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = seen >> j & 1 ? v[j] : 0xff800000u;  // -infinity
            };
            float part[4] = {m, m, m, m};
            auto largest = [&](const uint32_t (&v)[32]) {
#pragma unroll
                for (int j = 0; j < 32; j += 2) part[j / 2 & 3] = max3(part[j / 2 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            };
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld_wait(u[x]);
            s_read();
            if (masked) {
#pragma unroll
                for (int x = 0; x < 4; ++x) mask(u[x], 32 * x);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) largest(u[x]);
            const float top = fmaxf(max3(part[0], part[1], part[2]), part[3]);
            // the products of the tile before read P and write O
            if (C::kApart && n > 0) {
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_full[t], (done - 1) & 1, fail));
                if (!ok) break;
                tc_fence_after();
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
            // sums of the tile's alone (onto l each would be rounded at l's size), which begin as its first
            // pairs: from zeros a prompt of 8192 takes 399 us for 386
            uint64_t acc0, acc1;
            auto exponentials = [&](const uint32_t (&v)[32], uint32_t to, bool begin) {
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint64_t y = fma2(pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sl, bb);
                    float e0, e1;
                    unpair(y, e0, e1);
                    e0 = exp2_fast(e0);
                    e1 = exp2_fast(e1);
                    p[j] = pack_bf16(e0, e1);
                    uint64_t &acc = j & 1 ? acc1 : acc0;
                    acc = begin && j < 2 ? pair(e0, e1) : add2(acc, pair(e0, e1));
                }
                tmem_st(to, p);  // over columns that are in registers by now
            };
            auto half_done = [&](int h) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[t][h]);
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                exponentials(u[2 * h], p_at + 32 * h, h == 0);
                exponentials(u[2 * h + 1], p_at + 32 * h + 16, false);
                half_done(h);
            }
            acc0 = add2(acc0, acc1);
            float l0, l1;
            unpair(acc0, l0, l1);
            l += l0 + l1;
        }
        have = ok && piece_there(p);
        if (ok && mine_of > 0) ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_full[t], (C::kApart ? done - 1 : o_done++) & 1, fail));
        // The next piece's queries come while this one's results go (and not for a half without a
        // tile, which would run ahead of its barriers' readers).
        bool pending = ok && have && next.tiles(t) > 0;
        if (pending) copy_queries(next);
        float m2 = m == -INFINITY ? m : m * sl2;  // in log2 units
        float f0 = 1.0f, f1 = 0.0f;  // of this half's sums, of the other's
        const bool both = halves && k.nt > 1;
        if (both && t == 1) {
            // the even tiles' half takes these sums out of tensor memory with its own
            if (ok) {
                sh.ml[wrow + lane] = make_float2(m2, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.ml_ready);
                if (pending) queries_there();
                pending = false;
                ok = __all_sync(kFullMask, mbar_wait_fast(&sh.o_read, merged++ & 1, fail));
            }
        } else if (both) {
            ok = ok && __all_sync(kFullMask, mbar_wait_fast(&sh.ml_ready, merged++ & 1, fail));
            if (ok) {
                const float2 other = sh.ml[wrow + lane];
                const float top = fmaxf(m2, other.x), ref = top == -INFINITY ? 0.0f : top;
                f0 = exp2_fast(m2 - ref);
                f1 = exp2_fast(other.x - ref);
                l = l * f0 + other.y * f1;
                m2 = top;
            }
        }
        if (!ok) {
            sh.fail = 1;
            break;
        }
        if (!(halves && t == 1)) {
            tc_fence_after();
            const bool direct = k.part < 0;
            const float inv = pos < 0 ? 0.0f : 1.0f / l;  // 0 / 0 where all logits are -infinity
            const int64_t part = (int64_t)k.part * kRows + local;  // of the workspace
            float *sums = reinterpret_cast<float *>(d.ws + ws_sums(gridDim.x)) + part * D;
            const int64_t to = (int64_t)(k.first + token) * a.Hq + (int64_t)k.h * d.G + (row - token * d.G);
            uint16_t *out = a.out + to * D;
            // Straight from the registers: shared memory is busy with the products' operands.
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
                uint32_t o[32];
                if (mine_of > 0) {
                    tmem_ld(o_at + 32 * x, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;
                }
                if (both) {
                    uint32_t w[32];
                    tmem_ld(o_at + D + 32 * x, w);
                    tmem_ld_wait(w);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f0 + __uint_as_float(w[j]) * f1);
                }
                if (direct) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                }
                if (valid) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        if (j < 16 || !direct)
                            st_32(d.wide || !direct, direct ? (void *)(out + 32 * x + 2 * j) : (void *)(sums + 32 * x + j), o + j);
                }
                if (x == 0 && pending) {
                    queries_there();
                    pending = false;
                }
            }
            if (both) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.o_read);
            }
            if (sh.fix && valid) {
                // values that the products were spared, added where a row sees them (an infinity
                // or NaN, so any probability will do)
                for (int i = 0; i < k.nt; ++i) {
                    const int key = k.key(i);
                    if (!k.edge(key, a.window, a.sinks)) continue;
                    for (int j = key; j <= min(pos, key + kTile - 1); ++j) {
                        if (a.window && j <= pos - a.window && j >= a.sinks) continue;
                        const int page = page_of(a.kv, a.seq, k.b, j / a.kv.page_size);
                        if (page < 0) continue;
                        const int r = j % a.kv.page_size;
                        const uint8_t *src = a.kv.v + page * a.kv.page_stride + r * a.kv.row_stride + k.h * a.kv.head_stride;
                        const uint32_t scale =
                            FP8 ? scale_bf16(a.kv.v_scales[((int64_t)page * a.kv.Hkv + k.h) * a.kv.page_size + r]) : 0;
#pragma unroll 1
                        for (int w = 0; w < D / 2; ++w) {
                            uint32_t y;
                            if constexpr (FP8) {
                                uint32_t lo, hi;
                                half_pairs(reinterpret_cast<const uint16_t *>(src)[w], lo, hi);
                                y = mul_bf16(bf16_pair(lo), scale);
                            } else {
                                y = reinterpret_cast<const uint32_t *>(src)[w];
                            }
                            y &= (not_finite(y) >> 15) * 0xffffu;
                            if (!y) continue;
                            if (direct) {
                                uint32_t *at = reinterpret_cast<uint32_t *>(out) + w;
                                *at = pack_bf16(bf16_lo(*at) + bf16_lo(y), bf16_hi(*at) + bf16_hi(y));
                            } else {
                                sums[2 * w] += bf16_lo(y);
                                sums[2 * w + 1] += bf16_hi(y);
                            }
                        }
                    }
                }
            }
            if (valid && direct) {
                if (a.lse) a.lse[to] = l == 0.0f ? -INFINITY : (m2 + log2f(l)) / kLog2e;
            } else if (valid) {
                *reinterpret_cast<float2 *>(d.ws + ws_ml(gridDim.x) + part * 8) = make_float2(m2, l);
            }
        }
        if (pending) queries_there();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[(p - 1) % kPieces]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        const int role = warp - 8;
        // The loads of a piece, the run's tiles n, n + 1, ...: keys, values, keys, ...; with two loaders
        // the `mine` ones (0: keys).  A lane a box, whose entry in the block table is looked up a
        // tile ahead.
        auto load = [&](const Piece &k, int mine, int &n) {
            const int box = d.box, boxes = kTile / box;
            constexpr int bytes = FP8 ? kTile * D : C::kStage, pitch = FP8 ? C::kRawPitch : C::kStage;
            uint64_t *fulls = FP8 ? sh.raw_full : sh.full, *empties = FP8 && !C::kInside ? sh.raw_empty : sh.empty;
            uint8_t *to = (FP8 ? smem + C::kRawAt : ring) + lane * box * (FP8 ? D : 128);
            uint32_t entry = 0;
            int row = 0;
            bool there = false;
            auto look = [&](int i) {
                const int key = k.key(i) + lane * box, e = key / a.kv.page_size;
                there = i < k.nt && lane < boxes && k.wanted(key, box);
                row = key - e * a.kv.page_size;
                entry = ld_dep_if(there, a.seq.table + (int64_t)k.b * a.seq.max_pages + (there ? e : 0));
            };
            look(0);
            for (int i = 0; i < k.nt; ++i) {
                const bool ok = there && entry < (uint32_t)a.kv.pages;
                if (there && !ok) raise_status(a.seq.status, EP_ERR_BAD_PAGE);
                const int page = ok ? entry : a.kv.pages, r = ok ? row : 0;  // outside: zeros, and no reads
                look(i + 1);
                for (int v = 0; v < 2; ++v, ++n) {
                    const int s = n % kStages;
                    const bool empty = n < kStages || mbar_wait_fast(&empties[s], (n / kStages - 1) & 1, fail);
                    if (!__all_sync(kFullMask, empty)) return false;
                    // Both loaders see every phase of every stage, and none goes on without them: a
                    // wait that comes a phase late or early would take one for another.
                    if (TWO && v != mine) {
                        if (lane == 0) mbar_arrive(&fulls[s]);
                        continue;
                    }
                    if (elect_one()) expect_bytes(&fulls[s], bytes);
                    __syncwarp();
                    if (lane < boxes) {
                        const CUtensorMap *map = v ? &vmap : &kmap;
#pragma unroll
                        for (int x = 0; x < (FP8 ? 1 : C::kPanels); ++x)
                            tma_load_4d(to + s * pitch + x * C::kPanel, map, 128 * x, k.h, r, page, &fulls[s]);
                    }
                    __syncwarp();
                }
            }
            return true;
        };
        if (role == (FP8 || TWO ? 6 : 0)) {
            // ---- the run's pieces, and their loads ----
            int b = sh.found_b, h, j = 0, n = 0, p = 0;
            int64_t at = sh.found_at;
            Span sp = seq_span(a.seq, a.kv.page_size, b);
            {
                const int64_t one = all_places(d, sp, lane);  // of a head
                h = (int)((x0 - at) / one);
                at += h * one;
                for (;; j += 32) {  // the block where the run begins
                    int64_t n = j + lane < row_blocks(d, sp) ? places(d, row_block(d, sp, j + lane)) : 0, incl = n;
#pragma unroll
                    for (int s = 1; s < 32; s <<= 1) {
                        const int64_t o = __shfl_up_sync(kFullMask, incl, s);
                        if (lane >= s) incl += o;
                    }
                    const uint32_t past = __ballot_sync(kFullMask, at + incl > x0);
                    if (past || j + 32 >= row_blocks(d, sp)) {
                        const int src = past ? __ffs(past) - 1 : 31;
                        at += __shfl_sync(kFullMask, incl - n, src);
                        j += src;
                        break;
                    }
                    at += __shfl_sync(kFullMask, incl, 31);
                }
            }
            bool ok = true;
            while (ok) {
                Piece k;
                bool some = false;
                while (!some && at < x1) {
                    k = row_block(d, sp, j);
                    k.b = b;
                    k.h = h;
                    const int steps = k.steps();
                    if (d.ws) {
                        // steps [s0, s1) of the block
                        const int s0 = (int)max(x0 - at, (int64_t)0), s1 = (int)min((int64_t)steps, x1 - at);
                        const bool starts = at >= x0, ends = at + steps <= x1;
                        some = steps == 0 ? starts : s0 < s1;
                        if (some && !(starts && ends)) {
                            const int scale = k.halves() ? 2 : 1;
                            k.part = 2 * blockIdx.x + starts;
                            k.i0 = s0 * scale;
                            k.nt = min(s1 * scale, k.nt) - k.i0;
                            if (starts && lane == 0)
                                reinterpret_cast<int4 *>(d.ws)[blockIdx.x] =
                                    make_int4(b, h, j, (int)((at + steps - 1) / per) - (int)blockIdx.x);
                        }
                        at += steps + k.beside();
                    } else {
                        some = true;
                        ++at;
                    }
                    if (++j == row_blocks(d, sp)) {
                        j = 0;
                        if (++h == a.kv.Hkv) {
                            h = 0;
                            do {
                                if (++b < a.seq.B) sp = seq_span(a.seq, a.kv.page_size, b);
                            } while (b < a.seq.B && sp.n == 0);
                            if (b >= a.seq.B) at = x1;  // the list's end
                        }
                    }
                }
                if (!some) k.nt = -1;
                for (int r = lane; some && r < k.rows; r += 32) {  // its queries, into L2
                    const int row = k.row0 + r, token = row / d.G;
                    const uint16_t *src = a.q + (k.first + token) * a.q_stride + ((int64_t)k.h * d.G + (row - token * d.G)) * D;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src) : "memory");
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + D - 1) : "memory");
                }
                ok = __all_sync(kFullMask, p < kPieces || mbar_wait_fast(&sh.piece_empty[p % kPieces], (p / kPieces - 1) & 1, fail));
                if (!ok) break;
                if (lane == 0) {
                    sh.pieces[p % kPieces] = k;
                    mbar_arrive(&sh.piece_full[p % kPieces]);
                }
                __syncwarp();
                ++p;
                if (!some) break;
                ok = load(k, 0, n);
            }
            if (!ok) sh.fail = 1;
            if (lane == 0) sh.issued[0] = n;
            if (!TWO && lane == 0) sh.issued[1] = n;
        } else if (TWO && role == 7) {
            // ---- the loads of values ----
            bool ok = true;
            int n = 0;
            Piece k;
            for (int p = 0; ok && next_piece(p, k); ++p) ok = load(k, 1, n);
            if (!ok) sh.fail = 1;
            if (lane == 0) sh.issued[1] = n;
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---- products of row tile t ----
            constexpr uint32_t qk = bf16_instr(kTile, false), pv = bf16_instr(D, true);
            const int t = warp - kMmaWarp;
            const uint64_t da = tile_desc(smem_addr(smem + t * C::kStage));
            const uint32_t s_at = tmem + t * kTile, p_at = tmem + C::kP + t * C::kPStep, o_at = tmem + C::kO + t * D;
            auto logits = [&](int stage) {
                const uint64_t db = tile_desc(smem_addr(ring + stage * C::kStage));
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t at = (x / 4) * (C::kPanel / 16) + 2 * (x % 4);
                    mma_bf16(s_at, da + at, db + at, qk, x > 0);
                }
                mma_commit(&sh.s_full[t]);
            };
            // The place in the ring of this row tile's next keys and values, and the parity of its phase.
            struct Place {
                int it, s, parity;
                __device__ __forceinline__ void set(int n) {
                    it = n;
                    s = n % kStages;
                    parity = n / kStages & 1;
                }
                __device__ __forceinline__ void add(int n) {  // n < kStages, or twice that
                    it += n;
                    s += n;
                    while (s >= kStages) s -= kStages, parity ^= 1;
                }
            };
            auto full = [&](const Place &at) { return mbar_wait_fast(&sh.full[at.s], at.parity, fail); };
            // The next n places are the other half's.  A wait for a phase is sound only if the phase
            // before it is over.  Where the row tiles take turns, a turn says that the other warp has
            // waited for its places before it, and they are skipped; else this warp waits for them too,
            // in order, and hands them back.  (Doing so everywhere, 8-bit prompts of heads of 128 took
            // 563 us for 460: more code beside the conversion's.)
            constexpr bool walk = C::kApart;
            auto pass = [&](Place &at, int n) {
                for (; n > 0; --n, at.add(1)) {
                    if (!__all_sync(kFullMask, full(at))) return false;
                    if (elect_one()) mbar_arrive(&sh.empty[at.s]);
                    __syncwarp();
                }
                return true;
            };
            int base = 0, done = 0, blocks = 0, queries = 0;  // ring index, tiles, turns, pieces with tiles so far
            bool ok = true;
            Piece k;
            for (int p = 0; ok && next_piece(p, k); ++p, base += 2 * k.nt) {
                if (k.nt == 0) continue;
                const bool halves = k.halves();
                const int mine = k.tiles(t), step = halves ? 4 : 2;
                // a tile is free when both warps' products have read it, or one's have and the other has
                // passed it (with turns: or one's have, which then arrives twice)
                auto release = [&](const Place &at) {
                    mma_commit(&sh.empty[at.s]);
                    if (!walk && halves) mma_commit(&sh.empty[at.s]);
                };
                Place kt, vt;
                kt.set(base + (!walk && halves ? 2 * t : 0));
                ok = mine == 0 || !walk || pass(kt, ring_others_before(halves, t, 0));
                vt = kt;
                vt.add(1);
                ok = ok && (mine == 0 || (mbar_wait_fast(&sh.q_full[t], queries++ & 1, fail) && full(kt)));
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                tc_fence_after();
                if (mine > 0 && elect_one()) {
                    logits(kt.s);
                    release(kt);
                }
                __syncwarp();
                for (int n = 0; n < mine; ++n, ++done, ++blocks) {
                    const bool more = n + 1 < mine;
                    const int key = k.key(halves ? 2 * n + t : n);
                    ok = full(vt) && (FP8 || !k.edge(key, a.window, a.sinks) ||
                                      mbar_wait_fast(&sh.v_ok[(vt.it >> 1) & 3], (vt.it >> 3) & 1, fail));
                    const uint64_t db = value_desc(smem_addr(ring + vt.s * C::kStage));
                    kt.add(walk ? 2 : step);
                    if (C::kApart && more) {
                        ok = __all_sync(kFullMask, ok && mbar_wait_fast(&sh.s_free[t], done & 1, fail)) &&
                             pass(kt, ring_others_before(halves, t, n + 1));
                        ok = __all_sync(kFullMask, ok && full(kt));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            logits(kt.s);
                            release(kt);
                        }
                        __syncwarp();
                    }
                    ok = __all_sync(kFullMask, ok && mbar_wait_fast(&sh.p_ready[t][0], done & 1, fail));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) mma_bf16_tmem(o_at, p_at + 8 * x, db + x * (2048 / 16), pv, n > 0 || x > 0);
                    }
                    __syncwarp();
                    if constexpr (C::kApart) {
                        ok = __all_sync(kFullMask, mbar_wait_fast(&sh.p_ready[t][1], done & 1, fail));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int x = 4; x < 8; ++x) mma_bf16_tmem(o_at, p_at + 8 * x, db + x * (2048 / 16), pv, true);
                            mma_commit(&sh.o_full[t]);
                            release(vt);
                        }
                        __syncwarp();
                        vt.add(step);
                        continue;
                    }
                    // 8-bit keys may come late, converted: these products do not wait for them
                    constexpr bool late = FP8;
                    // The tiles take turns, so that one's exponentials run under the other's products:
                    // left alone they fall into step, and each waits for the other in both.
                    ok = t + blocks == 0 || mbar_wait_fast(&sh.turn[t], (blocks + t - 1) & 1, fail);
                    ok = ok && mbar_wait_fast(&sh.p_ready[t][1], done & 1, fail) && (late || !more || full(kt));
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 4; x < 8; ++x) mma_bf16_tmem(o_at, p_at + 8 * x, db + x * (2048 / 16), pv, true);
                        if (!late && more) logits(kt.s);
                        release(vt);
                        if (!late && more) release(kt);
                        if (!more) mma_commit(&sh.o_full[t]);
                        if (!late || !more) mbar_arrive(&sh.turn[t ^ 1]);
                    }
                    if (late && more) {
                        ok = __all_sync(kFullMask, full(kt));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            logits(kt.s);
                            release(kt);
                            mbar_arrive(&sh.turn[t ^ 1]);
                        }
                    }
                    __syncwarp();
                    vt.add(step);
                }
                if (walk) ok = ok && pass(kt, ring_others_after(halves, t, k.nt));
                if (!C::kApart && ok && mine < k.tiles(0)) {  // an odd number in halves: a turn without a tile
                    ok = __all_sync(kFullMask, mbar_wait_fast(&sh.turn[t], (blocks + t - 1) & 1, fail));
                    ++blocks;
                    if (ok && elect_one()) mbar_arrive(&sh.turn[t ^ 1]);
                    __syncwarp();
                }
            }
            if (!ok) sh.fail = 1;
            // tensor memory and the barriers outlive the last product
            if (elect_one()) mma_commit(&sh.drain);
            __syncwarp();
            if (!mbar_wait(&sh.drain, 0, nullptr)) sh.fail = 1;
        } else if (!FP8 && role == (TWO ? 0 : 3)) {
            // ---- values that are not finite, in tiles that not all rows see.  It passes every
            // tile, so that the barriers' phases are never two ahead of it. ----
            bool ok = true;
            int it = 0;
            Piece k;
            for (int p = 0; ok && next_piece(p, k); ++p) {
                for (int n = 0; ok && n < 2 * k.nt; ++n, ++it) {
                    const int s = it % kStages, key = k.key(n >> 1);
                    ok = __all_sync(kFullMask, mbar_wait_fast(&sh.full[s], (it / kStages) & 1, fail));
                    if (!ok) break;
                    if ((n & 1) && k.edge(key, a.window, a.sinks)) {
                        const uint32_t st = smem_addr(ring + s * C::kStage);
#pragma unroll 2
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
                        if (n & 1) mbar_arrive(&sh.v_ok[(it >> 1) & 3]);
                        mbar_arrive(&sh.empty[s]);
                    }
                }
            }
            if (!ok) sh.fail = 1;
        } else if (FP8 && role < 4) {
            // ---- E4M3 rows to bf16, a thread a row ----
            const int r = role * 32 + lane;
            bool ok = true;
            Piece k;
            // A row's place in the cache: its entry in the block table is read a tile ahead of its
            // scales, which are a tile ahead of their use, so that nothing waits for a load that has
            // just been issued.
            struct Row {
                int entry, off;
                bool there;
            };
            const int psize = a.kv.page_size, step_entries = kTile / psize, step_off = kTile % psize;
            auto next_row = [&](int i, Row &x) {
                const int j = k.key(i) + r;
                if (i == 0 || k.i0 + i == k.ns) {
                    x.entry = j / psize;
                    x.off = j - x.entry * psize;
                } else {  // a tile further
                    x.entry += step_entries;
                    x.off += step_off;
                    if (x.off >= psize) x.off -= psize, ++x.entry;
                }
                x.there = i < k.nt && k.wanted(j, 1);
            };
            auto page = [&](const Row &x) {
                return ld_dep_if(x.there, a.seq.table + (int64_t)k.b * a.seq.max_pages + (x.there ? x.entry : 0));
            };
            // scale bytes of the row's key and value; 2^0 where there are none
            auto scales = [&](const Row &x, uint32_t page, uint32_t &sk, uint32_t &sv) {
                const bool there = x.there && page < (uint32_t)a.kv.pages;
                const int64_t at = there ? (int64_t)page * (a.kv.Hkv * psize) + (k.h * psize + x.off) : 0;
                sk = ld_byte_if(there, a.kv.k_scales + at, 127);
                sv = ld_byte_if(there, a.kv.v_scales + at, 127);
            };
            int s = 0, parity = 0, it = 0;  // stage, the parity of its phase, tiles so far
            for (int p = 0; ok && next_piece(p, k); ++p) {
                uint32_t sk, sv, then;
                Row at;
                next_row(0, at);
                scales(at, page(at), sk, sv);
                next_row(1, at);
                then = page(at);
                for (int i = 0; ok && i < k.nt; ++i) {
                    const uint32_t fk = scale_bf16(sk), fv = scale_bf16(sv);
                    scales(at, then, sk, sv);
                    next_row(i + 2, at);
                    then = page(at);
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        ok = ok && mbar_wait_fast(&sh.raw_full[s], parity, fail) &&
                             (C::kInside || it < kStages || mbar_wait_fast(&sh.empty[s], parity ^ 1, fail));
                        ok = __all_sync(kFullMask, ok);
                        if (!ok) break;
                        const uint32_t src = smem_addr(smem + C::kRawAt + s * C::kRawPitch) + r * D;
                        const uint32_t dst = smem_addr(ring + s * C::kStage) + r * 128;
                        auto chunk = [&](int ch) { return dst + (ch >> 3) * C::kPanel + 16 * ((ch & 7) ^ (r & 7)); };
#pragma unroll 1
                        for (int c0 = 0; c0 < D / 16; c0 += 2) {
                            uint4 x[2];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t from = src + 16 * (c0 + c);
                                from ^= (from >> 3) & (D == 128 ? 0x70 : 0x30);  // the TMA's swizzle, by the address
                                x[c] = lds16(from);
                            }
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                                uint32_t y[8];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint32_t h[2];
                                    half_pairs(w[j], h[0], h[1]);
#pragma unroll
                                    for (int z = 0; z < 2; ++z) y[2 * j + z] = mul_bf16(bf16_pair(h[z]), v ? fv : fk);
                                }
                                sts16(chunk(2 * (c0 + c)), make_uint4(y[0], y[1], y[2], y[3]));
                                sts16(chunk(2 * (c0 + c) + 1), make_uint4(y[4], y[5], y[6], y[7]));
                            }
                        }
                        if (v && k.edge(k.key(i), a.window, a.sinks)) {
                            uint32_t bad = 0;
#pragma unroll 1
                            for (int ch = 0; ch < D / 8; ++ch) {
                                const uint4 y = lds16(chunk(ch));
                                const uint32_t some = not_finite(y.x) | not_finite(y.y) | not_finite(y.z) | not_finite(y.w);
                                if (some) sts16(chunk(ch), make_uint4(finite_part(y.x), finite_part(y.y), finite_part(y.z), finite_part(y.w)));
                                bad |= some;
                            }
                            if (bad && k.wanted(k.key(i) + r, 1)) sh.fix = 1;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sh.full[s]);
                            if (!C::kInside) mbar_arrive(&sh.raw_empty[s]);
                        }
                        ++it;
                        if (++s == kStages) s = 0, parity ^= 1;
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
        if ((int)threadIdx.x < kStages) {
            int last = max(sh.issued[0], sh.issued[1]) - 1 - (int)threadIdx.x;
            if (last >= sh.issued[last & 1]) last -= kStages;
            if (last >= 0) mbar_wait(FP8 ? &sh.raw_full[last % kStages] : &sh.full[last % kStages], (last / kStages) & 1, nullptr);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free<512>(tmem);
    }
}

// The sums of the row blocks that several SMs share, a warp two rows; 16 blocks for each that may
// begin one.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ PrefillArgs d, int blocks) {
    constexpr int N = D / 32, kAhead = 2;  // channels a lane, sums in flight (few SMs share most blocks: 8 took 4 us more of 385)
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = blockIdx.x >> 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint4 rec = ld_dep_v4(d.ws + 16 * c0);
    const int n = (int)rec.w;  // SMs after the first
    if (n == 0) return;
    const Piece k = row_block(d, seq_span(a.seq, a.kv.page_size, (int)rec.x), (int)rec.z);
    const float *ml = reinterpret_cast<const float *>(d.ws + ws_ml(blocks));
    const float *sums = reinterpret_cast<const float *>(d.ws + ws_sums(blocks)) + N * lane;
    for (int r = (blockIdx.x & 15) * 8 + warp; r < k.rows; r += 128) {
        auto at = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0)) * kRows + r; };
        float m = -INFINITY, l = 0.0f, top = -INFINITY, base = 0.0f, sum = 0.0f, acc[N];
#pragma unroll
        for (int x = 0; x < N; ++x) acc[x] = 0.0f;
        for (int w0 = 0; w0 <= n; w0 += 32) {  // the SMs of whose m and l the lanes hold
            m = w0 + lane <= n ? ld_dep(ml + 2 * at(w0 + lane)) : -INFINITY;
            l = w0 + lane <= n ? ld_dep(ml + 2 * at(w0 + lane) + 1) : 0.0f;
            const int end = min(n + 1 - w0, 32);
            for (int i0 = 0; i0 < end; i0 += kAhead) {
                float v[kAhead][N];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float *src = sums + at(min(w0 + i0 + i, n)) * D;
                    if constexpr (N == 4) {
                        const uint4 q = ld_dep_v4(src);
                        v[i][0] = __uint_as_float(q.x), v[i][1] = __uint_as_float(q.y);
                        v[i][2] = __uint_as_float(q.z), v[i][3] = __uint_as_float(q.w);
                    } else {
#pragma unroll
                        for (int x = 0; x < N; ++x) v[i][x] = ld_dep(src + x);
                    }
                }
                if (w0 + i0 == 0) {  // after the first loads are on their way
                    top = m;
                    for (int i = lane + 32; i <= n; i += 32) top = fmaxf(top, ld_dep(ml + 2 * at(i)));
#pragma unroll
                    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
                    base = top == -INFINITY ? 0.0f : top;
                }
                const float f = exp2_fast(m - base), fl = l * f;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float g = __shfl_sync(kFullMask, f, i0 + i), gl = __shfl_sync(kFullMask, fl, i0 + i);
                    if (i0 + i >= end) break;
                    sum += gl;
#pragma unroll
                    for (int x = 0; x < N; ++x) acc[x] += v[i][x] * g;
                }
            }
        }
        const int token = (k.row0 + r) / d.G;
        const float inv = k.pos0 + token < 0 ? 0.0f : 1.0f / sum;
        const int64_t to = (int64_t)(k.first + token) * a.Hq + (int64_t)rec.y * d.G + (k.row0 + r - token * d.G);
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + to * D + N * lane);
#pragma unroll
        for (int x = 0; x < N; x += 2) dst[x / 2] = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
        if (a.lse && lane == 0) a.lse[to] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
    }
}

template <int D, bool FP8, bool TWO = false>
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
    const int blocks = sm_count();
    const cudaError_t err = launch_large<prefill_kernel<D, FP8, TWO>>(
        blocks, Cfg<D, FP8, TWO>::kThreads, Cfg<D, FP8, TWO>::kSmem, stream, kmap, vmap, d);
    if (err != cudaSuccess || !d.ws) return err;
    return launch_kernel(join_kernel<D>, 16 * blocks, 256, 0, stream, true, d, blocks);
}

}  // namespace

// The caller's may begin on 16 bytes.
size_t attn_prefill_workspace(int D) { return ws_bytes(sm_count(), D) + 16; }

cudaError_t launch_attn_prefill(const AttnArgs &a, void *workspace, cudaStream_t stream) {
    PrefillArgs d = {};
    d.a = a;
    d.G = a.Hq / a.kv.Hkv;
    d.box = a.kv.page_size & -a.kv.page_size;  // a box lies within a page
    if (d.box > kTile) d.box = kTile;
    d.ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + 31) / 32 * 32);
    // 32 bytes a store where the rows allow it: in two, a prompt of 8192 takes 388 us for 381, an 8-bit
    // one of 5 chunks 466 for 460
    d.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    const bool fp8 = a.kv.k_scales != nullptr;
    if (a.kv.D == 64) return fp8 ? launch<64, true>(d, stream) : launch<64, false>(d, stream);
    if (fp8) return launch<128, true>(d, stream);
    // One warp issues a request of TMA in about 110 clocks: 64 of 8 rows a step of 128 keys take
    // longer than the step.  Two loaders, for requests of 8 / 16 / 64 rows: chunks of 700 tokens
    // after 6000, 64 heads, 412 / 378 / 367 us, with one 659 / 403 / 357; 5 tokens after 3000 73 / 66
    // / 65, with one 82 / 64 / 62.  Rows of 128 bytes are half the requests.
    return d.box <= 16 ? launch<128, false, true>(d, stream) : launch<128, false>(d, stream);
}

}  // namespace ep
