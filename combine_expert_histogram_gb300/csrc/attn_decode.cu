// ep_attn_decode: attention of one new token a sequence over the paged cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  m the largest so far
//
// in one pass over the visible keys.  HBM-bound: a cache row is read once for all query
// heads that share it, up to 16 of them, which are the columns of 16 x 8 x 16 matrix
// instructions with 16 keys, then 16 channels of the values, as the rows (so few columns
// would leave 7/8 of a product in tensor memory unused).
//
// The work, a unit being 8 KB of one key head's keys and values, is one list over sequences
// and heads, of which every block takes an equal run, wherever sequences begin and end.  In
// it each of eight warps has every eighth unit, a ring of its own in shared memory that tiled
// TMA loads fill ahead, across the ends of heads and sequences, and sums of its own
// (m, l, o), which the warps add at the end of a head.  A head that several blocks share
// leaves its sums in the workspace, and the block that arrives last adds them (a second kernel
// for that took 5 us more: 3 from the last block's end to its first instruction).
//
// What it takes: 128 sequences of 800 - 8000 keys, 32 heads on 4, 1.16 GB, 178 us (6.5 TB/s); 3
// sequences of 210000 - 300000, 64 heads on 8, in 8 bits, 1.67 GB, 251 us (6.7 TB/s); one of 4096
// keys 10.9 us, of which 4 are the launch and the last join, 2 the first load's answer.
//
// Twelve warps with units of 4 KB (for 8-bit rows and heads of 64, whose units are small in keys)
// were slower, 353 us for 279 then: more merges, and fewer registers for a unit in flight.
#include "attn.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kHeads = 16;           // query heads of an item at most
// units a block takes at least (one sequence of 4096 keys, 32 heads on 4: 12.7 / 12.0 / 11.0 / 11.6 us with
// 8 / 12 / 16 / 24; of 1000 10.1 / 10.3 / 10.3 / 11.1)
constexpr int kLeast = 2 * kWarps;
// units of time that an item costs beside its own (128 sequences of up to 500 keys: 33.0 / 28.3 /
// 27.9 / 27.5 us with 8 / 12 / 16 / 24; of up to 8000, in 8 bits, 105 / 101 / 99 / 100)
constexpr int kItem = 16;
constexpr float kLog2e = 1.4426950408889634f;
// log2 of how far m may be behind the largest logit (so that most units need no maximum over the
// lanes), and what FP8 weights are raised by: fp16 from 2^15 down to 2^-32 of the largest
constexpr float kLag = 8.0f, kBoost = 7.0f;

// What a block leaves of a head that others share: [block][first or last][row].
struct Part {
    float m, l;  // in log2 units
};
struct Shared {
    uint64_t full[kWarps][3];
    int64_t sums[kWarps], found_at;
    int found_b, fail;
    Part part[kWarps][8];
};
template <int D, bool FP8>
struct Cfg {
    static constexpr int kRow = FP8 ? D : 2 * D;             // bytes of a cache row
    static constexpr int kUnit = 4096 / kRow;                // keys of a unit
    static constexpr int kGroups = kUnit / 8;                // of 8 rows, which a page holds together
    static constexpr int kPitch = kRow < 128 ? kRow : 128;   // a panel's row
    static constexpr int kPanels = kRow / kPitch;
    static constexpr int kPanel = kUnit * kPitch;
    static constexpr int kTile = kUnit * kRow;               // keys, then values
    static constexpr int kStages = 3;
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kScales = FP8 ? kWarps * 2 * 2 * kUnit : 0;  // of two units
    static constexpr int kMerge = kWarps * 8 * D * 4;  // eight heads of every warp's o
    static constexpr int kSmem = kRing + kMerge + kScales + (int)sizeof(Shared);
};

// The workspace: counts of arrivals [block][row] (of the heads that begin in a block), 0
// between calls; parts; sums.
__host__ __device__ constexpr size_t ws_parts(int blocks) { return (size_t)blocks * kHeads * 4; }
__host__ __device__ constexpr size_t ws_sums(int blocks) {
    return ws_parts(blocks) + (size_t)blocks * 2 * kHeads * sizeof(Part);
}
__host__ __device__ constexpr size_t ws_bytes(int blocks, int D) {
    return ws_sums(blocks) + (size_t)blocks * 2 * kHeads * D * 4;
}

struct DecodeArgs {
    AttnArgs a;
    int G, groups, heads, items;  // query heads a key head, in `groups` of up to `heads`; items a sequence
    int box, boxes;               // cache rows of a TMA box, boxes a unit
    uint8_t *ws;
};

// The visible keys of a sequence's newest token: [lo, L) and [0, S), S <= lo, as n units of
// U keys: ns of the first keys, then those from unit `first` on.
struct Keys {
    int L, lo, S, n, ns, first;
    __device__ __forceinline__ bool sees(int j) const { return j < L && (j >= lo || j < S); }
};
template <int U>
__device__ __forceinline__ Keys visible(const AttnArgs &a, int b) {
    Keys k;
    k.L = max(ld_dep(a.seq.kv_len + b), 0);
    const int most = a.seq.max_pages * a.kv.page_size;
    if (k.L > most) {
        raise_status(a.seq.status, EP_ERR_BAD_PAGE);
        k.L = most;
    }
    k.lo = a.window ? max(k.L - a.window, 0) : 0;
    k.S = a.sinks;
    if (k.S >= k.lo) k.lo = k.S = 0;
    k.first = k.lo / U;
    k.ns = min((k.S + U - 1) / U, k.first);
    // a sequence without a key has one unit that sees none
    k.n = max(k.ns + (k.L + U - 1) / U - k.first, 1);
    return k;
}

// x / y of numbers >= 0, in 32 bits where that does.
__device__ __forceinline__ int64_t divided(int64_t x, int64_t y) {
    if ((x | y) >> 32 == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}

// A place in the list of work: an item (sequence, key head, group of query heads).
template <int U>
struct Place {
    int b, item;
    int64_t at;  // the item's first place in the list
    Keys k;
    int64_t pad;  // > 0: an item's places are its units, rounded up to a multiple of this
    __device__ __forceinline__ int64_t places() const {
        return pad == 0 ? k.n + kItem : divided(k.n + pad - 1, pad) * pad;
    }
    __device__ __forceinline__ void next(const DecodeArgs &d) {
        at += places();
        if (++item == d.items) {
            item = 0;
            if (++b < d.a.seq.B) k = visible<U>(d.a, b);
        }
    }
    __device__ __forceinline__ int key(int unit) const {
        return (unit < k.ns ? unit : unit - k.ns + k.first) * U;
    }
};

template <bool T>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (T)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values, two of a row a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// c (16 x 8) += a (16 x 16) b (16 x 8), fp16 or bf16.
template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (HALF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A load that does not look into L1: another block's words.
template <int N>
__device__ __forceinline__ auto ld_l2(const void *p) {
    if constexpr (N == 2) {
        uint2 v;
        asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
        return v;
    } else {
        uint4 v;
        asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p)
                     : "memory");
        return v;
    }
}
// A query head's result, by one warp; `top` in log2 units.  A head that sees no key is 0; one
// that does, and whose logits are all -infinity, 0 / 0.
template <int D>
__device__ __forceinline__ void store_head(const AttnArgs &a, int64_t to, int lane, bool keys, float top,
                                           float sum, const float (&acc)[D / 32]) {
    const float inv = keys ? 1.0f / sum : 0.0f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + to * D + D / 32 * lane);
#pragma unroll
    for (int x = 0; x < D / 32; x += 2) dst[x / 2] = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
    if (a.lse && lane == 0) a.lse[to] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

// Heads of which this block has a part: the block where they begin, how many follow that one,
// row of the output.
struct Share {
    int c0, n, heads;
    int64_t row0;
};
// The sum of all blocks' parts of a head, by one warp.
template <int D>
__device__ __forceinline__ void join_head(const AttnArgs &a, const Share &t, int r, const Part *parts,
                                          const float *sums, int lane) {
    constexpr int N = D / 32, kAhead = 20;  // channels a lane, sums in flight
    auto at = [&](int i) { return (size_t)(2 * (t.c0 + i) + (i == 0)) * kHeads + r; };
    auto part = [&](int i) {
        const uint2 q = ld_l2<2>(&parts[at(min(i, t.n))]);
        return i <= t.n ? Part{__uint_as_float(q.x), __uint_as_float(q.y)} : Part{-INFINITY, 0.0f};
    };
    const float *from = sums + N * lane;
    Part mine = part(lane);
    float top = mine.m, base = 0.0f, sum = 0.0f, acc[N];
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] = 0.0f;
    for (int w0 = 0; w0 <= t.n; w0 += 32) {  // the blocks of whose m and l the lanes hold
        const int end = min(t.n + 1 - w0, 32);
        for (int i0 = 0; i0 < end; i0 += kAhead) {
            decltype(ld_l2<N>(from)) v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) v[i] = ld_l2<N>(from + at(min(w0 + i0 + i, t.n)) * D);
            if (w0 + i0 == 0) {  // after the first loads are on their way
                for (int i = lane + 32; i <= t.n; i += 32) top = fmaxf(top, part(i).m);
#pragma unroll
                for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
                base = top == -INFINITY ? 0.0f : top;
            } else if (i0 == 0) {
                mine = part(w0 + lane);
            }
            const float f = exp2_fast(mine.m - base), fl = mine.l * f;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float y = __shfl_sync(kFullMask, f, i0 + i), yl = __shfl_sync(kFullMask, fl, i0 + i);
                if (i0 + i >= end) break;
                sum += yl;
                acc[0] += __uint_as_float(v[i].x) * y;
                acc[1] += __uint_as_float(v[i].y) * y;
                if constexpr (N == 4) {
                    acc[2] += __uint_as_float(v[i].z) * y;
                    acc[3] += __uint_as_float(v[i].w) * y;
                }
            }
        }
    }
    store_head<D>(a, t.row0 + r, lane, true, top, sum, acc);
}

// A warp's stream of units: what is to be loaded next.
template <int D, bool FP8>
struct Loader {
    using C = Cfg<D, FP8>;
    Place<C::kUnit> p;
    int64_t x0, x1;       // the block's run
    int u, end, h;        // the warp's next unit in the item, the piece's end in it; key head
    int left, held;       // units of which the lanes (still) hold the pages
    int page, row;        // lane: of box lane % (boxes a unit); the page past the last: none
    int slot, scale_slot, behind;  // behind: whose scales are not yet in shared memory, or -1
    uint2 scales;         // lane: eight of those
    bool more;

    __device__ __forceinline__ void piece(const DecodeArgs &d, int warp) {
        h = d.groups == 1 ? p.item : p.item / d.groups;
        u = (int)(max(x0, p.at) - p.at) + warp;
        end = (int)min((int64_t)p.k.n, x1 - p.at);
        left = 0;
    }
    __device__ __forceinline__ void pages(const DecodeArgs &d, int boxes, int lane) {
        const AttnArgs &a = d.a;
        const int at = lane / boxes, unit = u + kWarps * at;
        page = a.kv.pages;
        row = 0;
        if (unit < end) {
            const int key = p.key(unit) + d.box * (lane - at * boxes);
            if (key < p.k.L && (key + d.box > p.k.lo || key < p.k.S)) {
                const int entry = key / a.kv.page_size;
                const int q = page_of(a.kv, a.seq, p.b, entry);
                if (q >= 0) page = q;
                row = key - entry * a.kv.page_size;
            }
        }
        left = held;
    }
    __device__ __forceinline__ void store_scales(uint32_t to, int lane) {
        if (FP8 && behind >= 0) {
            if (lane < 2 * C::kGroups)
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to + behind * 2 * C::kUnit + 8 * lane),
                             "r"(scales.x), "r"(scales.y)
                             : "memory");
            behind = -1;
        }
    }
    // Ask for the next unit, if there is one.
    __device__ __forceinline__ void issue(const DecodeArgs &d, const CUtensorMap *kmap, const CUtensorMap *vmap,
                                          uint32_t ring, uint32_t scale_ring, uint64_t *full, int warp, int lane) {
        const AttnArgs &a = d.a;
        store_scales(scale_ring, lane);
        while (more && u >= end) {
            p.next(d);
            more = p.at < x1;
            if (more) piece(d, warp);
        }
        if (!more) return;
        const int boxes = d.boxes;
        if (left == 0) pages(d, boxes, lane);
        const int from = boxes * (held - left);
        const uint32_t st = ring + slot * 2 * C::kTile;
        const bool leader = elect_one();
        if (leader) expect_bytes(full + slot, 2 * C::kTile);
        for (int x = 0; x < boxes; ++x) {
            const int px = __shfl_sync(kFullMask, page, from + x), rx = __shfl_sync(kFullMask, row, from + x);
            if (leader) {
#pragma unroll
                for (int n = 0; n < C::kPanels; ++n) {
                    const uint32_t to = st + n * C::kPanel + x * d.box * C::kPitch;
                    tma_load_4d(to, kmap, 128 * n, h, rx, px, full + slot);
                    tma_load_4d(to + C::kTile, vmap, 128 * n, h, rx, px, full + slot);
                }
            }
        }
        if constexpr (FP8) {
            const int r = 8 * (lane % C::kGroups), x = r / d.box;
            const int px = __shfl_sync(kFullMask, page, from + x), rx = __shfl_sync(kFullMask, row, from + x);
            scales = make_uint2(0, 0);
            if (lane < 2 * C::kGroups && px < a.kv.pages) {
                const uint8_t *src = lane < C::kGroups ? a.kv.k_scales : a.kv.v_scales;
                const int64_t at = ((int64_t)px * a.kv.Hkv + h) * a.kv.page_size + rx + (r - x * d.box);
                asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(scales.x), "=r"(scales.y) : "l"(src + at) : "memory");
            }
            behind = scale_slot;
            scale_slot ^= 1;
        }
        u += kWarps;
        --left;
        slot = slot + 1 == C::kStages ? 0 : slot + 1;
    }
};

// NH: tiles of eight query heads.
template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ DecodeArgs d) {
    using C = Cfg<D, FP8>;
    // all of the block's shared memory: the ring (the swizzle wants 1024-byte alignment; static
    // arrays would push it off), eight heads' sums, the scales
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + C::kRing + C::kMerge + C::kScales);
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * 2 * C::kTile;
    float *merge = reinterpret_cast<float *>(smem + C::kRing);
    const uint32_t scale_ring = smem_addr(smem) + C::kRing + C::kMerge + warp * 2 * 2 * C::kUnit;
    uint64_t *full = sh.full[warp];
    int *arrivals = reinterpret_cast<int *>(d.ws);
    Part *parts = reinterpret_cast<Part *>(d.ws + ws_parts(gridDim.x));
    float *out_sums = reinterpret_cast<float *>(d.ws + ws_sums(gridDim.x));
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * C::kStages; ++i) mbar_init(&sh.full[0][i], 1);
        sh.fail = 0;
        mbar_init_fence();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---- the block's run of the list, and its first item ----
    const int64_t blocks = gridDim.x;
    int64_t total = 0, per, x0, x1;
    Place<C::kUnit> p;
    p.pad = 0;
    if (a.seq.B <= 32) {
        // few sequences, where latency counts: every warp by itself (and in 32 bits where
        // that does)
        Keys k = {};
        int64_t n = 0;
        if (lane < a.seq.B) {
            k = visible<C::kUnit>(a, lane);
            n = (int64_t)(k.n + kItem) * d.items;
        }
        auto scan = [&](int64_t incl) {
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int64_t o = __shfl_up_sync(kFullMask, incl, s);
                if (lane >= s) incl += o;
            }
            return incl;
        };
        int64_t incl = scan(n);
        total = __shfl_sync(kFullMask, incl, 31);
        per = max(divided(total + blocks - 1, blocks), (int64_t)kLeast);
        // Runs that end with their item, where that makes them at most 12 units (2 us)
        // longer: a block with two items' parts comes 3 us later than the others (one sequence of 16000
        // keys: 14.7 us, 15.7 with runs that may not be longer).
        const int64_t spare = blocks - (int64_t)a.seq.B * d.items;
        if (spare > 0) {
            const int64_t units = total - (int64_t)a.seq.B * d.items * kItem;
            const int64_t longer = max(divided(units + spare - 1, spare), (int64_t)kLeast);
            if (longer <= per + 12) {
                per = p.pad = longer;
                if (lane < a.seq.B) n = divided(k.n + per - 1, per) * per * d.items;
                incl = scan(n);
                total = __shfl_sync(kFullMask, incl, 31);
            }
        }
        x0 = blockIdx.x * per;
        x1 = min(x0 + per, total);
        __syncthreads();  // the barriers are initialised
        if (x0 >= x1) return;
        p.b = __ffs(__ballot_sync(kFullMask, x0 < incl)) - 1;
        p.at = __shfl_sync(kFullMask, incl - n, p.b);
        p.k = {__shfl_sync(kFullMask, k.L, p.b),  __shfl_sync(kFullMask, k.lo, p.b), __shfl_sync(kFullMask, k.S, p.b),
               __shfl_sync(kFullMask, k.n, p.b),  __shfl_sync(kFullMask, k.ns, p.b), __shfl_sync(kFullMask, k.first, p.b)};
    } else {
        // exclusive sums of the sequences' units, kThreads at a time; the first ones are kept
        int64_t excl0 = 0, n0 = 0;
        auto scan = [&](int b0, int64_t &n, int64_t &excl) {
            const int b = b0 + threadIdx.x;
            n = b < a.seq.B ? (int64_t)(visible<C::kUnit>(a, b).n + kItem) * d.items : 0;
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
            for (int i = 0; i < kWarps; ++i) {
                if (i == warp) below = all;
                all += sh.sums[i];
            }
            excl = incl - n + below;
            return all;
        };
        for (int b0 = 0; b0 < a.seq.B; b0 += kThreads) {
            int64_t n, excl;
            total += scan(b0, n, excl);
            if (b0 == 0) n0 = n, excl0 = excl;
        }
        per = max(divided(total + blocks - 1, blocks), (int64_t)kLeast);
        x0 = blockIdx.x * per;
        x1 = min(x0 + per, total);
        if (x0 >= x1) return;
        int64_t before = 0;
        for (int b0 = 0;; b0 += kThreads) {
            int64_t n = n0, excl = excl0, all = total;
            if (a.seq.B > kThreads) all = scan(b0, n, excl);
            if (x0 >= before + excl && x0 < before + excl + n) {
                sh.found_b = b0 + threadIdx.x;
                sh.found_at = before + excl;
            }
            before += all;
            if (before > x0 || b0 + kThreads >= a.seq.B) break;
        }
        __syncthreads();
        p.b = sh.found_b;
        p.at = sh.found_at;
        p.k = visible<C::kUnit>(a, p.b);
    }
    p.item = (int)divided(x0 - p.at, p.places());
    p.at += p.item * p.places();

    Loader<D, FP8> load;
    load.p = p;
    load.x0 = x0;
    load.x1 = x1;
    load.held = 32 / d.boxes;
    load.slot = load.scale_slot = 0;
    load.behind = -1;
    load.more = true;
    load.piece(d, warp);
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) load.issue(d, &kmap, &vmap, ring, scale_ring, full, warp, lane);

    const int row = lane >> 2, c = lane & 3;  // of the matrix fragments
    int slot = 0, scale_slot = 0;
    uint32_t phase = 0;
    // The queries of an item: head `row` of each tile is the second factor's column.  FP8: a
    // lane's E4M3 key bytes are D / 4 neighbours, of which a step takes four.
    uint32_t word[NH][D / 8];
    auto fetch = [&](const Place<C::kUnit> &at) {
        const int h = at.item / d.groups, g = at.item - h * d.groups;
        const int heads = min(d.heads, d.G - g * d.heads);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int r = row + 8 * n;
            const uint16_t *src = a.q + at.b * a.q_stride + (int64_t)(h * d.G + g * d.heads + r) * D;
            if constexpr (!FP8) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    word[n][i] = ld_dep_if(r < heads, src + 8 * i + 2 * c);
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 v = ld_dep_v4_if(r < heads, src + D / 4 * c + 8 * i);
                    word[n][4 * i] = v.x;
                    word[n][4 * i + 1] = v.y;
                    word[n][4 * i + 2] = v.z;
                    word[n][4 * i + 3] = v.w;
                }
            }
        }
    };
    Share first = {}, last = {};  // heads that begin before the run, that end behind it
    int first_before[NH];
    if (x0 >= p.at + p.k.n) p.next(d);  // the run begins behind the item's units
    if (p.at < x1) fetch(p);
    while (p.at < x1) {
        const int h = p.item / d.groups, g = p.item - h * d.groups;
        const int q0 = h * d.G + g * d.heads, heads = min(d.heads, d.G - g * d.heads);
        uint32_t q[NH][D / 16][2];
        float to_log2[NH][2];  // logits in log2 units, of the heads 2 c and 2 c + 1
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            to_log2[n][0] = to_log2[n][1] = a.scale * kLog2e;
            if constexpr (!FP8) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) q[n][i / 2][i & 1] = word[n][i];
            } else {
                // as fp16 next to 2^8 at most, off by less than 2^-32 of the head's largest
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(word[n][i])), fabsf(bf16_hi(word[n][i]))));
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
                // up = 2^k with amax * up in [2^7, 2^8), within what fp32 has of both
                const int e = min(max((int)(__float_as_uint(amax) >> 23), 8), 254);
                const float up = __uint_as_float((uint32_t)(261 - e) << 23);
                const float down = __uint_as_float((uint32_t)max(e - 7, 0) << 23);
#pragma unroll
                for (int i = 0; i < 2; ++i) to_log2[n][i] *= __shfl_sync(kFullMask, down, 4 * (2 * c + i));
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    q[n][i / 2][i & 1] = pack_half(bf16_lo(word[n][i]) * up, bf16_hi(word[n][i]) * up);
            }
        }
        // of the heads 2 c and 2 c + 1: largest logit, sum of probabilities (this lane's keys'),
        // FP8: largest logit with its value's scale
        float o[NH][D / 16][4], m[NH][2], l[NH][2], mv[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) m[n][i] = mv[n][i] = -INFINITY, l[n][i] = 0.0f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][t][i] = 0.0f;
        }

        const int piece0 = (int)(max(x0, p.at) - p.at), piece1 = (int)min((int64_t)p.k.n, x1 - p.at);
        for (int u = piece0 + warp; u < piece1; u += kWarps) {
            if (!__all_sync(kFullMask, mbar_wait_fast(full + slot, (phase >> slot) & 1, &sh.fail))) {
                sh.fail = 1;
                load.more = false;
            }
            phase ^= 1u << slot;
            __syncwarp();
            load.issue(d, &kmap, &vmap, ring, scale_ring, full, warp, lane);
            const uint32_t st = ring + slot * 2 * C::kTile, sv = st + C::kTile;
            const uint32_t sc = scale_ring + scale_slot * 2 * C::kUnit;
            scale_slot ^= 1;
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
            const int key = p.key(u);
            const bool whole = key + C::kUnit <= p.k.L && key >= p.k.lo;
            if (!whole) {  // values that are not seen may be anything, and 0 * NaN is NaN
                for (int x = lane; x < C::kTile / 16; x += 32) {
                    const int r = x * 16 % C::kPanel / C::kPitch;
                    if (!p.k.sees(key + r))
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(sv + 16 * x), "r"(0) : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
            }

            // ---- logits, 16 keys a tile ----
            constexpr int KT = C::kUnit / 16;
            float s[KT][NH][4];  // keys row, row + 8; heads 2 c, 2 c + 1
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][n][i] = 0.0f;
            float ev[KT][2];  // FP8: log2 of the values' scales
            if constexpr (!FP8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        const int r = 16 * t + (lane & 15), ch = 2 * k + (lane >> 4);
                        uint32_t f[4];
                        ldmatrix4<false>(f, st + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7)));
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma<false>(s[t][n], f, q[n][k][0], q[n][k][1]);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        const int r = 16 * t + row, ch = D / 64 * c + j;
                        uint32_t at = st + r * C::kPitch + 16 * ch;
                        at ^= (at >> 3) & (D == 128 ? 0x70 : 0x30);  // the TMA's swizzle, by the address
                        const uint4 x = lds16(at), y = lds16(at + 8 * C::kPitch);
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t f[4];
                            half_pairs(xw[i], f[0], f[2]);
                            half_pairs(yw[i], f[1], f[3]);
#pragma unroll
                            for (int n = 0; n < NH; ++n) mma<true>(s[t][n], f, q[n][4 * j + i][0], q[n][4 * j + i][1]);
                        }
                    }
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t ek, e;
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(ek) : "r"(sc + 16 * t + 8 * i + row) : "memory");
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(sc + C::kUnit + 16 * t + 8 * i + row) : "memory");
                        // 2^(ek - 127), NaN for 255; 0 for ek = 0, which is off by less than the logits'
                        // last bit: 2^-127 of a sum below 2^17 |q|.  The product of the scales first: the
                        // queries were raised, and a sum times the key's scale alone may be past fp32.
                        const float f = __uint_as_float(ek == 255 ? 0x7fffffffu : ek << 23);
#pragma unroll
                        for (int n = 0; n < NH; ++n) {
                            s[t][n][2 * i] *= f * to_log2[n][0];
                            s[t][n][2 * i + 1] *= f * to_log2[n][1];
                        }
                        // e - 127, by a number whose last bits are e
                        ev[t][i] = e == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(0x4b000000u | e) - 8388735.0f;
                    }
            }
            if constexpr (!FP8) {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[t][n][i] *= to_log2[n][i & 1];
            }
            if (!whole) {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!p.k.sees(key + 16 * t + 8 * i + row)) {
                            ev[t][i] = 0.0f;  // the scale may be anything too
#pragma unroll
                            for (int n = 0; n < NH; ++n) s[t][n][2 * i] = s[t][n][2 * i + 1] = -INFINITY;
                        }
            }
            float top[NH][2], topv[NH][2];
            bool grown = false;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[n][i] = topv[n][i] = -INFINITY;
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        top[n][i] = fmaxf(top[n][i], fmaxf(s[t][n][i], s[t][n][2 + i]));
                        if constexpr (FP8)
                            topv[n][i] = fmaxf(topv[n][i], fmaxf(s[t][n][i] + ev[t][0], s[t][n][2 + i] + ev[t][1]));
                    }
                    grown |= top[n][i] > m[n][i] + kLag || (FP8 && topv[n][i] > mv[n][i] + kLag);
                }
            if (__any_sync(kFullMask, grown)) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float a1 = fmaxf(m[n][i], top[n][i]), a2 = fmaxf(mv[n][i], topv[n][i]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) {
                            a1 = fmaxf(a1, __shfl_xor_sync(kFullMask, a1, x));
                            if constexpr (FP8) a2 = fmaxf(a2, __shfl_xor_sync(kFullMask, a2, x));
                        }
                        // a head that has seen no key yet has nothing to scale down
                        const float f = a1 == -INFINITY ? 1.0f : exp2_fast(m[n][i] - a1);
                        const float fo = !FP8 ? f : a2 == -INFINITY ? 1.0f : exp2_fast(mv[n][i] - a2);
                        l[n][i] *= f;
#pragma unroll
                        for (int t = 0; t < D / 16; ++t) {
                            o[n][t][i] *= fo;
                            o[n][t][2 + i] *= fo;
                        }
                        m[n][i] = a1;
                        mv[n][i] = a2;
                    }
            }
            float base[NH][2], basev[NH][2];
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // a head that has seen no key yet subtracts 0 from its -infinities
                    base[n][i] = m[n][i] == -INFINITY ? 0.0f : m[n][i];
                    // the value's scale belongs to the weight
                    basev[n][i] = kBoost - (mv[n][i] == -INFINITY ? 0.0f : mv[n][i]);
                }
            // ---- probabilities, and o += v p, sixteen keys at a time ----
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                uint32_t hi[NH][2], lo[NH][2];  // keys 2 c, 2 c + 1 (and + 8) of head `row`
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = s[t][n][2 * i], y = s[t][n][2 * i + 1];
                        const float ex = exp2_fast(x - base[n][0]), ey = exp2_fast(y - base[n][1]);
                        l[n][0] += ex;
                        l[n][1] += ey;
                        if constexpr (FP8) {
                            hi[n][i] = transposed(pack_half(exp2_fast(x + (ev[t][i] + basev[n][0])),
                                                            exp2_fast(y + (ev[t][i] + basev[n][1]))));
                        } else {
                            // p as two bf16, its upper bits and what they leave, off by 2^-16 of it
                            // (one would be off by 2^-8, and the products are not what bounds the
                            // kernel).  p's last bit is set, so that neither is below 0, and the second
                            // is 0 only where the first is: an infinite value times both stays infinite.
                            const uint32_t bx = __float_as_uint(ex) | 1, by = __float_as_uint(ey) | 1;
                            const uint32_t w = __byte_perm(bx, by, 0x7632);
                            hi[n][i] = transposed(w);
                            lo[n][i] = transposed(
                                pack_bf16(__uint_as_float(bx) - bf16_lo(w), __uint_as_float(by) - bf16_hi(w)));
                        }
                    }
                if constexpr (!FP8) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const int r = 16 * t + (lane & 7) + ((lane >> 4) << 3), ch = 2 * x + ((lane >> 3) & 1);
                        uint32_t f[4];
                        ldmatrix4<true>(f, sv + (ch >> 3) * C::kPanel + r * 128 + 16 * ((ch & 7) ^ (r & 7)));
#pragma unroll
                        for (int n = 0; n < NH; ++n) {
                            mma<false>(o[n][x], f, hi[n][0], hi[n][1]);
                            mma<false>(o[n][x], f, lo[n][0], lo[n][1]);
                        }
                    }
                } else {
                    // the lane's four keys, D / 8 channels from D / 8 * row on: rows `row` and
                    // `row` + 8 of the product's tile x are channels D / 8 * row + 2 x and + 1
                    uint32_t v[4][D / 32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
                        uint32_t at = sv + r * C::kPitch + D / 8 * row;
                        at ^= (at >> 3) & (D == 128 ? 0x70 : 0x30);
                        if constexpr (D == 128) {
                            const uint4 x = lds16(at);
                            v[i][0] = x.x;
                            v[i][1] = x.y;
                            v[i][2] = x.z;
                            v[i][3] = x.w;
                        } else {
                            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                         : "=r"(v[i][0]), "=r"(v[i][1])
                                         : "r"(at)
                                         : "memory");
                        }
                    }
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        uint32_t f[4];
                        half_pairs(__byte_perm(v[0][x], v[1][x], 0x5140), f[0], f[1]);
                        half_pairs(__byte_perm(v[2][x], v[3][x], 0x5140), f[2], f[3]);
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma<true>(o[n][2 * x], f, hi[n][0], hi[n][1]);
                        half_pairs(__byte_perm(v[0][x], v[1][x], 0x7362), f[0], f[1]);
                        half_pairs(__byte_perm(v[2][x], v[3][x], 0x7362), f[2], f[3]);
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma<true>(o[n][2 * x + 1], f, hi[n][0], hi[n][1]);
                    }
                }
            }
        }

        Place<C::kUnit> after = p;
        after.next(d);
        if (NH == 1 && after.at < x1) fetch(after);  // its latency passes under the merge

        // ---- the warps' sums together, eight heads at a time ----
        const bool starts = p.at >= x0, ends = p.at + p.k.n <= x1;
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            if (8 * n >= heads) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][i] += __shfl_xor_sync(kFullMask, l[n][i], x);
                const int r = 2 * c + i;
                if (row == 0) sh.part[warp][r] = {m[n][i], l[n][i]};
                // FP8: from the scaled weights' unit to the probabilities', in two steps, as one of 2^-134
                // (a value's scale of 2^-127) would be 0
                const float f = !FP8 ? 1.0f : m[n][i] == -INFINITY ? 0.0f : exp2_fast(0.5f * (mv[n][i] - m[n][i] - kBoost));
                float *to = merge + (warp * 8 + r) * D;
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // channel 16 t + row + 8 x, FP8: D/8 row + 2 t + x, whose place is
                        // 8 (2 t + x) + row there
                        const int at = 16 * t + row + 8 * x;
                        to[at ^ (8 * c)] = FP8 ? o[n][t][2 * x + i] * f * f : o[n][t][2 * x + i];
                    }
            }
            __syncthreads();
            const int r = 8 * n + warp;  // this warp's head
            if (r < heads) {
                constexpr int N = D / 32;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.part[i][warp].m);
                const float base = top == -INFINITY ? 0.0f : top;
                float acc[N];
#pragma unroll
                for (int x = 0; x < N; ++x) acc[x] = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float f = exp2_fast(sh.part[i][warp].m - base);
                    sum += sh.part[i][warp].l * f;
                    const float *from = merge + (i * 8 + warp) * D;
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        const int ch = N * lane + x, at = FP8 ? ch % (D / 8) * 8 + ch / (D / 8) : ch;
                        acc[x] += from[at ^ (8 * (warp >> 1))] * f;
                    }
                }
                if (starts && ends) {
                    store_head<D>(a, (int64_t)p.b * a.Hq + q0 + r, lane, p.k.L > 0, top, sum, acc);
                } else {
                    const size_t to = (size_t)(2 * blockIdx.x + starts) * kHeads + r;
                    float *dst = out_sums + to * D + N * lane;
#pragma unroll
                    for (int x = 0; x < N; ++x) dst[x] = acc[x];
                    if (lane == 0) parts[to] = {top, sum};
                }
            }
            __syncthreads();
        }
        if (!(starts && ends)) {
            Share &t = starts ? last : first;
            t.c0 = starts ? (int)blockIdx.x : (int)divided(p.at, per);
            t.n = (int)divided(p.at + p.k.n - 1, per) - t.c0;
            t.row0 = (int64_t)p.b * a.Hq + q0;
            t.heads = heads;
            if (!starts) {
                __threadfence();
#pragma unroll
                for (int n = 0; n < NH; ++n)
                    if (8 * n + warp < heads && lane == 0) first_before[n] = atomicAdd(arrivals + t.c0 * kHeads + 8 * n + warp, 1);
            }
        }
        if (NH > 1 && after.at < x1) fetch(after);
        p = after;
    }

    // ---- heads that several blocks share: the warp that comes last to one adds their sums, in
    // the blocks' order.  At the end of the run: nothing of the block's waits for it ----
    if (last.heads) __threadfence();
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const int r = 8 * n + warp;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const Share t = which ? last : first;
            if (r >= t.heads) continue;
            int before = 0;
            if (lane == 0) {
                int *count = arrivals + t.c0 * kHeads + r;
                before = which ? atomicAdd(count, 1) : first_before[n];
                if (before == t.n) *count = 0;
                // a workspace that was not zeros
                if (before < 0 || before > t.n) raise_status(a.seq.status, EP_ERR_INVALID_ARG);
            }
            before = __shfl_sync(kFullMask, before, 0);
            if (before != t.n) continue;
            __threadfence();
            join_head<D>(a, t, r, parts, out_sums, lane);
        }
    }
    __syncwarp();
    if (sh.fail) {
        if (threadIdx.x == 0) raise_status(a.seq.status, EP_ERR_TIMEOUT);
        // a load that was given up may still be landing: wait, again with a limit
        for (int i = 0; i < C::kStages; ++i) mbar_wait(full + i, ((phase >> i) & 1) ^ 1, nullptr);
    }
}

template <int D, bool FP8>
cudaError_t launch(DecodeArgs d, cudaStream_t stream) {
    using C = Cfg<D, FP8>;
    const KvArgs &kv = d.a.kv;
    d.box = kv.page_size & -kv.page_size;  // a box lies within a page
    if (d.box > C::kUnit) d.box = C::kUnit;
    d.boxes = C::kUnit / d.box;
    CUtensorMap kmap, vmap;
    const int64_t dims[4] = {C::kRow, kv.Hkv, kv.page_size, kv.pages};
    const int64_t strides[3] = {kv.head_stride, kv.row_stride, kv.page_stride};
    const int box[4] = {C::kPitch, 1, d.box, 1};
    const auto swizzle = C::kPitch < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!encode_bytes(&kmap, kv.k, 4, dims, strides, box, swizzle) ||
        !encode_bytes(&vmap, kv.v, 4, dims, strides, box, swizzle))
        return cudaErrorInvalidValue;
    const int blocks = sm_count();
    return d.heads <= 8 ? launch_large<decode_kernel<D, FP8, 1>>(blocks, kThreads, C::kSmem, stream, kmap, vmap, d)
                        : launch_large<decode_kernel<D, FP8, 2>>(blocks, kThreads, C::kSmem, stream, kmap, vmap, d);
}

}  // namespace

size_t attn_decode_workspace(int, int, int, int D) { return ws_bytes(sm_count(), D); }

cudaError_t launch_attn_decode(const AttnArgs &a, void *workspace, cudaStream_t stream) {
    DecodeArgs d = {};
    d.a = a;
    d.G = a.Hq / a.kv.Hkv;
    d.groups = (d.G + kHeads - 1) / kHeads;
    d.heads = (d.G + d.groups - 1) / d.groups;
    d.items = a.kv.Hkv * d.groups;
    d.ws = static_cast<uint8_t *>(workspace);
    const bool fp8 = a.kv.k_scales != nullptr;
    if (a.kv.D == 64) return fp8 ? launch<64, true>(d, stream) : launch<64, false>(d, stream);
    return fp8 ? launch<128, true>(d, stream) : launch<128, false>(d, stream);
}

}  // namespace ep
