// ep_attn_decode: attention of one new token a sequence over the paged cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  m the largest so far
//
// in one pass over the visible keys.  HBM-bound: a cache row is read once for all query
// heads that share it, up to 16 of them, which are the rows of a 16 x 8 x 16 matrix
// instruction (few rows: the 128-row instructions of tensor memory would be idle for
// 7/8; the memory's rate leaves these 1/4 used).
//
// The work, 16 keys of one key head being a unit, is one list over sequences and heads, of
// which every block takes an equal run, wherever sequences begin and end.  In it each of
// eight warps has every eighth unit, a ring of its own in shared memory that
// asynchronous copies fill ahead, across the ends of heads and sequences, and sums of its own
// (m, l, o), which the warps add at the end of a head.  A head that several blocks share
// leaves its sums in the workspace, and a second kernel adds them in order.
#include "attn.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kUnit = 16;            // keys of a unit
constexpr int kHeads = 16;           // query heads of an item
constexpr int kLeast = 2 * kWarps;   // units a block takes at least
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool FP8>
struct Cfg {
    static constexpr int kRow = FP8 ? D : 2 * D;             // bytes of a cache row
    static constexpr int kTile = kUnit * kRow;               // keys, then values
    static constexpr int kStage = 2 * kTile + (FP8 ? 32 : 0);  // and their scales
    static constexpr int kStages = (FP8 ? 20480 : 24576) / (2 * kTile);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * 8 * D * 4;  // eight rows of every warp's o
    static constexpr int kSmem = kRing + kMerge;
};

// What a block leaves of a head that others share: [block][first or last][row].
struct Part {
    float m, l;  // in log2 units
};
__host__ __device__ constexpr size_t ws_parts(int blocks) { return (size_t)blocks * 16; }
__host__ __device__ constexpr size_t ws_sums(int blocks) {
    return ws_parts(blocks) + (size_t)blocks * 2 * kHeads * sizeof(Part);
}
__host__ __device__ constexpr size_t ws_bytes(int blocks, int D) {
    return ws_sums(blocks) + (size_t)blocks * 2 * kHeads * D * 4;
}

struct DecodeArgs {
    AttnArgs a;
    int G, groups, items;  // query heads a key head, groups of 16 of them, items a sequence
    uint8_t *ws;
};

// The visible keys of a sequence's newest token: [lo, L) and [0, S), S <= lo, as n units.
struct Keys {
    int L, lo, S, n, first;  // units [0, n - ...) of the first keys, then from unit `first` on
    int ns;
};
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
    k.first = k.lo / kUnit;
    k.ns = min((k.S + kUnit - 1) / kUnit, k.first);
    // a sequence without a key has one unit that sees none
    k.n = max(k.ns + (k.L + kUnit - 1) / kUnit - k.first, 1);
    return k;
}

// A place in the list of work: an item (sequence, key head, group of query heads).
struct Place {
    int b, item;
    int64_t at;  // the item's first unit in the list
    Keys k;
    __device__ __forceinline__ void next(const DecodeArgs &d) {
        at += k.n;
        if (++item == d.items) {
            item = 0;
            if (++b < d.a.seq.B) k = visible(d.a, b);
        }
    }
    __device__ __forceinline__ int key(int unit) const {
        return (unit < k.ns ? unit : unit - k.ns + k.first) * kUnit;
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
// Two E4M3 values (the low and the high half's bytes) -> two fp16, exactly.
__device__ __forceinline__ uint32_t half_pair(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// A warp's stream of units: what is to be loaded next.
template <int D, bool FP8>
struct Loader {
    using C = Cfg<D, FP8>;
    Place p;
    int64_t x0, x1;       // the block's run
    int u, end;           // the warp's next unit in the item, the piece's end in it
    int left;             // units whose pages the lanes hold
    int64_t off, scale;   // lane: the row of half lane & 1 of unit u + 8 (lane / 2), or -1
    int slot;
    bool more;

    __device__ __forceinline__ void piece(int warp) {
        u = (int)(max(x0, p.at) - p.at) + warp;
        end = (int)min((int64_t)p.k.n, x1 - p.at);
        left = 0;
    }
    __device__ __forceinline__ void pages(const DecodeArgs &d, int lane) {
        const AttnArgs &a = d.a;
        const int unit = u + kWarps * (lane / 2);
        off = -1;
        scale = 0;
        if (unit < end) {
            const int key = p.key(unit) + 8 * (lane & 1);
            if (key < p.k.L && (key + 8 > p.k.lo || key < p.k.S)) {
                const int entry = key / a.kv.page_size, row = key - entry * a.kv.page_size;
                const int page = page_of(a.kv, a.seq, p.b, entry);
                if (page >= 0) {
                    off = page * a.kv.page_stride + row * a.kv.row_stride;
                    scale = (int64_t)page * a.kv.Hkv * a.kv.page_size + row;
                }
            }
        }
        left = 16;
    }
    // Ask for the next unit, if there is one; one group of copies either way.
    __device__ __forceinline__ void issue(const DecodeArgs &d, uint32_t ring, int warp, int lane) {
        const AttnArgs &a = d.a;
        while (more && u >= end) {
            p.next(d);
            more = p.at < x1;
            if (more) piece(warp);
        }
        if (more) {
            if (left == 0) pages(d, lane);
            constexpr int CH = C::kRow / 16, RP = 32 / CH;  // chunks a row, rows a pass
            const int h = p.item / d.groups, key = p.key(u), from = 2 * (16 - left);
            const int64_t head = h * a.kv.head_stride;
            const uint32_t st = ring + slot * C::kStage;
            const int c = lane % CH;
            int64_t at[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) at[i] = __shfl_sync(kFullMask, off, from + i);
#pragma unroll
            for (int i = 0; i < kUnit / RP; ++i) {
                const int r = i * RP + lane / CH, j = key + r, half = i * RP / 8;
                const bool live = at[half] >= 0 && j < p.k.L && (j >= p.k.lo || j < p.k.S);
                const int64_t o = live ? at[half] + head + (r & 7) * a.kv.row_stride + 16 * c : 0;
                // the swizzles that make this unit's reads free of bank conflicts
                const int ck = FP8 ? (D == 128 ? c ^ ((r & 1) << 2) : c) : c ^ (r & 7);
                const int cv = FP8 ? (D == 128 ? c ^ (r & 6) : c) : c ^ (r & 7);
                copy16(st + r * C::kRow + 16 * ck, a.kv.k + o, live);
                copy16(st + C::kTile + r * C::kRow + 16 * cv, a.kv.v + o, live);
            }
            if constexpr (FP8) {
                const int64_t s = __shfl_sync(kFullMask, scale, from + (lane & 1));
                const bool live = (lane & 1 ? at[1] : at[0]) >= 0;
                if (lane < 4)
                    copy8(st + 2 * C::kTile + 8 * lane,
                          (lane < 2 ? a.kv.k_scales : a.kv.v_scales) +
                              (live ? s + (int64_t)h * a.kv.page_size : 0),
                          live);
            }
            u += kWarps;
            --left;
        }
        slot = slot + 1 == C::kStages ? 0 : slot + 1;
        copy_commit();
    }
};

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const DecodeArgs d) {
    using C = Cfg<D, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t sums[kWarps];
    __shared__ int64_t found_at;
    __shared__ int found_b;
    __shared__ Part part[kWarps][kHeads];
    const AttnArgs &a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStage;
    float *merge = reinterpret_cast<float *>(smem + C::kRing);
    int4 *record = reinterpret_cast<int4 *>(d.ws);
    Part *parts = reinterpret_cast<Part *>(d.ws + ws_parts(gridDim.x));
    float *out_sums = reinterpret_cast<float *>(d.ws + ws_sums(gridDim.x));
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the block's run of the list ----
    int64_t total = 0;
    for (int b0 = 0; b0 < a.seq.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int64_t n = b < a.seq.B ? visible(a, b).n : 0;
#pragma unroll
        for (int s = 16; s; s >>= 1) n += __shfl_xor_sync(kFullMask, n, s);
        total += n;
    }
    if (lane == 0) sums[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += sums[i];
    total *= d.items;
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kLeast);
    const int64_t x0 = blockIdx.x * per, x1 = min(x0 + per, total);
    if (threadIdx.x == 0) record[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (x0 >= x1) return;
    int64_t before = 0;
    for (int b0 = 0;; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int64_t n = b < a.seq.B ? (int64_t)visible(a, b).n * d.items : 0;
        int64_t incl = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, incl, s);
            if (lane >= s) incl += o;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int64_t all = 0, below = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i == warp) below = all;
            all += sums[i];
        }
        incl += before + below;
        if (x0 >= incl - n && x0 < incl) {
            found_b = b;
            found_at = incl - n;
        }
        before += all;
        if (before > x0 || b0 + kThreads >= a.seq.B) break;
    }
    __syncthreads();
    Place p;
    p.b = found_b;
    p.k = visible(a, p.b);
    p.item = (int)((x0 - found_at) / p.k.n);
    p.at = found_at + (int64_t)p.item * p.k.n;

    Loader<D, FP8> load;
    load.p = p;
    load.x0 = x0;
    load.x1 = x1;
    load.slot = 0;
    load.more = true;
    load.piece(warp);
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) load.issue(d, ring, warp, lane);

    const int row = lane >> 2, c = lane & 3;  // of the matrix fragments
    int slot = 0;
    for (; p.at < x1; p.next(d)) {
        const int h = p.item / d.groups, g = p.item - h * d.groups;
        const int q0 = h * d.G + g * kHeads, heads = min(kHeads, d.G - g * kHeads);
        // ---- queries: the rows `row` and `row + 8` of the first factor ----
        uint32_t q[D / 16][4];
        float to_log2[2];  // logits in log2 units, of these rows
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = row + 8 * half;
            const uint16_t *src = a.q + p.b * a.q_stride + (int64_t)(q0 + r) * D;
            to_log2[half] = a.scale * kLog2e;
            if constexpr (!FP8) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[s][half + 2 * i] =
                            r < heads ? (uint32_t)ld_dep(reinterpret_cast<const int32_t *>(src + 16 * s + 8 * i + 2 * c)) : 0u;
            } else {
                // a lane's E4M3 key bytes are 16 neighbours, so the channels that a step
                // takes are 4 s .. 4 s + 3 of each lane's 16; as fp16 next to 2^8 at
                // most, which is exact down to 2^-32 of the row's largest
                uint32_t w[D / 64][8];
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 v = r < heads ? ld_dep_v4(src + 64 * j + 16 * c + 8 * i)
                                                  : make_uint4(0, 0, 0, 0);
                        w[j][4 * i] = v.x;
                        w[j][4 * i + 1] = v.y;
                        w[j][4 * i + 2] = v.z;
                        w[j][4 * i + 3] = v.w;
                    }
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[j][i])), fabsf(bf16_hi(w[j][i]))));
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
                // up = 2^k with amax * up in [2^7, 2^8), within what fp32 has of both
                const int e = min(max((int)(__float_as_uint(amax) >> 23), 8), 254);
                const float up = __uint_as_float((uint32_t)min(254 - e + 7, 254) << 23);
                to_log2[half] *= __uint_as_float((uint32_t)max(e - 7, 0) << 23);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t v = w[s / 4][2 * (s % 4) + i];
                        q[s][half + 2 * i] = pack_half(bf16_lo(v) * up, bf16_hi(v) * up);
                    }
            }
        }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float mv[2] = {-INFINITY, -INFINITY};  // FP8: largest logit with its value's scale
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] = 0.0f;

        const int piece0 = (int)(max(x0, p.at) - p.at), piece1 = (int)min((int64_t)p.k.n, x1 - p.at);
        for (int u = piece0 + warp; u < piece1; u += kWarps) {
            copy_wait<C::kStages - 2>();
            __syncwarp();
            load.issue(d, ring, warp, lane);
            const uint32_t st = ring + slot * C::kStage, sv = st + C::kTile;
            slot = slot + 1 == C::kStages ? 0 : slot + 1;

            // ---- logits of 16 rows and 16 keys ----
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = 0.0f;
            float ev[2][2];  // FP8: log2 of the values' scales, of the lane's four keys
            if constexpr (!FP8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int r = (lane & 7) + ((lane >> 4) << 3), ch = 2 * k + ((lane >> 3) & 1);
                    uint32_t b[4];
                    ldmatrix4<false>(b, st + r * C::kRow + 16 * (ch ^ (r & 7)));
                    mma<false>(s[0], q[k], b[0], b[1]);
                    mma<false>(s[1], q[k], b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const int r = 8 * t + row, ch = 4 * j + c;
                        const uint4 v = lds16(st + r * C::kRow + 16 * (D == 128 ? ch ^ ((r & 1) << 2) : ch));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma<true>(s[t], q[4 * j + i], half_pair(w[i]), half_pair(w[i] >> 16));
                    }
                const uint32_t sc = st + 2 * C::kTile;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t ek, evb;  // two keys' bytes
                    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(ek) : "r"(sc + 8 * t + 2 * c) : "memory");
                    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(evb) : "r"(sc + 16 + 8 * t + 2 * c) : "memory");
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = scale_value((ek >> 8 * i) & 255);
                        s[t][i] *= f;
                        s[t][2 + i] *= f;
                        const uint32_t e = (evb >> 8 * i) & 255;
                        ev[t][i] = e == 255 ? __uint_as_float(0x7fffffffu) : (float)((int)e - 127);
                    }
                }
            }
            const int key = p.key(u);
            const bool whole = key + kUnit <= p.k.L && key >= p.k.lo;
            float top[2] = {m[0], m[1]}, topv[2] = {mv[0], mv[1]};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = key + 8 * t + 2 * c + (i & 1);
                    s[t][i] *= to_log2[i >> 1];
                    if (!whole && !(j < p.k.L && (j >= p.k.lo || j < p.k.S))) s[t][i] = -INFINITY;
                    top[i >> 1] = fmaxf(top[i >> 1], s[t][i]);
                    if constexpr (FP8)
                        topv[i >> 1] = fmaxf(topv[i >> 1], s[t][i] == -INFINITY ? -INFINITY : s[t][i] + ev[t][i & 1]);
                }
            bool grown = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], x));
                    if constexpr (FP8) topv[r] = fmaxf(topv[r], __shfl_xor_sync(kFullMask, topv[r], x));
                }
                grown |= top[r] > m[r] || (FP8 && topv[r] > mv[r]);
            }
            // a row that has seen no key yet subtracts 0 from its -infinities
            float base[2], basev[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                base[r] = top[r] == -INFINITY ? 0.0f : top[r];
                basev[r] = topv[r] == -INFINITY ? 0.0f : topv[r];
            }
            if (__any_sync(kFullMask, grown)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = exp2_fast(m[r] - base[r]);
                    const float fo = FP8 ? exp2_fast(mv[r] - basev[r]) : f;
                    l[r] *= f;
#pragma unroll
                    for (int t = 0; t < D / 8; ++t) {
                        o[t][2 * r] *= fo;
                        o[t][2 * r + 1] *= fo;
                    }
                    m[r] = top[r];
                    mv[r] = topv[r];
                }
            }
            // ---- probabilities, and o += p v ----
            float w[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = exp2_fast(s[t][i] - base[i >> 1]);
                    l[i >> 1] += e;
                    // the value's scale belongs to the weight: next to 2^10 at most, fp16
                    w[t][i] = !FP8 ? e
                              : s[t][i] == -INFINITY ? 0.0f
                                                     : exp2_fast(s[t][i] + ev[t][i & 1] - basev[i >> 1] + 10.0f);
                }
            if constexpr (!FP8) {
                // p as two bf16, its own and what that leaves: one would be off by 2^-9 in
                // every probability, and the products are not what bounds the kernel
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = w[i >> 1][2 * (i & 1)], y = w[i >> 1][2 * (i & 1) + 1];
                    hi[i] = pack_bf16(x, y);
                    lo[i] = pack_bf16(x - bf16_lo(hi[i]), y - bf16_hi(hi[i]));
                }
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    const int r = lane & 15, ch = 2 * t + (lane >> 4);
                    uint32_t b[4];
                    ldmatrix4<true>(b, sv + r * C::kRow + 16 * (ch ^ (r & 7)));
                    mma<false>(o[2 * t], hi, b[0], b[1]);
                    mma<false>(o[2 * t + 1], hi, b[2], b[3]);
                    mma<false>(o[2 * t], lo, b[0], b[1]);
                    mma<false>(o[2 * t + 1], lo, b[2], b[3]);
                }
            } else {
                uint32_t pw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pw[i] = pack_half(w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1]);
                // the lane's four keys, D / 8 channels from D / 8 * row on: column `row` of
                // the product's tile t is channel D / 8 * row + t
                uint32_t v[4][D / 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 2 * c + (i & 1) + 8 * (i >> 1);
                    if constexpr (D == 128) {
                        const uint4 x = lds16(sv + r * C::kRow + 16 * (row ^ (r & 6)));
                        v[i][0] = x.x;
                        v[i][1] = x.y;
                        v[i][2] = x.z;
                        v[i][3] = x.w;
                    } else {
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                     : "=r"(v[i][0]), "=r"(v[i][1])
                                     : "r"(sv + r * C::kRow + 8 * row)
                                     : "memory");
                    }
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint32_t a0 = __byte_perm(v[0][x], v[1][x], 0x5140), a1 = __byte_perm(v[0][x], v[1][x], 0x7362);
                    const uint32_t b0 = __byte_perm(v[2][x], v[3][x], 0x5140), b1 = __byte_perm(v[2][x], v[3][x], 0x7362);
                    mma<true>(o[4 * x], pw, half_pair(a0), half_pair(b0));
                    mma<true>(o[4 * x + 1], pw, half_pair(a0 >> 16), half_pair(b0 >> 16));
                    mma<true>(o[4 * x + 2], pw, half_pair(a1), half_pair(b1));
                    mma<true>(o[4 * x + 3], pw, half_pair(a1 >> 16), half_pair(b1 >> 16));
                }
            }
        }

        // ---- the warps' sums together, eight rows at a time ----
        const bool starts = p.at >= x0, ends = p.at + p.k.n <= x1;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(kFullMask, l[r], 1);
            l[r] += __shfl_xor_sync(kFullMask, l[r], 2);
            if (c == 0) part[warp][row + 8 * r] = {m[r], l[r]};
            if constexpr (FP8) {  // from the scaled weights' unit to the probabilities'
                const float f = m[r] == -INFINITY ? 0.0f : exp2_fast(mv[r] - m[r] - 10.0f);
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    o[t][2 * r] *= f;
                    o[t][2 * r + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (8 * half >= heads) break;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                // FP8: the fragment's column 2 c + i of tile t is channel D/8 (2 c + i) + t
                float *at = merge + (warp * 8 + row) * D;
                if constexpr (!FP8) {
                    *reinterpret_cast<float2 *>(at + ((8 * t + 2 * c) ^ (8 * row & (D - 1)))) =
                        make_float2(o[t][2 * half], o[t][2 * half + 1]);
                } else {
                    at[((D / 8 * 2 * c + t) ^ (8 * row & (D - 1)))] = o[t][2 * half];
                    at[((D / 8 * (2 * c + 1) + t) ^ (8 * row & (D - 1)))] = o[t][2 * half + 1];
                }
            }
            __syncthreads();
            const int r = 8 * half + warp;  // this warp's row
            if (r < heads) {
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) top = fmaxf(top, part[i][r].m);
                const float base = top == -INFINITY ? 0.0f : top;
                float acc[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float f = exp2_fast(part[i][r].m - base);
                    sum += part[i][r].l * f;
                    const float *at = merge + (i * 8 + warp) * D + ((D / 32 * lane) ^ (8 * warp & (D - 1)));
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) acc[x] += at[x] * f;
                }
                if (starts && ends) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    const int64_t to = (int64_t)p.b * a.Hq + q0 + r;
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + to * D + D / 32 * lane);
#pragma unroll
                    for (int x = 0; x < D / 32; x += 2) dst[x / 2] = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
                    if (a.lse && lane == 0) a.lse[to] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
                } else {
                    const size_t to = (size_t)(2 * blockIdx.x + starts) * kHeads + r;
                    float *dst = out_sums + to * D + D / 32 * lane;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) dst[x] = acc[x];
                    if (lane == 0) parts[to] = {top, sum};
                }
            }
            __syncthreads();
        }
        if (starts && !ends && threadIdx.x == 0)  // the block where a shared head begins
            record[blockIdx.x] = make_int4(p.b, q0, heads, (int)((p.at + p.k.n - 1) / per) - (int)blockIdx.x);
    }
    copy_wait<0>();
}

// A shared head's sums, from the block where it begins on: one warp a row.
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const DecodeArgs d, int blocks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 *record = reinterpret_cast<const int4 *>(d.ws);
    const Part *parts = reinterpret_cast<const Part *>(d.ws + ws_parts(blocks));
    const float *sums = reinterpret_cast<const float *>(d.ws + ws_sums(blocks));
    const int c0 = blockIdx.x >> 1, r = warp + 8 * (blockIdx.x & 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint4 rec = ld_dep_v4(record + c0);
    const int n = (int)rec.w;  // blocks after the first
    if (n == 0 || r >= (int)rec.z) return;
    auto at = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0)) * kHeads + r; };
    float top = -INFINITY;
    for (int i = lane; i <= n; i += 32) top = fmaxf(top, ld_dep(&parts[at(i)].m));
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) acc[x] = 0.0f;
#pragma unroll 4
    for (int i = 0; i <= n; ++i) {
        const float f = exp2_fast(ld_dep(&parts[at(i)].m) - base);
        sum += ld_dep(&parts[at(i)].l) * f;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) acc[x] += ld_dep(sums + at(i) * D + D / 32 * lane + x) * f;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t to = (int64_t)rec.x * d.a.Hq + rec.y + r;
    uint32_t *dst = reinterpret_cast<uint32_t *>(d.a.out + to * D + D / 32 * lane);
#pragma unroll
    for (int x = 0; x < D / 32; x += 2) dst[x / 2] = pack_bf16(acc[x] * inv, acc[x + 1] * inv);
    if (d.a.lse && lane == 0) d.a.lse[to] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

template <int D, bool FP8>
cudaError_t launch(const DecodeArgs &d, cudaStream_t stream) {
    const int blocks = sm_count();
    const cudaError_t err = launch_large<decode_kernel<D, FP8>>(blocks, kThreads, Cfg<D, FP8>::kSmem, stream, d);
    if (err != cudaSuccess) return err;
    return launch_kernel(join_kernel<D>, 2 * blocks, kThreads, 0, stream, true, d, blocks);
}

}  // namespace

size_t attn_decode_workspace(int, int, int, int D) { return ws_bytes(sm_count(), D); }

cudaError_t launch_attn_decode(const AttnArgs &a, void *workspace, cudaStream_t stream) {
    DecodeArgs d = {};
    d.a = a;
    d.G = a.Hq / a.kv.Hkv;
    d.groups = (d.G + kHeads - 1) / kHeads;
    d.items = a.kv.Hkv * d.groups;
    d.ws = static_cast<uint8_t *>(workspace);
    const bool fp8 = a.kv.k_scales != nullptr;
    if (a.kv.D == 64) return fp8 ? launch<64, true>(d, stream) : launch<64, false>(d, stream);
    return fp8 ? launch<128, true>(d, stream) : launch<128, false>(d, stream);
}

}  // namespace ep
