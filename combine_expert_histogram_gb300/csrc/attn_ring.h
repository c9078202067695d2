// How a warp of the prompts' products goes through the ring of key and value tiles, for
// the kernel and for a model of its barriers on the host.
//
// The ring's places are the keys and values of a piece's tiles in order: keys of tile 0, values of tile 0,
// keys of tile 1, ...  A barrier tells its phases by parity alone, so a wait for one is
// sound only if the phase before it is known to be over and the next one cannot be
// over yet.  Both hold if each warp waits for every place in order, and a place is taken
// again only after each warp has handed it back.  A piece of at most one row tile has
// its even tiles in one half, its odd ones in the other; between its own places a half's warp also
// waits for the other half's and hands them back unread (or takes its turn behind the other warp,
// which has waited for them).
#pragma once

#ifdef __CUDACC__
#define EP_RING_FN __host__ __device__ constexpr
#else
#define EP_RING_FN constexpr
#endif

namespace ep {

// Tiles of a piece of nt that warp t multiplies.
EP_RING_FN int ring_tiles(bool halves, int t, int nt) { return halves ? (nt + 1 - t) / 2 : nt; }
// Places of the other half between the values of warp t's tile n - 1 (the piece's begin, for n = 0) and
// the keys of its tile n.
EP_RING_FN int ring_others_before(bool halves, int t, int n) { return halves ? (n > 0 ? 2 : 2 * t) : 0; }
// Those behind its last tile (all of them, if it has none).
EP_RING_FN int ring_others_after(bool halves, int t, int nt) { return halves && nt > 0 && (nt & 1) == t ? 2 : 0; }

}  // namespace ep

#undef EP_RING_FN
