// qe_pages_walk.cuh -- what the attention kernels ask of a mode (PaMode): the walk over its line of tiles, where a tile's keys lie in
// the cache, which of them a row sees, and which rows of a block of values nobody sees.
#pragma once
#include "qe_pages_shared.cuh"

namespace qe {

// Where the keys of a row's tiles lie: a place for each, or one after the gap that a window leaves.
template <int NH, int MODE>
struct PaRowKeys {
  // the piece of block i that begins with its key `off` (of this lane)
  __device__ __forceinline__ PaPiece at(const PaParams& p, const PaCursor<NH, MODE>& c, int i, int off) const {
    const int v = i * PA_BN + off, key = MODE == PA_WINDOW && v >= p.sa ? v + c.shift(p) : v;
    const bool some = key < c.q.s.len;
    return PaPiece{some ? p.t.table[(long long)c.q.s.row * p.t.stride + (key >> p.pg.lgS)] : -1, key & (p.pg.S - 1), some ? 255 : PA_NO_KEYS};
  }
};

template <int NH, int MODE>
struct PaWalk {
  using Cursor = PaCursor<NH, MODE>;
  using Place = PaPlace;
  static constexpr int PLACES = 2;
  using Keys = PaRowKeys<NH, MODE>;
  // finds the CTA's piece of the line; false where it has none
  template <int NT>
  static __device__ __forceinline__ bool find(const PaParams& p, Place* pl, long long* s_w, int*) {
    pa_find<NH, NT, MODE>(p, pl, s_w);
    // (two cuts that fall into the same place leave an empty piece)
    return pl[0].i < p.c.n && (pl[0].i != pl[1].i || pl[0].h != pl[1].h || pl[0].j != pl[1].j || pl[0].b != pl[1].b);
  }
};
template <int NH>
struct PaWalk<NH, PA_SHARED> {
  using Cursor = PaSharedCursor<NH>;
  using Place = PaSharedPlace;
  static constexpr int PLACES = PA_PLACES<NH>;
  using Keys = PaSharedKeys<NH>;
  template <int NT>
  static __device__ __forceinline__ bool find(const PaParams& p, Place* pl, long long* s_w, int* space) {
    pa_find_shared<NH, NT>(p, pl, reinterpret_cast<int*>(s_w), space);
    return pl[0].before(pl[1]);
  }
};

// What a warp's lane copies of each block: a piece of a page, in a wide copy all its channels, else 64 of them.
template <int CB>
struct PaCopy {
  int rows, piece, cb;     // tokens; which of the block's pieces, and column block
  int pieces;              // of a block
  bool mine;
  __device__ __forceinline__ PaCopy(const PaParams& p) {
    const int lane = threadIdx.x & 31, lg = p.wide ? min(p.pg.lgS, 7) : 3;
    rows = 1 << lg;
    pieces = PA_BN >> lg;
    piece = lane & (pieces - 1);
    cb = lane >> (7 - lg);
    mine = cb < (p.wide ? 1 : CB);
  }
  // entry: the page, or any other number for zeros
  __device__ __forceinline__ void send(const PaParams& p, const CUtensorMap* map, unsigned slot, bool there, int page, int head, int tok, unsigned bar) const {
    const unsigned to = slot + piece * rows * 128 * CB + cb * PA_CELL;
    if (p.wide) pa_tma5(to, map, 0, 0, tok >> 3, there ? page * p.of_page + head * p.of_head : p.all, bar);   // (out of the pool: zeros)
    else pa_tma5(to, map, cb, tok, head, there ? page : p.pg.P, bar);
  }
};
// a token's row in a slot, in bytes; its channels from 64 on are PA_CELL further
template <int CB>
__device__ __forceinline__ unsigned pa_slot_row(int r) {
  return (r >> 3) * (CB * PA_CELL) + (r & 7) * 128;
}

// How many rows of each of a slot's pieces hold values (shared prefixes: pieces of many sequences end where they like).
template <int MODE, int SLOTS>
struct PaValid {
  __device__ __forceinline__ bool none(int, int, const PaParams&) const { return false; }
};
template <int SLOTS>
struct PaValid<PA_SHARED, SLOTS> {
  uint8_t rows[SLOTS][16];
  __device__ __forceinline__ void set(int slot, int piece, int n) { rows[slot][piece] = (uint8_t)n; }
  __device__ __forceinline__ bool none(int slot, int r, const PaParams& p) const {
    const int lg = p.wide ? min(p.pg.lgS, 7) : 3;
    return (r & ((1 << lg) - 1)) >= rows[slot][r >> lg];
  }
};

// Which keys the row of a softmax thread of qe_pages_halves.cuh sees, counted from key `from` of the tile on: those below vis that are
// below `open` or from `low` on.  all_vis, all_low: the strictest of the warp's rows.  A lane without a row computes whatever it
// finds, and nobody reads it.
template <int NH, int MODE>
struct PaSight {
  int vis, low, open, all_vis, all_low, end, gap;   // end: values from here on are nobody's; gap: as are those of [open, gap)
  int mine0, mine1;                                 // shared: the warp's rows see own keys of [mine0, mine1) of their stream
  __device__ __forceinline__ PaSight(const PaParams& p, const typename PaWalk<NH, MODE>::Cursor& c, int half, int t, bool live, bool any_live, int from) {
    constexpr int FAR = 1 << 30;
    open = low = gap = all_low = -FAR;
    if constexpr (MODE == PA_SHARED) {
      open = c.gr.prefix - from;
      vis = FAR;
      if (any_live) {
        int lo, hi;
        c.range(p, half, c.t0 + t, lo, hi);
        if (live) {
          vis = hi - from;
          low = lo - from;
        }
        mine0 = __reduce_min_sync(~0u, live ? lo : FAR);
        mine1 = __reduce_max_sync(~0u, live ? hi : -FAR);
      }
      end = open;   // (own keys: PaValid)
    } else {
      const int back = MODE == PA_WINDOW ? c.shift(p) + from : from, first = max(c.q.s.len - c.q.s.m + c.j * NH * p.T + 1 - back, -FAR);
      vis = !live ? FAR : (p.causal ? first + t : c.q.s.len - back);
      all_vis = __reduce_min_sync(~0u, vis);
      end = c.q.s.len - back;
      if constexpr (MODE == PA_WINDOW) {
        open = p.win.sinks - from;
        gap = first - p.win.window;
        if (live) low = vis - p.win.window;
        all_low = __reduce_max_sync(~0u, low);
      }
    }
  }
  __device__ __forceinline__ bool strange(int at) const { return at + PA_BN > end || (MODE == PA_WINDOW && at < gap && at + PA_BN > open); }
  __device__ __forceinline__ bool none(int key) const { return key >= end || (MODE == PA_WINDOW && key >= open && key < gap); }
  // whether some row of the warp may not see some of the 64 keys from `at` on
  __device__ __forceinline__ bool partly(int at) const {
    if constexpr (MODE == PA_SHARED) return at + 64 > open;
    return at + 64 > all_vis || (MODE == PA_WINDOW && at < all_low && at + 64 > open);
  }
  // whether no row of the warp sees any key of the block from `at` on (`back`: how far this thread's half of it is behind its first key)
  __device__ __forceinline__ bool nothing(int at, int back) const {
    return MODE == PA_SHARED && at >= open + back && (at + PA_BN <= mine0 || at >= mine1);
  }
  // -inf in the place of the logits that the row does not see, whatever lies there
  __device__ __forceinline__ void mask(int at, unsigned (&s)[64]) const {
    const int v = vis - at;
    if constexpr (MODE == PA_PLAIN) {
#pragma unroll
      for (int c = 0; c < 64; ++c)
        if (c >= v) s[c] = 0xFF800000u;
    } else {
      // (a bit for each key: comparisons of two ranges become branches that each row takes its own way, 3300 to 9900 cycles a block)
      const unsigned long long seen = below(v) & (below(open - at) | ~below(low - at));
      const unsigned w[2] = {(unsigned)seen, (unsigned)(seen >> 32)};
#pragma unroll
      for (int c = 0; c < 64; ++c) s[c] = w[c >> 5] & (1u << (c & 31)) ? s[c] : 0xFF800000u;
    }
  }
  static __device__ __forceinline__ unsigned long long below(int n) {   // bits [0, n)
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
  }
};

// The same for a key of qe_pages_few.cuh and the tile's (up to N) rows: row c is of token c / G.
template <int N, int MODE>
struct PaFewSight {
  int off, every, len;      // the tile's first token sees the keys up to `off` (but for the gap); all rows see those below `every`
  int sinks, gap, all_gap;  // window: nobody sees [sinks, gap), some row not [sinks, all_gap)
  int lo[MODE == PA_SHARED ? N : 1], hi[MODE == PA_SHARED ? N : 1];
  __device__ __forceinline__ PaFewSight(const PaParams& p, const typename PaWalk<1, MODE>::Cursor& c) {
    if constexpr (MODE == PA_SHARED) {
      every = len = c.gr.prefix;
      const int t = threadIdx.x & 31;
      int a, b;
      c.range(p, 0, c.t0 + t, a, b);
      const int have = c.tokens(p);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int tok = i / p.G;
        const int x = __shfl_sync(~0u, a, tok), y = __shfl_sync(~0u, b, tok);
        lo[i] = tok < have ? x : 0;
        hi[i] = tok < have ? y : 1 << 30;
      }
    } else {
      const int shift = c.shift(p);
      len = c.q.s.len - shift;
      off = c.q.s.len - c.q.s.m + c.j * p.T - shift;
      every = p.causal ? off + 1 : len;
      if constexpr (MODE == PA_WINDOW) {
        sinks = p.win.sinks;
        gap = off + 1 - p.win.window;
        all_gap = gap + p.T - 1;
      }
    }
  }
  __device__ __forceinline__ bool partly(int at) const {   // of the block from key `at` on
    return at + PA_BN > every || (MODE == PA_WINDOW && at < all_gap && at + PA_BN > sinks);
  }
  __device__ __forceinline__ bool strange(int at) const { return at + PA_BN > len || (MODE == PA_WINDOW && at < gap && at + PA_BN > sinks); }
  __device__ __forceinline__ bool none(int key) const { return key >= len || (MODE == PA_WINDOW && key >= sinks && key < gap); }
  __device__ __forceinline__ void mask(const PaParams& p, int key, unsigned (&s)[N]) const {
    if constexpr (MODE == PA_SHARED) {
#pragma unroll
      for (int c = 0; c < N; ++c)
        if ((key >= hi[c]) | ((key >= len) & (key < lo[c]))) s[c] = 0xFF800000u;   // -inf, whatever lies there
    } else {
      // rows [from, to) see this key
      const int from = key >= len ? N : (p.causal ? min(max(key - off, 0), N) * p.G : 0);
      int to = N;
      if constexpr (MODE == PA_WINDOW)
        if (key >= sinks) to = min(max(min(key - off, N) + p.win.window, 0), N) * p.G;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if ((c < from) | (MODE == PA_WINDOW && c >= to)) s[c] = 0xFF800000u;
    }
  }
};

}  // namespace qe
