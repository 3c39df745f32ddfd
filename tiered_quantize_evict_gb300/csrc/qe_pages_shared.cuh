// qe_pages_shared.cuh -- the line of blocks of an attention whose sequences share prefixes in groups.
//
// A tile is up to NH T packed tokens of a group, of one sequence or many, and one KV head.  Its keys are the prefix, then what each of
// the tile's sequences has of its own (up to what its last token in the tile sees, in whole pieces of pages), one after the other:
// short ends of several sequences fill a block together.  A row sees the prefix and a range of the rest.
//
// With two halves the keys are two streams: the prefix and what the first half's sequences have, and what the second half's have.  The
// blocks behind the prefix come from both in turn, and each is for its half alone: the other half's softmax and products are at the
// block before and the one behind meanwhile (a block that one half is at and the other waits for took 2.0 us, where reading it takes 1.4).
//
// The line is, for each KV head, the groups' tiles in order, each as long as its blocks and what it costs besides.
#pragma once
#include "qe_pages_attn.cuh"

namespace qe {

// Where groups and sequences are looked up: in the call's arrays (row and len NULL), or in a copy of what they come to.
struct PaSource {
  const int *start, *prefix, *q_start, *row, *len;
  __device__ __forceinline__ int row_of(const PaParams& p, int s) const { return row ? row[s] : (p.c.rows ? p.c.rows[s] : s); }
  __device__ __forceinline__ int len_of(const PaParams& p, int s, int r) const { return len ? len[s] : row_len(p.pg, p.t, r, false); }
};
__device__ __forceinline__ PaSource pa_arrays(const PaParams& p) { return PaSource{p.gr.start, p.gr.prefix, p.c.q_start, nullptr, nullptr}; }

// A group: its sequences [s0, s1), packed tokens [q0, q1), tokens of the prefix (whole pages) and the row that has them.
struct PaGroup {
  int s0, s1, q0, q1, prefix, row;
};
__device__ __forceinline__ PaGroup pa_group(const PaParams& p, const PaSource& from, int g) {
  PaGroup r;
  r.s0 = min(max(from.start[g], 0), p.c.n);
  r.s1 = min(max(from.start[g + 1], r.s0), p.c.n);
  const int want = from.prefix[g];
  r.q0 = min(max(from.q_start[r.s0], 0), p.c.total);
  r.q1 = min(max(from.q_start[r.s1], r.q0), p.c.total);
  const bool some = r.s0 < r.s1;
  r.row = some ? from.row_of(p, r.s0) : -1;
  r.prefix = min(max(want, 0), some ? from.len_of(p, r.s0, r.row) : 0) & -p.pg.S;
  return r;
}

// A sequence of a group: packed tokens [a, a + m), row, length.
struct PaMember {
  int a, m, row, len;
  // own keys that the tokens before packed token `end` see together
  __device__ __forceinline__ int own(const PaParams& p, const PaGroup& g, int end) const {
    return max(0, (p.causal ? len - m + min(m, end - a) : len) - g.prefix);
  }
};
__device__ __forceinline__ PaMember pa_member(const PaParams& p, const PaSource& from, const PaGroup& g, int s) {
  PaMember r;
  const int a = from.q_start[s], b = from.q_start[s + 1];
  r.row = from.row_of(p, s);
  r.len = from.len_of(p, s, r.row);
  r.a = min(max(a, g.q0), g.q1);
  r.m = min(max(b, r.a), g.q1) - r.a;
  return r;
}

// 32 sequences from `base` on, one to a lane, with the place of their own keys in the stream of the packed tokens [t0, t1) (before: the
// keys that come before them).
struct PaBatch {
  PaMember s;
  int at, end;         // own keys of the stream [at, end), in whole pieces; empty where the sequence has none of the tokens
  bool more;           // sequences behind may have some
  __device__ __forceinline__ void load(const PaParams& p, const PaSource& from, const PaGroup& g, int base, int t0, int t1, int before) {
    const int lane = threadIdx.x & 31, i = base + lane, piece = pa_piece(p);
    s = PaMember{t1, 0, -1, 0};
    int own = 0;
    if (i < g.s1) {
      s = pa_member(p, from, g, i);
      if (max(s.a, t0) < min(s.a + s.m, t1)) own = (s.own(p, g, t1) + piece - 1) & -piece;
    }
    int y = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int z = __shfl_up_sync(~0u, y, k);
      if (lane >= k) y += z;
    }
    end = before + y;
    at = end - own;
    more = base + 32 < g.s1 && !__any_sync(~0u, i < g.s1 && s.a >= t1);
  }
  __device__ __forceinline__ int total() const { return __shfl_sync(~0u, end, 31); }
  // the lane whose member's x is the first above v, where x does not decrease over the lanes (32: none)
  static __device__ __forceinline__ int first_above(int x, int v) {
    int n = 0;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1)
      if (__shfl_sync(~0u, x, n + k - 1) <= v) n += k;
    return n + (__shfl_sync(~0u, x, min(n, 31)) <= v ? 1 : 0);
  }
};

// a stream's sequences begin at `first`, its keys behind `before` others, and it ends with packed token t1's
struct PaStream {
  int first, t0, t1, before;
};

// A tile's keys: what a walk and the place that it starts at have in common.
struct PaSharedTile {
  PaGroup gr;
  int first, mid;       // sequences of the tile's first token, and of its second half's
  int t0, t1;           // the tile's packed tokens
  int np, na, nz;       // blocks with keys of the prefix; those and the rest of the first stream; the second stream's
};

// Places in shared memory: where the CTA's walk starts, where it ends, and with one half the tiles behind the first, as far as they are
// kept: what a warp would have to gather of the arrays again, between two tiles (64 groups of 8 sequences 148 -> 142 us; the softmax of
// two halves has no registers for it: 64 sequences 70 -> 88).
constexpr int PA_KEPT = 3;
template <int NH>
constexpr int PA_PLACES = NH == 1 ? 3 + PA_KEPT : 2;
struct PaSharedPlace {
  int h, g, j, b;      // KV head (that of the end of the line: their number; of a tile that is not kept: -1), group, tile of the group, block
  PaSharedTile tile;   // what a walk from here on starts with
  __device__ __forceinline__ bool before(const PaSharedPlace& o) const {
    return h != o.h ? h < o.h : (g != o.g ? g < o.g : (j != o.j ? j < o.j : b < o.b));
  }
};

// A walk from one place to another, tile by tile, by a whole warp.
template <int NH>
struct PaSharedCursor : PaSharedTile {
  int h, g, j, b, nb;   // the place; blocks of the tile
  int eh, eg, ej, eb;   // where the walk ends
  const PaSharedPlace* kept;
  __device__ __forceinline__ PaStream stream(const PaParams& p, int z) const {
    if (NH == 1) return PaStream{first, t0, t1, gr.prefix};
    return z ? PaStream{mid, t0 + p.T, t1, np * PA_BN} : PaStream{first, t0, min(t1, t0 + p.T), gr.prefix};
  }
  __device__ __forceinline__ void tile(const PaParams& p, const PaSource& from) {
    t0 = gr.q0 + j * NH * p.T;
    t1 = min(gr.q1, t0 + NH * p.T);
    np = (gr.prefix + PA_BN - 1) >> 7;
    nz = 0;
    first = mid = gr.s0 + pages_count_below(from.q_start + gr.s0 + 1, gr.s1 - gr.s0, t0);
    // (every half has a block, so that rows without keys are written too)
    na = max(1, (keys(p, from, gr.s1, stream(p, 0)) + PA_BN - 1) >> 7);
    if (second_half(p)) {
      mid = gr.s0 + pages_count_below(from.q_start + gr.s0 + 1, gr.s1 - gr.s0, t0 + p.T);
      nz = max(np == 0 ? 1 : 0, ((keys(p, from, gr.s1, stream(p, 1)) + PA_BN - 1) >> 7) - np);
    }
    nb = na + nz;
  }
  // keys of a stream before those of sequence `until`
  __device__ __forceinline__ int keys(const PaParams& p, const PaSource& from, int until, const PaStream& z) const {
    PaBatch x;
    int at = z.before;
#pragma unroll 1
    for (int base = z.first; base < until; base += 32) {
      x.load(p, from, gr, base, z.t0, z.t1, at);
      if (until - base < 32) return __shfl_sync(~0u, x.at, until - base);
      at = x.total();
      if (!x.more) break;
    }
    return at;
  }
  // block i of the tile: its stream and first key there (prefix blocks are the first stream's, and of both halves)
  __device__ __forceinline__ int block(int i, int& at) const {
    if (NH == 1 || i < np) {
      at = i * PA_BN;
      return 0;
    }
    const int x = i - np, a = na - np, both = min(a, nz), z = x < 2 * both ? x & 1 : a < nz;
    at = (np + (x < 2 * both ? x >> 1 : x - both)) * PA_BN;
    return z;
  }
  __device__ __forceinline__ bool is_for(int half, int i) const {
    int at;
    return NH == 1 || i < np || block(i, at) == half;
  }
  // how many of the blocks before block i are for a half
  __device__ __forceinline__ int blocks_for(int half, int i) const {
    if (NH == 1 || i <= np) return i;
    const int x = i - np, a = na - np, both = min(a, nz);
    return np + (x < 2 * both ? (x + 1 - half) >> 1 : both + ((a < nz) == half ? x - 2 * both : 0));
  }
  __device__ __forceinline__ int count_for(int half) const { return blocks_for(half, b + count()) - blocks_for(half, b); }
  __device__ __forceinline__ void set(const PaParams& p, const PaSharedPlace* pl) {
    h = pl[0].h;
    g = pl[0].g;
    j = pl[0].j;
    b = pl[0].b;
    eh = pl[1].h;
    eg = pl[1].g;
    ej = pl[1].j;
    eb = pl[1].b;
    kept = pl + 2;
    static_cast<PaSharedTile&>(*this) = pl[0].tile;
    nb = na + nz;
  }
  __device__ __forceinline__ bool last_tile() const { return h == eh && g == eg && j == ej; }
  __device__ __forceinline__ int count() const { return last_tile() ? eb - b : nb - b; }
  __device__ __forceinline__ void next_tile(const PaParams& p) {
    if (last_tile()) {   // the walk is over
      b = eb;
      return;
    }
    b = 0;
    if (NH == 1 && kept) {
      if (kept->h >= 0) {
        h = kept->h;
        g = kept->g;
        j = kept->j;
        static_cast<PaSharedTile&>(*this) = kept->tile;
        nb = na + nz;
        ++kept;
        return;
      }
      kept = nullptr;
    }
    ++j;
    if ((long long)gr.q0 + (long long)j * NH * p.T >= gr.q1) {
      j = 0;
      ++g;
      while (true) {     // the next group that has tokens
        const int lane = threadIdx.x & 31, x = g + lane;
        unsigned any = 0;
        if (g < p.gr.n) {
          bool some = false;
          if (x < p.gr.n) {
            const int s0 = min(max(p.gr.start[x], 0), p.c.n), s1 = min(max(p.gr.start[x + 1], s0), p.c.n);
            const int q0 = min(max(p.c.q_start[s0], 0), p.c.total);
            some = min(p.c.q_start[s1], p.c.total) > q0;
          }
          any = __ballot_sync(~0u, some);
        }
        if (any) {
          g += __ffs(any) - 1;
          break;
        }
        g += 32;
        if (g >= p.gr.n) {
          g = 0;
          if (++h >= p.pg.H) {   // the end of the line
            nb = 0;
            return;
          }
        }
      }
      gr = pa_group(p, pa_arrays(p), g);
    }
    tile(p, pa_arrays(p));
  }
  __device__ __forceinline__ bool second_half(const PaParams& p) const { return NH == 2 && t0 + p.T < t1; }
  __device__ __forceinline__ int head() const { return h; }
  __device__ __forceinline__ int tok(const PaParams&) const { return t0; }
  __device__ __forceinline__ int tokens(const PaParams&) const { return t1 - t0; }
  __device__ __forceinline__ int shift(const PaParams&) const { return 0; }

  // the range [lo, hi) of a stream's keys behind the prefix that its packed token t (of this lane) sees
  __device__ __forceinline__ void range(const PaParams& p, int half, int t, int& lo, int& hi) const {
    const PaStream z = stream(p, half);
    PaBatch x;
    int at = lo = hi = z.before;
#pragma unroll 1
    for (int base = z.first; base < gr.s1; base += 32) {
      x.load(p, pa_arrays(p), gr, base, z.t0, z.t1, at);
      const int n = PaBatch::first_above(x.s.a + x.s.m, t), from = min(n, 31);
      const int a = __shfl_sync(~0u, x.s.a, from), m = __shfl_sync(~0u, x.s.m, from), len = __shfl_sync(~0u, x.s.len, from), k = __shfl_sync(~0u, x.at, from);
      if (n < 32 && t >= a && t < a + m) {
        lo = k;
        hi = k + max(0, (p.causal ? len - m + (t - a) + 1 : len) - gr.prefix);
      }
      at = x.total();
      if (!x.more) break;
    }
  }
};

// What the warp that copies keys and values knows of a piece of a page: the table's entry, the piece's first token in the page, and how
// many of its tokens are the sequence's where not all of them are (255 else; PA_NO_KEYS: there are no keys here, and no entry).
constexpr int PA_NO_KEYS = 256;
struct PaPiece {
  int entry, tok, valid;
};
template <int NH>
struct PaSharedKeys {
  PaBatch x, y;         // the batch of the stream of the last call, and the other stream's
  int xb, yb;           // their first sequences
  int z, h, g, j;       // which stream x is of; of which tile (h < 0: none yet)
  __device__ __forceinline__ PaSharedKeys() : z(0), h(-1) {}
  // the piece of block i that begins with its key `off` (of this lane); i does not decrease from call to call within a tile
  __device__ __forceinline__ PaPiece at(const PaParams& p, const PaSharedCursor<NH>& c, int i, int off) {
    PaPiece r{-1, 0, PA_NO_KEYS};
    int key = -1, row = -1, len = 0, v;
    const int zi = c.block(i, v);
    v += off;
    if (i < c.np && v < c.gr.prefix) {
      key = v;
      row = c.gr.row;
      len = INT_MAX;
    }
    if (__any_sync(~0u, key < 0)) {
      if (c.h != h || c.g != g || c.j != j) {
        h = c.h;
        g = c.g;
        j = c.j;
        xb = yb = -1;
      }
      if (NH == 2 && zi != z) {
        z = zi;
        const PaBatch t = x;
        x = y;
        y = t;
        const int tb = xb;
        xb = yb;
        yb = tb;
      }
      const PaStream s = c.stream(p, z);
      if (xb < 0) {
        xb = s.first;
        x.load(p, pa_arrays(p), c.gr, xb, s.t0, s.t1, s.before);
      }
      while (true) {
        const int n = PaBatch::first_above(x.end, v), from = min(n, 31);
        const int rw = __shfl_sync(~0u, x.s.row, from), ln = __shfl_sync(~0u, x.s.len, from), a = __shfl_sync(~0u, x.at, from);
        if (key < 0 && n < 32 && v >= a) {
          key = c.gr.prefix + (v - a);
          row = rw;
          len = ln;
        }
        if (!x.more || !__any_sync(~0u, key < 0)) break;
        const int at = x.total();
        xb += 32;
        x.load(p, pa_arrays(p), c.gr, xb, s.t0, s.t1, at);
      }
    }
    if (key >= 0 && key < len) {
      r.entry = p.t.table[(long long)row * p.t.stride + (key >> p.pg.lgS)];
      r.tok = key & (p.pg.S - 1);
      r.valid = len - key < (p.wide ? pa_piece(p) : 8) ? len - key : 255;
    }
    return r;
  }
};

// Reports what a call got wrong, by a warp of each CTA that has nothing else to do: 32 groups and 32 sequences to a CTA, in turn (by the
// first CTA alone, chains of loads for all of them one after the other, it was what bounded calls of many: 8192 sequences in groups of 16
// 392 -> 124 us, 65536 3674 -> 1153).
__device__ __forceinline__ bool pa_checks_shared(const PaParams& p) { return blockIdx.x * 32 < max(p.c.n, p.gr.n); }
static __device__ __noinline__ void pa_check_shared(const PaParams& p) {
  const int first = blockIdx.x * 32 + (threadIdx.x & 31), step = gridDim.x * 32;
  for (int k = first; k < p.gr.n; k += step) {
    const int a = p.gr.start[k], b = p.gr.start[k + 1], want = p.gr.prefix[k];
    bool bad = a < 0 || b < a || b > p.c.n || (k == 0 && a != 0) || (k == p.gr.n - 1 && b != p.c.n);
    if (!bad && a < b) bad = want < 0 || want > row_len(p.pg, p.t, p.c.rows ? p.c.rows[a] : a, false);
    if (bad) pages_report(p.pg, QE_PAGES_ERR_ROW);
  }
  for (int i = first; i < p.c.n; i += step) {
    const SeqInfo s = seq_info(p.pg, p.t, p.c, i, true);
    int lo = 0, hi = p.gr.n;         // the last group that does not begin behind the sequence
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.gr.start[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int whole = max(p.gr.prefix[lo], 0) & -p.pg.S;
    if (s.m > 0 && whole > 0 && whole > (p.causal ? s.len - s.m : s.len)) pages_report(p.pg, QE_PAGES_ERR_ROW);
  }
}

// Every CTA finds its piece, as pa_find does: the groups' numbers of tiles, then the tiles, a warp for each, then the two cuts among
// them.  `space` is shared memory for pa_find_ints(NT) numbers.  Where there is a thread for each sequence and group, what the arrays hold
// is read once, side by side, and looked up there.  (Bound by fetching its instructions, once in a launch, and by latency: the same with a
// line of sequences, whose tiles then had to be found, took 10 us for one group of 64.)
constexpr int PA_TILE_INTS = 2 + sizeof(PaSharedTile) / sizeof(int);   // group, tile of the group, the tile
constexpr int pa_find_ints(int nt) { return 6 * nt + 3 + nt * PA_TILE_INTS; }
// a tile counts as so many blocks at most (a row of 2^27 tokens), so that a block's tiles are added up in 32 bits
constexpr int PA_MOST_BLOCKS = 1 << 20;
template <int NH, int NT>
__device__ __noinline__ void pa_find_shared(const PaParams& p, PaSharedPlace* pl, int* s_w, int* space) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tt = NH * p.T, c = blockIdx.x;
  constexpr int W = NT / 32;
  int *start = space, *prefix = start + NT + 1, *q_start = prefix + NT, *row = q_start + NT + 1, *len = row + NT, *s_first = len + NT,
      *s_tile = s_first + NT + 1;
  auto scan = [&](int x, int& total) {   // sum of the threads' before this one
    int y = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int z = __shfl_up_sync(~0u, y, k);
      if (lane >= k) y += z;
    }
    if (lane == 31) s_w[warp] = y;
    __syncthreads();
    int v = lane < W ? s_w[lane] : 0;
    const int before = __reduce_add_sync(~0u, lane < warp ? v : 0);
    total = __reduce_add_sync(~0u, v);
    __syncthreads();
    return before + y - x;
  };
  PaSource from = pa_arrays(p);
  if (p.c.n <= NT && p.gr.n <= NT) {
    if (tid < p.gr.n) {
      start[tid + 1] = from.start[tid + 1];
      prefix[tid] = from.prefix[tid];
    }
    if (tid < p.c.n) {
      q_start[tid + 1] = from.q_start[tid + 1];
      const int r = from.row_of(p, tid);
      row[tid] = r;
      len[tid] = row_len(p.pg, p.t, r, false);
    }
    if (tid == NT - 1) {
      start[0] = from.start[0];
      q_start[0] = from.q_start[0];
    }
    from = PaSource{start, prefix, q_start, row, len};
  }
  if (tid < 2) pl[tid].h = p.pg.H, pl[tid].g = pl[tid].j = pl[tid].b = 0;
  if (NH == 1 && tid == 0) pl[2].h = pl[2 + PA_KEPT].h = -1;
  __syncthreads();
  long long line = 0;
  int pieces = 0, head[2] = {p.pg.H, p.pg.H};
  long long cut[2] = {0, 0};
  // one pass over the tiles where each has a thread; else the line is measured in a first
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long at = 0;
#pragma unroll 1
    for (int gb = 0; gb < p.gr.n; gb += NT) {
      int tiles = 0, all_tiles;
      if (gb + tid < p.gr.n) {
        const PaGroup g = pa_group(p, from, gb + tid);
        tiles = (g.q1 - g.q0 + tt - 1) / tt;
      }
      const int mine = scan(tiles, all_tiles);
      s_first[tid + 1] = mine + tiles;
      if (tid == 0) s_first[0] = 0;
      __syncthreads();
#pragma unroll 1
      for (int xb = 0; xb < all_tiles; xb += NT) {
#pragma unroll 1
        for (int x = xb + warp; x < min(all_tiles, xb + NT); x += W) {
          // (bounded: groups that overlap, which is an error, could have more tiles than 32 bits count)
          const int k = min(pages_count_below(s_first + 1, NT, x), min(NT, p.gr.n - gb) - 1);
          PaSharedCursor<NH> cur;
          cur.gr = pa_group(p, from, gb + k);
          cur.j = min(max(x - s_first[k], 0), max(cur.gr.q1 - cur.gr.q0 - 1, 0) / tt);
          cur.tile(p, from);
          if (lane == 0) {
            int* to = s_tile + (x - xb) * PA_TILE_INTS;
            to[0] = gb + k;
            to[1] = cur.j;
            *reinterpret_cast<PaSharedTile*>(to + 2) = cur;
          }
        }
        __syncthreads();
        const int* info = s_tile + tid * PA_TILE_INTS;
        const PaSharedTile* t = reinterpret_cast<const PaSharedTile*>(info + 2);
        const int nb = xb + tid < all_tiles ? min(t->na + t->nz, PA_MOST_BLOCKS) : 0;
        int sum;
        const int len = nb > 0 ? PA_TILE_COST + nb : 0, before = scan(len, sum);
        const bool once = p.gr.n <= NT && all_tiles <= NT;
        if (pass == 0 && once) line = sum;
        if ((pass == 0 && once) || (pass == 1 && pieces == 0)) {   // the line is known: the cuts
          const long long all = line * p.pg.H, most = all / PA_LEAST;
          pieces = most < 1 ? 1 : (most > gridDim.x ? (int)gridDim.x : (int)most);
          if (c < pieces && all > 0) {
            const long long each = div_ll(all, pieces);
            const int over = (int)(all - each * pieces);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const long long to = each * (c + k) + over * (c + k) / pieces;
              head[k] = (int)div_ll(to, line);
              cut[k] = to - head[k] * line;
            }
          }
        }
        if (once || pass == 1) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (head[k] < p.pg.H && cut[k] >= at + before && cut[k] < at + before + len) {
              // a cut in what the tile costs besides, or in a short tile, is one before the tile
              const int rem = (int)(cut[k] - at) - before - PA_TILE_COST, b = nb <= PA_WHOLE ? 0 : max(0, rem);
              pl[k].h = head[k];
              pl[k].g = info[0];
              pl[k].j = info[1];
              pl[k].b = b;
              pl[k].tile = *t;
              if (NH == 1 && k == 0) s_w[0] = tid;
              if (k == 0) p.rec[c] = PaRec{(long long)head[0] * p.c.total + t->t0, b, t->t0, t->t1 - t->t0, head[0], pieces};
            }
        }
        at += sum;
        __syncthreads();   // (s_tile is read)
        if (NH == 1 && once && head[0] < p.pg.H && tid < PA_KEPT * PA_TILE_INTS) {   // the tiles behind the first, behind the last the next head's
          const int e = tid / PA_TILE_INTS, i = tid - e * PA_TILE_INTS, x = s_w[0] + 1 + e, up = x / all_tiles;
          const int h = head[0] + up < p.pg.H ? head[0] + up : -1, v = s_tile[(x - up * all_tiles) * PA_TILE_INTS + i];
          if (i == 0) pl[2 + e].h = h, pl[2 + e].g = v;
          else if (i == 1) pl[2 + e].j = v;
          else reinterpret_cast<int*>(&pl[2 + e].tile)[i - 2] = v;
        }
        if (once) pass = 2;
      }
      if (all_tiles == 0 && p.gr.n <= NT) pass = 2;
    }
    line = pass == 0 ? at : line;
    if (pass == 0 && line == 0) break;
  }
  if (tid == 0 && (line == 0 || c >= pieces)) p.rec[c] = PaRec{-1, 0, 0, 0, 0, 0};
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (copies go where `space` is)
  __syncthreads();
}

}  // namespace qe
