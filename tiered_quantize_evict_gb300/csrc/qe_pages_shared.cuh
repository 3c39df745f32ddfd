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
// The line is, for each KV head, the groups' tiles in order.  It is measured in keys, sequence by sequence: what a tile costs besides its
// blocks and the prefix count where the tile begins, own keys where they are.  (Only the cuts go by this measure, and every CTA takes it alike; a
// walk counts the tiles' own blocks.)
#pragma once
#include "qe_pages_attn.cuh"

namespace qe {

constexpr int PA_TILE_KEYS = PA_TILE_COST * PA_BN;

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
  __device__ __forceinline__ bool empty() const { return q1 <= q0; }
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

struct PaSharedPlace {
  int h, g, j, b;      // KV head (that of the end of the line: their number), group, tile of the group, block
  PaSharedTile tile;   // what a walk from here on starts with
  int i;               // (while it is being found) sequence,
  long long rem;       // and how far behind its start on a head's line
  __device__ __forceinline__ bool before(const PaSharedPlace& o) const {
    return h != o.h ? h < o.h : (g != o.g ? g < o.g : (j != o.j ? j < o.j : b < o.b));
  }
};

// A walk from one place to another, tile by tile, by a whole warp.
template <int NH>
struct PaSharedCursor : PaSharedTile {
  int h, g, j, b, nb;   // the place; blocks of the tile
  int eh, eg, ej, eb;   // where the walk ends
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

// What the warp that copies keys and values knows of a piece of a page: the table's entry (INT_MIN: no keys here), the piece's first token in
// the page, and how many of its tokens are the sequence's where not all of them are (255 else).
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
    PaPiece r{INT_MIN, 0, 255};
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
      if (len - key < (p.wide ? pa_piece(p) : 8)) r.valid = len - key;
    }
    return r;
  }
};

// Every CTA finds its piece, as pa_find does.  `space` is shared memory for PA_FIND_INTS(NT) numbers: where there is a thread for each
// sequence and group, what the arrays hold is read once, side by side, and looked up there (a call over one group of 64 sequences: the
// piece is known after 4.5 us instead of 9).
constexpr int PA_FIND_INTS(int nt) { return 5 * nt + 2; }
template <int NH, int NT>
__device__ __noinline__ void pa_find_shared(const PaParams& p, PaSharedPlace* pl, long long* s_w, int* space) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tt = NH * p.T, piece = pa_piece(p);
  constexpr int W = NT / 32;
  const int c = blockIdx.x;
  auto scan = [&](long long x, long long& total) {
    long long y = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long z = __shfl_up_sync(~0u, y, k);
      if (lane >= k) y += z;
    }
    if (lane == 31) s_w[warp] = y;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const long long z = s_w[k];
      if (k < warp) before += z;
      all += z;
    }
    total = all;
    __syncthreads();
    return before + y - x;
  };
  PaSource from = pa_arrays(p);
  const bool held = p.c.n <= NT && p.gr.n <= NT;
  if (held) {
    int *start = space, *prefix = start + NT + 1, *q_start = prefix + NT, *row = q_start + NT + 1, *len = row + NT;
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
    __syncthreads();
    from = PaSource{start, prefix, q_start, row, len};
  }
  auto group_of = [&](int i) {   // the last that does not begin behind sequence i
    int lo = 0, hi = p.gr.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (from.start[mid] <= i) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  // A sequence on a head's line: what it has in a tile that began before (part), then the tiles that begin in it
  struct Part {
    PaGroup g;
    PaMember s;
    int own, j, c0, tiles;       // own keys before the chunk's (and half a piece); the tile it begins in; its tokens in a tile that began before; tiles that begin in it
    long long part;
  };
  auto on_line = [&](const PaGroup& g, const PaMember& s) {
    Part r;
    r.g = g;
    r.s = s;
    r.own = max(0, (p.causal ? s.len - s.m : s.len) - g.prefix) + piece / 2;
    const int o = s.a - g.q0;
    r.j = o / tt;
    const int into = o - r.j * tt;
    r.c0 = into > 0 ? min(s.m, tt - into) : 0;
    r.part = r.c0 > 0 ? r.own + (p.causal ? r.c0 : 0) : 0;
    r.tiles = (s.m - r.c0 + tt - 1) / tt;
    r.j += into > 0;
    return r;
  };
  auto tiles_before = [&](const Part& r, int k) {   // of the tiles that begin in the sequence
    long long x = (long long)k * (PA_TILE_KEYS + r.g.prefix + r.own);
    if (p.causal) x += (long long)k * r.c0 + (long long)k * (k + 1) / 2 * tt;
    return x;
  };
  auto length = [&](int i, bool report) {
    if (i >= p.c.n) return 0ll;
    const int gi = group_of(i);
    const PaGroup g = pa_group(p, from, gi);
    if (report) {
      const SeqInfo s = seq_info(p.pg, p.t, p.c, i, true);
      if (s.m > 0 && g.prefix > 0 && g.prefix > (p.causal ? s.len - s.m : s.len)) pages_report(p.pg, QE_PAGES_ERR_ROW);
    }
    if (i < g.s0 || i >= g.s1) return 0ll;   // (of no group)
    const PaMember s = pa_member(p, from, g, i);
    if (s.m == 0) return 0ll;
    const Part r = on_line(g, s);
    if (r.tiles == 0) return r.part;
    return r.part + tiles_before(r, r.tiles - 1) + PA_TILE_KEYS + g.prefix + r.own + (p.causal ? s.m : 0);
  };
  if (c == 0) {
    for (int k = tid; k < p.gr.n; k += NT) {
      const int a = p.gr.start[k], b = p.gr.start[k + 1];
      bool bad = a < 0 || b < a || b > p.c.n || (k == 0 && a != 0) || (k == p.gr.n - 1 && b != p.c.n);
      if (!bad && a < b) {
        const int want = p.gr.prefix[k];
        bad = want < 0 || want > row_len(p.pg, p.t, p.c.rows ? p.c.rows[a] : a, false);
      }
      if (bad) pages_report(p.pg, QE_PAGES_ERR_ROW);
    }
  }
  if (tid < 2) pl[tid].h = p.pg.H, pl[tid].g = pl[tid].j = pl[tid].b = 0, pl[tid].i = -1;
  // one pass where there is a thread for each sequence, else two
  long long line, x = length(tid, c == 0), pre = scan(x, line);
#pragma unroll 1
  for (int base = NT; base < p.c.n; base += NT) {
    long long tot;
    scan(length(base + tid, c == 0), tot);
    line += tot;
  }
  const long long all = line * p.pg.H, most = all / (PA_LEAST * PA_BN);
  const int pieces = most < 1 ? 1 : (most > gridDim.x ? (int)gridDim.x : (int)most);
  if (c < pieces && all > 0) {
    const long long each = div_ll(all, pieces);
    const int over = (int)(all - each * pieces);
    long long cut[2];
    int head[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long to = each * (c + k) + over * (c + k) / pieces;
      head[k] = (int)div_ll(to, line);
      cut[k] = to - head[k] * line;
    }
    long long at = 0;
#pragma unroll 1
    for (int base = 0; base < p.c.n; base += NT) {
      if (p.c.n > NT) {
        long long tot;
        x = length(base + tid, false);
        pre = at + scan(x, tot);
        at += tot;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (head[k] < p.pg.H && cut[k] >= pre && cut[k] < pre + x) {
          pl[k].h = head[k];
          pl[k].i = base + tid;
          pl[k].rem = cut[k] - pre;
        }
    }
  } else if (tid == 0) {
    p.rec[c] = PaRec{-1, 0, 0, 0, 0, 0};
  }
  __syncthreads();
  if (warp < 2 && pl[warp].i >= 0) {
    const int i = pl[warp].i;
    long long rem = pl[warp].rem;
    PaSharedCursor<NH> cur;
    cur.g = group_of(i);
    cur.gr = pa_group(p, from, cur.g);
    const Part r = on_line(cur.gr, pa_member(p, from, cur.gr, i));
    const bool in_part = rem < r.part;
    if (in_part) {
      cur.j = r.j - 1;
    } else {
      rem -= r.part;
      int lo = 0, hi = r.tiles;   // the last tile that begins at or before rem: 32 places a round
      long long before = 0;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, cand = lo + lane * step;
        const long long at = cand < hi ? tiles_before(r, cand) : LLONG_MAX;
        const int top = 31 - __clz(__ballot_sync(~0u, at <= rem));
        before = __shfl_sync(~0u, at, top);
        lo += top * step;
        hi = min(hi, lo + step);
      }
      cur.j = r.j + lo;
      rem -= before + PA_TILE_KEYS;
    }
    cur.tile(p, from);
    if (in_part) rem += cur.keys(p, from, i, PaStream{cur.first, cur.t0, cur.t1, cur.gr.prefix});
    // A cut in what the tile costs besides, or in a short tile, is one before the tile; one behind its blocks is before the next.  (Cuts
    // are 256 keys apart or more, which are at least 170 of a tile's and so another block: no two pieces start at the same block inside of
    // a tile, and a part that the join looks for has been written.)
    int b = cur.nb <= PA_WHOLE || rem <= 0 ? 0 : (int)(rem >> 7);
    cur.h = pl[warp].h;
    cur.eh = -1;
    if (b >= cur.nb) {
      cur.next_tile(p);
      b = 0;
    }
    const bool end = cur.h >= p.pg.H;
    if (lane == 0) {
      pl[warp].h = cur.h;
      pl[warp].g = end ? 0 : cur.g;
      pl[warp].j = end ? 0 : cur.j;
      pl[warp].b = b;
      pl[warp].tile = cur;
      if (warp == 0)
        p.rec[c] = end ? PaRec{-1, 0, 0, 0, 0, 0} : PaRec{(long long)cur.h * p.c.total + cur.t0, b, cur.t0, cur.t1 - cur.t0, cur.h, pieces};
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (copies go where `space` is)
  __syncthreads();
}

}  // namespace qe
