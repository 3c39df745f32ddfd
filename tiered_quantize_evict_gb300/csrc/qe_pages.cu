// qe_pages.cu -- the paged cache's kernels besides attention: appending with rotary positions,
// resizing, forking and compacting rows, copying pages, gathering rows.
//
// All of it moves data (no contraction): each kernel is bound by memory, or by launch latency when small.
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qe_common.cuh"
#include "qe_pages.cuh"

namespace qe {

// a launch that may start while the one before it still runs (it waits inside)
template <class K, class... A>
static cudaError_t launch_after(K kernel, unsigned blocks, unsigned threads, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------------------- append
template <bool FP16>
__device__ __forceinline__ float2 pages_unpack(unsigned x) {
  if constexpr (FP16) {
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    return __half22float2(h);
  }
  return make_float2(bf16lo_to_f32(x), bf16hi_to_f32(x));
}
template <bool FP16>
__device__ __forceinline__ unsigned pages_pack(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

constexpr int APPEND_MAX_TOKENS = 8, APPEND_THREADS = 256;
constexpr int APPEND_BLOCKS = 4;   // of an SM
constexpr int APPEND_DEEP = 3;     // rows that a thread loads at a time (2: 68.4 us where 3 takes 65.7; 6, with three blocks: 68.6)
// Tokens that a block takes at a time, times head_dim: 4 of 128 channels or 8 of 64, so that a thread has one angle at most.
constexpr int APPEND_CHANNELS = 2 * APPEND_THREADS;

// which sequence token tok belongs to (by a warp)
__device__ __forceinline__ int pages_find_seq(const ChunksView& c, int tok) { return pages_count_below(c.q_start + 1, c.n, tok); }

// A block rotates and stores its share of the packed tokens, a few at a time.  The angle of (token, pair) is taken once
// for all heads: position * turn mod 2^64 is the exact fraction of a turn (64-bit integers wrap at
// whole turns), whose upper 32 bits, as a signed number of 2^-31 half turns, go to sincospif -- no
// 64-bit floating point, and no loss at far positions.
// Bound by memory, and before that by a chain of dependent loads (sequence, its length, page): the positions and the first rows
// are on their way while a warp per token follows it.  All blocks run at once, with equal shares of the tokens (16K tokens of 48 heads of
// 128 channels: 65.7 us, 5.7 TB/s read and written; blocks of 4 tokens each: 68; 256 sequences of a token: 4.9 us).
template <bool FP16>
__global__ void __launch_bounds__(APPEND_THREADS, APPEND_BLOCKS) pages_append_kernel(const __grid_constant__ PagesAppendParams p) {
  __shared__ float2 s_cs[APPEND_MAX_TOKENS][64];
  __shared__ int s_pos[APPEND_MAX_TOKENS];         // cache position, < 0: none; INT_MIN: not a token of the call
  __shared__ long long s_at[APPEND_MAX_TOKENS];    // offset of head 0 in the pool, < 0: dropped
  griddep_wait();
  if (blockIdx.x == 0) check_starts(p.pg, p.c);
  const int most = APPEND_CHANNELS / p.pg.D, half = p.R / 2, Hq = p.q ? p.Hq : 0;
  // A thread keeps one token and one vector (8 adjacent channels; with halves 8 of the first half and their partners) and
  // walks the heads, so the sines and cosines stay in registers and several heads' loads are in flight.
  const int nv = p.halves ? p.R / 16 + (p.pg.D - p.R) / 8 : p.pg.D / 8;
  const int grp = threadIdx.x / nv, v = threadIdx.x - grp * nv;
  const bool paired = p.halves && v < p.R / 16;
  const int c0 = paired ? v * 8 : (p.halves ? p.R + (v - p.R / 16) * 8 : v * 8);   // first channel, and its partner's
  const int c1 = c0 + half;
  const int angles = paired ? 8 : (p.halves ? 0 : min(4, max(0, half - v * 4)));
  const int at = half ? (int)threadIdx.x / half : APPEND_MAX_TOKENS, ac = threadIdx.x - at * half;   // this thread's angle: token, pair
  const int end = (int)((long long)p.c.total * (blockIdx.x + 1) / gridDim.x);
  int t0 = (int)((long long)p.c.total * blockIdx.x / gridDim.x);
#pragma unroll 1
  for (int nt; t0 < end; t0 += nt) {
    nt = min(most, end - t0);
    const int slots = APPEND_THREADS / nv / nt;                // threads that share a token's heads
    const int t = grp / slots, h0 = grp - t * slots;
    const long long tok = t0 + t;
    // the token's rows: query heads, keys, values; first what a thread of slot h0 loads before it knows where they go
    constexpr int DEEP = APPEND_DEEP;
    uint4 x[DEEP], y[DEEP];
    auto load = [&](int rows, int h) {
#pragma unroll
      for (int k = 0; k < DEEP; ++k) {
        const int r = h + k * slots;
        if (r < rows) {
          const uint16_t* src = r < Hq ? p.q + tok * p.qts + r * p.qhs
                                       : (r < Hq + p.pg.H ? p.k + tok * p.kts + (r - Hq) * p.khs : p.v + tok * p.vts + (r - Hq - p.pg.H) * p.vhs);
          x[k] = *reinterpret_cast<const uint4*>(src + c0);
          if (paired) y[k] = *reinterpret_cast<const uint4*>(src + c1);
        }
      }
    };
    long long turns = 0;
    if (p.positions && at < nt) turns = p.positions[p.axis[ac] * p.pos_stride + t0 + at];
    if (t < nt) load(Hq + 2 * p.pg.H, h0);

    const int warp = threadIdx.x >> 5;
    if (warp < nt) {
      const int mine = t0 + warp, seq = pages_find_seq(p.c, mine);
      if ((threadIdx.x & 31) == 0) {
        int pos = INT_MIN;
        long long to = -1;
        if (seq < p.c.n) {
          const SeqInfo s = seq_info(p.pg, p.t, p.c, seq, true);
          if (mine >= s.q0 && mine < s.q0 + s.m) {
            pos = s.len - s.m + (mine - s.q0);
            if (pos >= 0 && s.len > 0) {
              const int page = page_at(p.pg, p.t, s.row, pos);
              if (page >= 0) to = p.layer * p.pg.ls + page * p.pg.ps + (pos & (p.pg.S - 1)) * p.pg.ts;
            }
          }
        }
        s_pos[warp] = pos;
        s_at[warp] = to;
      }
    }
    __syncthreads();
    if (at < nt) {
      if (!p.positions) turns = max(s_pos[at], 0);
      const int turn = (int)(((unsigned long long)turns * p.turn[ac]) >> 32);
      float sn, cs;
      sincospif((float)turn * 0x1p-31f, &sn, &cs);
      s_cs[at][ac] = make_float2(cs, sn);
    }
    __syncthreads();
    if (t < nt && s_pos[t] != INT_MIN) {
      float2 cs[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) cs[k] = k < angles ? s_cs[t][paired ? c0 + k : v * 4 + k] : make_float2(1.f, 0.f);
      const long long to = s_at[t];
      const int rows = to >= 0 ? Hq + 2 * p.pg.H : Hq;
#pragma unroll 1
      for (int h = h0; h < rows; h += DEEP * slots) {
        if (h != h0) load(rows, h);
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
          const int r = h + k * slots;
          if (r < rows) {
            unsigned *a = &x[k].x, *b = &y[k].x;
            const bool rot = r < Hq + p.pg.H;
            if (rot && paired) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 xa = pages_unpack<FP16>(a[e]), ya = pages_unpack<FP16>(b[e]), q0 = cs[2 * e], q1 = cs[2 * e + 1];
                a[e] = pages_pack<FP16>(xa.x * q0.x - ya.x * q0.y, xa.y * q1.x - ya.y * q1.y);
                b[e] = pages_pack<FP16>(xa.x * q0.y + ya.x * q0.x, xa.y * q1.y + ya.y * q1.x);
              }
            } else if (rot) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e < angles) {
                  const float2 xa = pages_unpack<FP16>(a[e]);
                  a[e] = pages_pack<FP16>(xa.x * cs[e].x - xa.y * cs[e].y, xa.x * cs[e].y + xa.y * cs[e].x);
                }
            }
            uint16_t* dst = r < Hq ? p.q_out + tok * p.ots + r * p.ohs
                                   : (rot ? p.pg.k + to + (r - Hq) * p.pg.hs : p.pg.v + to + (r - Hq - p.pg.H) * p.pg.hs);
            *reinterpret_cast<uint4*>(dst + c0) = x[k];
            if (paired) *reinterpret_cast<uint4*>(dst + c1) = y[k];
          }
        }
      }
    }
    __syncthreads();   // (positions, places and angles are read)
  }
}

cudaError_t launch_pages_append(const PagesAppendParams& p, int fp16, int n_sm, cudaStream_t st) {
  // all blocks run at once, with equal shares of the tokens
  const int blocks = p.c.total < n_sm * APPEND_BLOCKS ? p.c.total : n_sm * APPEND_BLOCKS;
  return fp16 ? launch_after(pages_append_kernel<true>, blocks, APPEND_THREADS, st, p) : launch_after(pages_append_kernel<false>, blocks, APPEND_THREADS, st, p);
}

// ---------------------------------------------------------------------------- planning
//
// One block plans a call, so that everything it decides is in one order: which entries are valid, how many
// pages each needs, and the lowest free pages for them.  The second kernel does the work with all SMs.
//
// Workspace: header, row moves [n], owners [n_rows], pages taken [n_pages], pairs [n_pages or n],
// new places [n_pages].
struct PlanHeader {
  int n_pairs;     // pages to copy
  int go;          // 0: the call changes nothing
  int n_live;
  int pad;
};

struct PlanSpace {
  PlanHeader* head;
  PagesRowMove* mv;
  int* owner;
  int* taken;
  PagesPair* pair;
  int* place;
};
static size_t plan_layout(void* ws, int n_pages, int n_rows, int n, PlanSpace* o) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += (bytes + 15) / 16 * 16;
    return static_cast<char*>(ws) + r;
  };
  PlanSpace s;
  s.head = reinterpret_cast<PlanHeader*>(take(sizeof(PlanHeader)));
  s.mv = reinterpret_cast<PagesRowMove*>(take(sizeof(PagesRowMove) * (size_t)n));
  s.owner = reinterpret_cast<int*>(take(sizeof(int) * (size_t)n_rows));
  s.taken = reinterpret_cast<int*>(take(sizeof(int) * (size_t)n_pages));
  s.pair = reinterpret_cast<PagesPair*>(take(sizeof(PagesPair) * (size_t)(n_pages > n ? n_pages : n)));
  s.place = reinterpret_cast<int*>(take(sizeof(int) * (size_t)n_pages));
  if (o) *o = s;
  return at;
}
size_t pages_manage_bytes(int n_pages, int n_rows, int n) { return plan_layout(nullptr, n_pages, n_rows, n, nullptr); }

constexpr int PLAN_THREADS = 1024;

// exclusive sum over the block's threads; the block's total through *total
__device__ __forceinline__ int plan_scan(int x, int* total) {
  __shared__ int s_w[PLAN_THREADS / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int z = __shfl_up_sync(~0u, y, k);
    if (lane >= k) y += z;
  }
  if (lane == 31) s_w[w] = y;
  __syncthreads();
  int v = s_w[lane];
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int z = __shfl_up_sync(~0u, v, k);
    if (lane >= k) v += z;
  }
  *total = __shfl_sync(~0u, v, 31);
  const int before = w ? __shfl_sync(~0u, v, w - 1) : 0;
  __syncthreads();
  return before + y - x;
}

// the `need` lowest free pages, in order, into taken; how many there are
__device__ int plan_take(const PagesView& pg, const int* refs, int need, int* taken) {
  int got = 0;
  for (int b = 0; b < pg.P && got < need; b += PLAN_THREADS) {
    const int i = b + threadIdx.x;
    const bool free = i < pg.P && refs[i] == 0;
    int tot;
    const int r = plan_scan(free, &tot);
    if (free && got + r < need) taken[got + r] = i;
    got += tot;
  }
  return got;
}

// FORK: row a[i] -> row b[i]; else: row a[i] gets length b[i] (0 where b is NULL)
template <bool FORK>
__device__ void plan_moves(const PagesView& pg, const TableView& t, const int* a, const int* b, int n, const PlanSpace& ws) {
  const long long most = pages_most(pg, t);
  const int tid = threadIdx.x;
  for (int i = tid; i < n; i += PLAN_THREADS) {
    const int row = FORK ? b[i] : a[i];
    if (row >= 0 && row < t.rows) ws.owner[row] = INT_MAX;
  }
  __syncthreads();
  for (int i = tid; i < n; i += PLAN_THREADS) {
    const int row = FORK ? b[i] : a[i];
    if (row >= 0 && row < t.rows) atomicMin(&ws.owner[row], i);
  }
  __syncthreads();
  int need = 0, pairs = 0;
  for (int base = 0; base < n; base += PLAN_THREADS) {
    const int i = base + tid;
    PagesRowMove m{-1, -1, 0, 0, 0, -1};
    int want = 0, copy = 0, from = -1, used = 0;
    if (i < n) {
      const int row = FORK ? b[i] : a[i], src = FORK ? a[i] : row;
      bool ok = row >= 0 && row < t.rows && src >= 0 && src < t.rows && ws.owner[row] == i;
      if (ok) {
        const int old_len = t.kv_len[row], len = FORK ? t.kv_len[src] : (b ? b[i] : 0);
        ok = old_len >= 0 && old_len <= most && len >= 0 && len <= most && !(FORK && old_len != 0);
        if (ok) {
          m.row = row;
          m.src = FORK ? src : -1;
          m.old_len = old_len;
          m.new_len = len;
          // the page that ends up partly filled (fork), or was or becomes so (resize) and must be the row's own
          const int edge = FORK ? len : min(old_len, len);
          used = edge & (pg.S - 1);
          if (used && (FORK || old_len != len)) {
            from = page_at(pg, t, src, edge);
            copy = from >= 0 && (FORK || t.refs[from] > 1);
          }
          if (!FORK) want = max(0, (int)(((long long)len + pg.S - 1) >> pg.lgS) - (int)(((long long)old_len + pg.S - 1) >> pg.lgS));
        }
      }
      if (!ok) pages_report(pg, QE_PAGES_ERR_ROW);
    }
    int tot, ptot;
    const int at = need + plan_scan(want + copy, &tot);
    const int pr = pairs + plan_scan(copy, &ptot);
    if (i < n) {
      m.first_new = at + copy;
      m.copy_page = copy ? at : -1;   // an index into the pages taken until they are known
      ws.mv[i] = m;
      if (copy) ws.pair[pr] = PagesPair{from, at, used, 0};
    }
    need += tot;
    pairs += ptot;
  }
  const int got = plan_take(pg, t.refs, need, ws.taken);
  __syncthreads();
  const bool go = got >= need;
  if (go) {
    for (int i = tid; i < n; i += PLAN_THREADS)
      if (ws.mv[i].copy_page >= 0) ws.mv[i].copy_page = ws.taken[ws.mv[i].copy_page];
    for (int i = tid; i < pairs; i += PLAN_THREADS) ws.pair[i].dst = ws.taken[ws.pair[i].dst];
  }
  if (tid == 0) {
    *ws.head = PlanHeader{go ? pairs : 0, go, 0, 0};
    if (!go) pages_report(pg, QE_PAGES_ERR_NO_PAGES);
  }
}

__device__ __forceinline__ void ref_down(const PagesView& pg, int* refs, int page) {
  if (page == QE_PAGES_DROPPED) return;   // given back already
  if (page < 0 || page >= pg.P) {
    pages_report(pg, QE_PAGES_ERR_PAGE);
    return;
  }
  if (atomicSub(&refs[page], 1) <= 0) {   // more references given up than counted
    atomicAdd(&refs[page], 1);
    pages_report(pg, QE_PAGES_ERR_PAGE);
  }
}

// Rows of head_dim channels, one warp: vector v of 16 bytes is channels 8 (v mod vpr) of row v / vpr.  COPY_DEEP loads per lane
// are in flight before the first store: memory is what bounds it (measured 6.2 TB/s read and written for 2 GB of pages against
// 4.9 TB/s with one).
constexpr int COPY_DEEP = 8;
__device__ __forceinline__ void copy_rows(const PagesView& pg, const uint16_t* from, uint16_t* to, int vectors) {
  const int lgv = pg.D == 128 ? 4 : 3, lane = threadIdx.x & 31;
  for (int v0 = lane; v0 < vectors; v0 += 32 * COPY_DEEP) {
    uint4 x[COPY_DEEP];
#pragma unroll
    for (int k = 0; k < COPY_DEEP; ++k) {
      const int v = v0 + 32 * k;
      if (v < vectors) x[k] = *reinterpret_cast<const uint4*>(from + (long long)(v >> lgv) * pg.ts + ((v & ((1 << lgv) - 1)) << 3));
    }
#pragma unroll
    for (int k = 0; k < COPY_DEEP; ++k) {
      const int v = v0 + 32 * k;
      if (v < vectors) *reinterpret_cast<uint4*>(to + (long long)(v >> lgv) * pg.ts + ((v & ((1 << lgv) - 1)) << 3)) = x[k];
    }
  }
}

struct CopyUnit {
  long long item;
  int l, kv, h;
};
// unit u of (item, layer, keys or values, head), heads innermost
__device__ __forceinline__ CopyUnit copy_unit(long long u, int L, int H) {
  CopyUnit c;
  if (u >> 32) {
    c.h = (int)(u % H);
    u /= H;
    c.kv = (int)(u & 1);
    u >>= 1;
    c.l = (int)(u % L);
    c.item = u / L;
  } else {
    unsigned x = (unsigned)u;
    c.h = x % (unsigned)H;
    x /= (unsigned)H;
    c.kv = x & 1;
    x >>= 1;
    c.l = x % (unsigned)L;
    c.item = x / (unsigned)L;
  }
  return c;
}

// Copies of whole or partly used pages, a warp per head of a page of a layer, of the keys or the values.
__device__ void copy_pairs(const PagesView& pg, const PagesPair* pair, const int* src, const int* dst, int n, unsigned bid,
                           unsigned blocks) {
  const unsigned per = blockDim.x >> 5;
  const long long units = (long long)n * pg.L * 2 * pg.H;
  for (long long u = (long long)bid * per + (threadIdx.x >> 5); u < units; u += (long long)blocks * per) {
    const CopyUnit c = copy_unit(u, pg.L, pg.H);
    const int s = pair ? pair[c.item].src : src[c.item], d = pair ? pair[c.item].dst : dst[c.item], rows = pair ? pair[c.item].rows : pg.S;
    if (s < 0 || s >= pg.P || d < 0 || d >= pg.P) {
      if ((threadIdx.x & 31) == 0) pages_report(pg, QE_PAGES_ERR_PAGE);
      continue;
    }
    if (s == d) continue;
    uint16_t* base = (c.kv ? pg.v : pg.k) + c.l * pg.ls + c.h * pg.hs;
    copy_rows(pg, base + s * pg.ps, base + d * pg.ps, rows * (pg.D / 8));
  }
}

// The work of a planned resize or fork, by block bid of several: table entries, reference counts, lengths, page copies.
// TEAM threads take a row.
template <bool FORK, int TEAM>
__device__ void apply_moves(const PagesView& pg, const TableView& t, int n, const PlanSpace& ws, int bid, int blocks) {
  const PlanHeader head = *ws.head;
  if (!head.go) return;
  const int tid = threadIdx.x % TEAM, teams = blockDim.x / TEAM;
  for (int i = bid * teams + threadIdx.x / TEAM; i < n; i += blocks * teams) {
    const PagesRowMove m = ws.mv[i];
    if (m.row < 0) continue;
    int* row = t.table + (long long)m.row * t.stride;
    const int oldp = (int)(((long long)m.old_len + pg.S - 1) >> pg.lgS), newp = (int)(((long long)m.new_len + pg.S - 1) >> pg.lgS);
    if (FORK) {
      const int* from = t.table + (long long)m.src * t.stride;
      const int full = m.new_len >> pg.lgS;
      for (unsigned u = tid; u < (unsigned)t.cols; u += TEAM) {   // (up to 2^31 - 2 columns)
        const int j = (int)u;
        int e = -1;
        if (j < full) {
          e = from[j];
          if (e >= 0 && e < pg.P) atomicAdd(&t.refs[e], 1);
          else if (e != QE_PAGES_DROPPED) {
            e = -1;
            pages_report(pg, QE_PAGES_ERR_PAGE);
          }
        } else if (j < newp && m.copy_page >= 0) {
          e = m.copy_page;
          t.refs[e] = 1;
        }
        row[j] = e;
      }
    } else {
      const int edge = min(m.old_len, m.new_len) >> pg.lgS;
      if (tid == 0 && m.copy_page >= 0) {
        ref_down(pg, t.refs, row[edge]);
        row[edge] = m.copy_page;
        t.refs[m.copy_page] = 1;
      }
      for (int j = min(oldp, newp) + tid; j < max(oldp, newp); j += TEAM) {
        if (j >= oldp) {
          const int e = ws.taken[m.first_new + j - oldp];
          row[j] = e;
          t.refs[e] = 1;
        } else {
          ref_down(pg, t.refs, row[j]);
          row[j] = -1;
        }
      }
    }
    if (tid == 0) t.kv_len[m.row] = m.new_len;
  }
  copy_pairs(pg, ws.pair, nullptr, nullptr, head.n_pairs, bid, blocks);
}

// ALL: the planning block does the work too (a call so small that a second launch would cost more: 10 -> 6 us)
template <bool FORK, bool ALL>
__global__ void __launch_bounds__(PLAN_THREADS) pages_plan_kernel(const __grid_constant__ PagesView pg, const __grid_constant__ TableView t,
                                                                  const int* a, const int* b, int n,
                                                                  const __grid_constant__ PlanSpace ws) {
  griddep_wait();
  griddep_launch_dependents();
  plan_moves<FORK>(pg, t, a, b, n, ws);
  if constexpr (ALL) {
    __syncthreads();
    apply_moves<FORK, 32>(pg, t, n, ws, 0, 1);
  }
}
template <bool FORK>
__global__ void __launch_bounds__(256) pages_apply_kernel(const __grid_constant__ PagesView pg, const __grid_constant__ TableView t, int n,
                                                          const __grid_constant__ PlanSpace ws) {
  griddep_wait();
  apply_moves<FORK, 256>(pg, t, n, ws, blockIdx.x, gridDim.x);
}

template <bool FORK>
static cudaError_t launch_planned(const PagesView& pg, const TableView& t, const int* a, const int* b, int n, void* ws, int n_sm,
                                  cudaStream_t st) {
  PlanSpace s;
  plan_layout(ws, pg.P, t.rows, n, &s);
  // at most a page per entry is copied (none where rows are only freed)
  const long long copied = !FORK && !b ? 0 : (long long)n * pg.L * 2 * pg.H * pg.S * pg.D * 2;
  // (one block: 4 rows of 19 pages forked and freed 12.8 us, with two launches each 14.4; 64 rows of 94 pages 50.8 against 48.2.  What
  // could be copied counts as if every entry copied a page: a fork or resize to lengths of a usual cache of several layers is two launches)
  if (copied <= 128 * 1024 && (long long)n * t.cols <= 2048) {
    return launch_after(pages_plan_kernel<FORK, true>, 1, PLAN_THREADS, st, pg, t, a, b, n, s);
  }
  const cudaError_t e = launch_after(pages_plan_kernel<FORK, false>, 1, PLAN_THREADS, st, pg, t, a, b, n, s);
  return e != cudaSuccess ? e : launch_after(pages_apply_kernel<FORK>, n_sm * 8, 256, st, pg, t, n, s);
}
cudaError_t launch_pages_resize(const PagesView& pg, const TableView& t, const int* rows, const int* new_len, int n, void* ws,
                                int n_sm, cudaStream_t st) {
  return launch_planned<false>(pg, t, rows, new_len, n, ws, n_sm, st);
}
cudaError_t launch_pages_fork(const PagesView& pg, const TableView& t, const int* src, const int* dst, int n, void* ws, int n_sm,
                              cudaStream_t st) {
  return launch_planned<true>(pg, t, src, dst, n, ws, n_sm, st);
}

// ---------------------------------------------------------------------------- compact
__global__ void __launch_bounds__(PLAN_THREADS) pages_plan_compact_kernel(const PagesView pg, const TableView t, const PlanSpace ws,
                                                                          int* n_live_out) {
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int live = 0;
  for (int i = tid; i < pg.P; i += PLAN_THREADS) live += t.refs[i] > 0;
  int n_live;
  plan_scan(live, &n_live);
  int holes = 0, movers = 0;
  for (int base = 0; base < pg.P; base += PLAN_THREADS) {
    const int i = base + tid;
    const int r = i < pg.P ? t.refs[i] : 0;
    const bool hole = i < n_live && r <= 0, mover = i >= n_live && r > 0;
    int th, tm;
    const int h = holes + plan_scan(hole, &th), m = movers + plan_scan(mover, &tm);
    if (hole) ws.taken[h] = i;
    if (mover) {
      ws.place[i] = m;   // its rank until the holes are all known
      ws.pair[m].src = i;
      ws.pair[m].rows = pg.S;
      ws.pair[m].refs = r;
    } else if (i < pg.P) {
      ws.place[i] = r > 0 ? i : -1;
    }
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += PLAN_THREADS) {   // as many holes as movers
    const int d = ws.taken[i];
    ws.pair[i].dst = d;
    ws.place[ws.pair[i].src] = d;
  }
  if (tid == 0) {
    *ws.head = PlanHeader{movers, 1, n_live, 0};
    if (n_live_out) *n_live_out = n_live;
  }
}

__global__ void __launch_bounds__(256) pages_compact_kernel(const PagesView pg, const TableView t, const PlanSpace ws, int* table_out,
                                                            int* refs_out) {
  griddep_wait();
  const PlanHeader head = *ws.head;
  const long long nt = (long long)gridDim.x * blockDim.x, id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = id; i < (long long)t.rows * t.cols; i += nt) {
    const long long r = i / t.cols, at = r * t.stride + (i - r * t.cols);
    const int e = t.table[at];
    int to = e;
    if (e >= 0) {
      to = e < pg.P ? ws.place[e] : -1;
      if (to < 0) {   // an entry that names no live page
        pages_report(pg, QE_PAGES_ERR_PAGE);
        to = -1;
      }
    }
    table_out[at] = to;
  }
  for (long long i = id; i < pg.P; i += nt) {
    if (i >= head.n_live) refs_out[i] = 0;
    else if (ws.place[i] == (int)i) refs_out[i] = t.refs[i];
  }
  for (long long i = id; i < head.n_pairs; i += nt) refs_out[ws.pair[i].dst] = ws.pair[i].refs;
  copy_pairs(pg, ws.pair, nullptr, nullptr, head.n_pairs, blockIdx.x, gridDim.x);
}

cudaError_t launch_pages_compact(const PagesView& pg, const TableView& t, int* table_out, int* refs_out, int* n_live, void* ws,
                                 int n_sm, cudaStream_t st) {
  PlanSpace s;
  plan_layout(ws, pg.P, t.rows, 0, &s);
  const cudaError_t e = launch_after(pages_plan_compact_kernel, 1, PLAN_THREADS, st, pg, t, s, n_live);
  return e != cudaSuccess ? e : launch_after(pages_compact_kernel, n_sm * 8, 256, st, pg, t, s, table_out, refs_out);
}

// ---------------------------------------------------------------------------- drop
// A warp takes DROP_ENTRIES table entries of a row at a time.  Where little goes it is bound by its launch: four bytes are read for each page
// that the window has left (256 rows of up to 32K tokens with nothing to give back: 3.4 us in a graph).  A page that goes is a chain of three
// accesses, and a lane has its 8 entries' one after the other: the same rows giving back 275102 pages, 4.4 MB, take 12 us.
constexpr int DROP_ENTRIES = 256;
// of the columns that a row can use
__host__ __device__ __forceinline__ int drop_parts(const PagesView& pg, const TableView& t) {
  const int most = (1 << 30) >> pg.lgS;
  return ((t.cols < most ? t.cols : most) + DROP_ENTRIES - 1) / DROP_ENTRIES;
}
__global__ void __launch_bounds__(256) pages_drop_kernel(const PagesView pg, const TableView t, const int* rows, int n, const PagesWindow w) {
  griddep_wait();
  const int lane = threadIdx.x & 31, parts = drop_parts(pg, t);
  const int first = (int)(((long long)w.sinks + pg.S - 1) >> pg.lgS);
  const long long units = (long long)n * parts;
  for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (long long)gridDim.x * 8) {
    const int i = (int)(u / parts), part = (int)(u - (long long)i * parts), row = rows[i];
    const int len = row_len(pg, t, row, part == 0 && lane == 0);
    const int end = min((max(len - w.window + 1, 0) >> pg.lgS), (part + 1) * DROP_ENTRIES);
    if (len == 0 || t.kv_len[row] != len) continue;   // (nothing goes by a length that is out of range)
    int* entry = t.table + (long long)row * t.stride;
    for (int j = max(first, part * DROP_ENTRIES) + lane; j < end; j += 32)
      // (exchanged: another entry of the call may name the row too)
      if (entry[j] != QE_PAGES_DROPPED) ref_down(pg, t.refs, atomicExch(&entry[j], QE_PAGES_DROPPED));
  }
}
cudaError_t launch_pages_drop(const PagesView& pg, const TableView& t, const int* rows, int n, const PagesWindow& w, int n_sm, cudaStream_t st) {
  const long long blocks = ((long long)n * drop_parts(pg, t) + 7) / 8;
  return launch_after(pages_drop_kernel, (unsigned)(blocks < n_sm * 8 ? blocks : n_sm * 8), 256, st, pg, t, rows, n, w);
}

// ---------------------------------------------------------------------------- copy, gather
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagesView pg, const int* src, const int* dst, int n) {
  griddep_wait();
  copy_pairs(pg, nullptr, src, dst, n, blockIdx.x, gridDim.x);
}
cudaError_t launch_pages_copy(const PagesView& pg, const int* src, const int* dst, int n, int n_sm, cudaStream_t st) {
  const long long blocks = ((long long)n * pg.L * 2 * pg.H + 7) / 8;   // a warp per unit
  return launch_after(pages_copy_kernel, (unsigned)(blocks < n_sm * 8 ? blocks : n_sm * 8), 256, st, pg, src, dst, n);
}

// a warp per head of one page's worth of tokens of one row, of the keys or the values
__global__ void __launch_bounds__(256) pages_gather_kernel(const PagesView pg, const TableView t, int layer, const int* rows, int n,
                                                           int start, int n_tok, uint16_t* k, uint16_t* v) {
  griddep_wait();
  const int first = start >> pg.lgS, np = ((start + n_tok - 1) >> pg.lgS) - first + 1, vpr = pg.D / 8, lane = threadIdx.x & 31;
  const long long units = (long long)n * np * 2 * pg.H;
  for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (long long)gridDim.x * 8) {
    const CopyUnit c = copy_unit(u, np, pg.H);
    const int p0 = (first + c.l) << pg.lgS, s = (int)c.item, row = rows ? rows[s] : s;
    const int len = row_len(pg, t, row, lane == 0);
    const int page = p0 < len ? page_at(pg, t, row, p0) : -1;
    const int a = max(start - p0, 0), b = min(start + n_tok - p0, pg.S);         // the page's tokens that are asked for
    const int have = page >= 0 ? min(max(len - p0, a), b) : a;                    // and are there
    const uint16_t* from = (c.kv ? pg.v : pg.k) + layer * pg.ls + (long long)max(page, 0) * pg.ps + c.h * pg.hs + a * pg.ts;
    uint16_t* to = (c.kv ? v : k) + (((long long)s * pg.H + c.h) * n_tok + (p0 + a - start)) * pg.D;
    const int lgv = pg.D == 128 ? 4 : 3, all = (b - a) * vpr, some = (have - a) * vpr;
    for (int v0 = lane; v0 < all; v0 += 32 * COPY_DEEP) {
      uint4 x[COPY_DEEP];
#pragma unroll
      for (int e = 0; e < COPY_DEEP; ++e) {
        const int i = v0 + 32 * e;
        x[e] = make_uint4(0, 0, 0, 0);
        if (i < some) x[e] = *reinterpret_cast<const uint4*>(from + (long long)(i >> lgv) * pg.ts + ((i & (vpr - 1)) << 3));
      }
#pragma unroll
      for (int e = 0; e < COPY_DEEP; ++e) {
        const int i = v0 + 32 * e;
        if (i < all) *reinterpret_cast<uint4*>(to + (long long)i * 8) = x[e];
      }
    }
  }
}
cudaError_t launch_pages_gather(const PagesView& pg, const TableView& t, int layer, const int* rows, int n, int start, int n_tok,
                                uint16_t* k, uint16_t* v, int n_sm, cudaStream_t st) {
  const int np = ((start + n_tok - 1) >> pg.lgS) - (start >> pg.lgS) + 1;
  const long long blocks = ((long long)n * np * 2 * pg.H + 7) / 8;
  return launch_after(pages_gather_kernel, (unsigned)(blocks < n_sm * 8 ? blocks : n_sm * 8), 256, st, pg, t, layer, rows, n, start, n_tok, k, v);
}

}  // namespace qe
