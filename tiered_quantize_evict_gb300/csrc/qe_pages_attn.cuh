// qe_pages_attn.cuh -- what the kernels of the chunk attention share: the line of blocks and its cuts, descriptors,
// tensor-memory and TMA instructions, bounded waits.  The mathematics and the layout are in qe_pages_attn.cu; the kernel for a few query
// rows is in qe_pages_few.cu.
#pragma once
#include <climits>
#include <cstring>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qe_common.cuh"
#include "qe_pages.cuh"
#include "qe_pages_fill.cuh"

namespace qe {

constexpr int PA_BN = 128;                       // keys of a block
constexpr int PA_MAX_CTAS = 1024;
constexpr unsigned long long PA_WAIT_NS = 200000000ull;    // how long a wait may take,
constexpr unsigned long long PA_BLOCK_NS = 10000ull;       // and for each block that is walked meanwhile (measured 1.4 us)
constexpr float PA_LAZY = 8.f;                   // log2 of how far a row's maximum may pass its reference
// log2 of what probabilities and sums are multiplied by: an fp16 probability below 2^-14 is subnormal, off by up to 2^-25 and zero from there
// down.  7 above the weight, and PA_LAZY more at most, they stay within fp16's 2^16, and a weight is off by 2^-32 at most.
template <bool FP16>
constexpr float PA_UP = FP16 ? 7.f : 0.f;
template <bool FP16>
constexpr float PA_DOWN = FP16 ? 0x1p-7f : 1.f;  // 2^-PA_UP

// what a CTA's piece of the line starts with (read by the join kernel)
struct PaRec {
  long long begin;     // place of the tile on the line; -1: no piece
  int b;               // block of the tile that the piece starts with
  int tok, ntok;       // the tile's first packed token, and how many
  int kvh;
  int pieces;          // CTAs that have a piece
};

struct PaParams {
  PagesView pg;
  TableView t;
  ChunksView c;
  uint16_t* out;
  float* lse;
  long long ots, ohs;
  int Hq, G, T, causal;
  int q_rows;              // rows of a query buffer
  int ctas;                // CTAs of the attention kernel: one per SM
  int expire;              // qe_debug_inject: 4 k + role, the k-th counted wait of these warps is taken as expired; 0: none
  float scale, scale2;     // of the logits; and times log2(e)
  PaRec* rec;              // [CTAs]; NULL: no tile is cut
  float2* part_ml;         // [CTAs][2][NH][128]: reference, sum
  float* part_o;           // [CTAs][2][NH][D / 4][128][4]
};

// ---------------------------------------------------------------------------- the line of blocks

// sum over i < n of floor((a i + b) / 128), a >= 0, b >= 0.  With a and c = b reduced below 128, g = gcd(a, 128) and L = 128 / g, the
// residues of a j + c over a period j < L are c mod g, + g, + 2 g, ...: a period's sum is (a / g - 1) (L - 1) / 2 + floor(c / g), and a
// period later every term is a / g larger.  What is left, fewer than L terms, is added up one by one (L is 2 where a tile is 64 tokens).
__device__ __forceinline__ long long floor_sum128(int n, int a, long long b) {
  long long ans = n * (b >> 7) + (long long)n * (n - 1) / 2 * (a >> 7);
  a &= 127;
  const int c = (int)(b & 127);
  const int lg = a ? __ffs(a) - 1 : 7, L = 128 >> lg, A = a >> lg;
  const int q = n >> (7 - lg), r = n & (L - 1);
  ans += (long long)q * (q - 1) / 2 * (L * A) + (long long)q * (((A - 1) * (L - 1) >> 1) + (c >> lg)) + (long long)r * A * q;
  int sum = 0;
#pragma unroll 4
  for (int j = 0; j < r; ++j) sum += (a * j + c) >> 7;
  return ans + sum;
}

// quotient of numbers that are mostly small
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// What a tile costs besides its blocks (its queries, its first maximum, its output), in blocks: measured about 3800 cycles, against
// 2800 of a block.
constexpr int PA_TILE_COST = 1;
// A tile of so few blocks is never cut: a block takes a CTA 1.4 us, a join 3 us.
constexpr int PA_WHOLE = 4;
constexpr int PA_LEAST = 2;      // length of a piece, at least

struct PaSeq {
  SeqInfo s;
  int tiles;
};
template <int NH>
__device__ __forceinline__ PaSeq pa_seq(const PaParams& p, int i, bool report) {
  PaSeq r;
  r.s = seq_info(p.pg, p.t, p.c, i, report);
  const int tt = NH * p.T;
  r.tiles = (r.s.m + tt - 1) / tt;
  return r;
}
// A tile is NH T tokens of a sequence and one KV head.  Its blocks (at least one, so that rows without keys are written too)
template <int NH>
__device__ __forceinline__ int pa_blocks(const PaParams& p, const SeqInfo& s, int j) {
  const int end = p.causal ? s.len - s.m + min(s.m, (j + 1) * NH * p.T) : s.len;
  return max(1, (end + PA_BN - 1) >> 7);
}
// length on the line of the tiles before tile j (j < tiles: those are all whole)
template <int NH>
__device__ __forceinline__ long long pa_before(const PaParams& p, const SeqInfo& s, int j) {
  if (!p.causal || j == 0) return (long long)j * (PA_TILE_COST + max(1, (s.len + PA_BN - 1) >> 7));
  const int tt = NH * p.T, off = s.len - s.m;
  const int none = off < 0 ? min(j, -off / tt) : 0;   // tiles that see no key
  return (long long)j * PA_TILE_COST + none + floor_sum128(j - none, tt, (long long)off + (long long)(none + 1) * tt + PA_BN - 1);
}
template <int NH>
__device__ __forceinline__ long long pa_head_length(const PaParams& p, const PaSeq& q) {
  return q.tiles == 0 ? 0 : pa_before<NH>(p, q.s, q.tiles - 1) + PA_TILE_COST + pa_blocks<NH>(p, q.s, q.tiles - 1);
}

// A place on the line: sequence, KV head, tile, block.  The end of the line is (n, 0, 0, 0).
struct PaPlace {
  int i, h, j, b;
  SeqInfo s;
  long long rem, head;   // (while it is being found) how far behind the sequence's start; length of a KV head
};

// A walk from one place to another, tile by tile.
template <int NH>
struct PaCursor {
  int i, h, j, b, nb;   // the place; blocks of the tile
  PaSeq q;
  int ei, eh, ej, eb;   // where the walk ends
  __device__ __forceinline__ void set(const PaParams& p, const PaPlace* pl) {
    i = pl[0].i;
    h = pl[0].h;
    j = pl[0].j;
    b = pl[0].b;
    ei = pl[1].i;
    eh = pl[1].h;
    ej = pl[1].j;
    eb = pl[1].b;
    q.s = pl[0].s;
    q.tiles = (q.s.m + NH * p.T - 1) / (NH * p.T);
    nb = pa_blocks<NH>(p, q.s, j);
  }
  // blocks left of the tile on this walk; 0: the walk is over
  __device__ __forceinline__ bool last_tile() const { return i == ei && h == eh && j == ej; }
  __device__ __forceinline__ int count() const { return last_tile() ? eb - b : nb - b; }
  __device__ __forceinline__ void next_tile(const PaParams& p) {
    if (last_tile()) {   // the walk is over
      b = eb;
      return;
    }
    b = 0;
    if (++j >= q.tiles) {
      j = 0;
      if (++h >= p.pg.H) {
        h = 0;
        do {
          if (++i >= p.c.n) {   // the end of the line
            nb = 0;
            return;
          }
          q = pa_seq<NH>(p, i, false);
        } while (q.tiles == 0);
      }
    }
    nb = pa_blocks<NH>(p, q.s, j);
  }
  __device__ __forceinline__ bool second_half(const PaParams& p) const { return NH == 2 && j * 2 * p.T + p.T < q.s.m; }
};

// Every CTA (of NT threads) finds its piece: sums the sequences' lengths on the line, cuts it, finds the places of its two cuts.  Up
// to 32 sequences are a warp's work: two warps do it, one for each cut, without barriers in between (one token over a short cache, the
// whole call: 9.7 -> 9.2 us).
template <int NH, int NT>
__device__ __noinline__ void pa_find(const PaParams& p, PaPlace* pl, long long* s_w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int W = NT / 32;
  const int c = blockIdx.x;
  auto warp_scan = [&](long long y) {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long z = __shfl_up_sync(~0u, y, k);
      if (lane >= k) y += z;
    }
    return y;
  };
  // exclusive prefix of x over the block, and the total
  auto scan = [&](long long x, long long& total) {
    const long long y = warp_scan(x);
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
  auto length = [&](int i, bool report, SeqInfo& s, long long& head) {
    if (i >= p.c.n) return 0ll;
    const PaSeq q = pa_seq<NH>(p, i, report);
    s = q.s;
    return (head = pa_head_length<NH>(p, q)) * p.pg.H;
  };
  // where the two cuts of piece c are on a line; false: there are not so many pieces
  long long cut[2];
  int pieces;
  auto make_cuts = [&](long long line) {
    const long long most = line / PA_LEAST;
    pieces = most < 1 ? 1 : (most > gridDim.x ? (int)gridDim.x : (int)most);
    const long long each = div_ll(line, pieces);
    const int over = (int)(line - each * pieces);
    cut[0] = each * c + over * c / pieces;
    cut[1] = each * (c + 1) + over * (c + 1) / pieces;
    const bool there = c < pieces && line > 0;
    if (!there && tid == 0 && p.rec) p.rec[c] = PaRec{-1, 0, 0, 0, 0, 0};
    return there;
  };
  SeqInfo s;
  long long head;
  if (p.c.n <= 32) {
    if (warp < 2) {
      const long long x = length(lane, c == 0 && warp == 0, s, head), y = warp_scan(x);
      const bool there = make_cuts(__shfl_sync(~0u, y, 31));
      const long long mine = warp == 0 ? cut[0] : cut[1];
      const bool here = there && mine >= y - x && mine < y;
      if (!__any_sync(~0u, here)) {
        if (lane == 0) pl[warp].i = p.c.n, pl[warp].h = pl[warp].j = pl[warp].b = 0;
      } else if (here) {
        pl[warp].i = lane;
        pl[warp].s = s;
        pl[warp].head = head;
        pl[warp].rem = mine - (y - x);
      }
      __syncwarp();
    }
  } else {
    if (tid < 2) pl[tid].i = p.c.n, pl[tid].h = pl[tid].j = pl[tid].b = 0;
    long long line, x = length(tid, c == 0, s, head), pre = scan(x, line);
#pragma unroll 1
    for (int base = NT; base < p.c.n; base += NT) {   // (more sequences than threads)
      long long tot;
      SeqInfo z;
      scan(length(base + tid, c == 0, z, head), tot);
      line += tot;
    }
    if (make_cuts(line)) {
      long long at = 0;
#pragma unroll 1
      for (int base = 0; base < p.c.n; base += NT) {
        if (base > 0 || p.c.n > NT) x = length(base + tid, false, s, head);
        if (p.c.n > NT) {
          long long tot;
          pre = at + scan(x, tot);
          at += tot;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (cut[k] >= pre && cut[k] < pre + x) {
            pl[k].i = base + tid;
            pl[k].s = s;
            pl[k].head = head;
            pl[k].rem = cut[k] - pre;
          }
      }
    }
    __syncthreads();
  }
  if (warp < 2 && pl[warp].i < p.c.n) {
    PaSeq q;
    q.s = pl[warp].s;
    q.tiles = (q.s.m + NH * p.T - 1) / (NH * p.T);
    long long rem = pl[warp].rem;
    const int h = (int)div_ll(rem, pl[warp].head);
    rem -= h * pl[warp].head;
    int lo = 0, hi = q.tiles;   // the last tile that begins at or before rem: 32 places a round
    long long before = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, cand = lo + lane * step;
      const long long at = cand < hi ? pa_before<NH>(p, q.s, cand) : LLONG_MAX;
      const int top = 31 - __clz(__ballot_sync(~0u, at <= rem));
      before = __shfl_sync(~0u, at, top);
      lo += top * step;
      hi = min(hi, lo + step);
    }
    rem -= before;
    // a cut in what the tile costs besides, or in a short tile, is one before the tile
    const int b = pa_blocks<NH>(p, q.s, lo) <= PA_WHOLE ? 0 : max(0, (int)rem - PA_TILE_COST);
    if (lane == 0) {
      pl[warp].h = h;
      pl[warp].j = lo;
      pl[warp].b = b;
      const int tt = NH * p.T;
      if (warp == 0 && p.rec) p.rec[c] = PaRec{cut[0] - rem, b, q.s.q0 + lo * tt, min(tt, q.s.m - lo * tt), h, pieces};
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------- instructions

__device__ __forceinline__ void pa_mma_ss(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void pa_mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0)
      : "memory");
}
// one lane of a converged warp
__device__ __forceinline__ bool pa_elect() {
  unsigned r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void pa_commit(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pa_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void pa_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void pa_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pa_tma4(unsigned dst, const CUtensorMap* map, int x, int y, int z, int w, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pa_tma3(unsigned dst, const CUtensorMap* map, int x, int y, int z, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// 32 float32 columns of this thread's tensor-memory lane; pa_wait_ld before their use
__device__ __forceinline__ void pa_ld32(unsigned t, unsigned* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
// 32 bytes to global memory: one store where the address allows it, else two
__device__ __forceinline__ void pa_store32(uint16_t* dst, const unsigned* r) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(r[0], r[1], r[2], r[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(r[4], r[5], r[6], r[7]);
  }
}
__device__ __forceinline__ void pa_ld16(unsigned t, unsigned* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void pa_st8(unsigned t, const unsigned* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void pa_st16(unsigned t, const unsigned* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// waits for this thread's tensor-memory loads; the registers pass through empty asm, so no use moves before it
template <int N>
__device__ __forceinline__ void pa_wait_ld(unsigned* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void pa_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

struct PaWait {
  const PagesView* pg;
  volatile int* abort;
  // Bounded wait for the phase; false when it expired or the CTA is leaving.  A warp that sits out whole tiles (the queries', the softmax
  // of a second half that a tile does not have) says how many blocks its CTA has walked by the time the wait ends: a tile of 2^25 keys
  // takes 0.4 s.
  __device__ __forceinline__ bool operator()(unsigned bar, unsigned parity, int blocks = 0) const {
    return mbar_try_wait(bar, parity) || slow(bar, parity, blocks);
  }
  __device__ __forceinline__ bool slow(unsigned bar, unsigned parity, int blocks) const {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > PA_WAIT_NS + blocks * PA_BLOCK_NS) {
        pages_report(*pg, QE_PAGES_ERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
    return true;
  }
  // The warps whose waits a test may take as expired, one wait per block or tile: those that send keys and values, issue products, send queries.
  enum Role { KEYS, PRODUCTS, QUERIES };
  static __device__ __forceinline__ int counted(const PaParams& p, Role role) { return (p.expire & 3) == role ? p.expire >> 2 : 0; }
  __device__ __forceinline__ bool count(int& left, unsigned bar, unsigned parity, int blocks = 0) const {
    if (--left != 0) return (*this)(bar, parity, blocks);
    pages_report(*pg, QE_PAGES_ERR_TIMEOUT);
    *abort = 1;
    return false;
  }
  // the same on the way out, for what has been issued
  __device__ __forceinline__ void drain(unsigned bar, unsigned parity) const {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
      if (globaltimer_ns() - t0 > PA_WAIT_NS) return;
  }
};

template <bool FP16>
__device__ __forceinline__ unsigned pa_pack(float lo, float hi) {
  unsigned d;
  if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool FP16>
__device__ __forceinline__ float2 pa_unpack(unsigned x) {
  if constexpr (FP16) {
    __half2 h;
    memcpy(&h, &x, 4);
    return __half22float2(h);
  }
  return make_float2(bf16lo_to_f32(x), bf16hi_to_f32(x));
}

// shared-memory descriptors: 128-byte swizzle, 8-row groups 1024 bytes apart.  K-major operands (Q, K); and V with
// channels as the rows of the operand (MN-major: 64 channels to a column block, blocks 128 tokens x 128 bytes apart).
constexpr unsigned long long PA_DESC_K = (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
constexpr unsigned long long PA_DESC_V = (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);

// Attention of tiles of at most 16 rows (qe_pages_few.cu).  With 17 to 32 rows as 32 columns it took 148 us where the one half of
// qe_pages_attn.cu takes 134 (8 drafts of 16 sequences of up to 16K tokens), so those stay there.
constexpr int PAGES_FEW_ROWS = 16;
cudaError_t launch_pages_few(const PaParams& p, const CUtensorMap* maps, int fp16, int device, cudaStream_t st);
cudaError_t launch_pages_join(const PaParams& p, int nh, int fp16, cudaStream_t st);

}  // namespace qe
