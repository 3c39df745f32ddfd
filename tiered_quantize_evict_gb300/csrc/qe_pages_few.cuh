// qe_pages_few.cuh -- attention over the cached pages for tiles of at most 16 query rows (decode steps, a few drafts).
//
// Bound by reading the cache, so everything else has to fit under it: the products are taken the other way round, keys (then
// channels) as the 128 rows of the tensor cores and the few query rows as N = 16 columns:
//   S^T = K Q^T (128 keys x N),   O^T += V^T P^T (head_dim channels x 2 N, keys inner),
// with the formulas and the split of the line of qe_pages_halves.cuh.  A block costs the tensor cores about 600 cycles instead of 1536,
// and a thread 4, 8 or 16 exponentials (as many as the tile has rows) instead of 64 (decode step of 16 sequences of up to 32K tokens: 302 -> 287 us with
// 128 channels, 236 -> 171 us with 64).
//  * P^T is written to shared memory in two parts per probability, rounded and remainder, as 2 N columns (about 17 significant bits
//    for bf16); the output adds the two columns of a row.  A key's 2 N columns are 64 bytes; the P of odd blocks is the other half
//    of the same 128-byte rows.
//  * R: rows that a tile can have (4, 8 or 16); the softmax leaves the other columns out: whatever lies there
//    as probabilities goes into columns of O that nobody reads (256 sequences of a token, 4 heads to a group, under a window of 512: 123 -> 100 us).
//  * A softmax thread has one key and all rows: references and running sums are per column, in registers; a column's maximum
//    is taken across the 128 threads only for a tile's first block and when a logit passes its reference by 2^8 (a vote over the four
//    warps otherwise).
// CTA: warps 0-3 softmax, 4 TMA of keys and values, 5 tensor-core issue, 6 TMA of the queries, 7 tensor memory (and TMA of values).
// mbarriers: kfull / kempty per slot, qfull / qempty per query buffer, s[i] (S i complete), p[i] (P i written; one arrival per
// softmax warp), o[i] (the P V of an even or odd block complete, as with NH = 1 there).  Waits are bounded as in qe_pages_halves.cuh.
#pragma once
#include "qe_pages_walk.cuh"

namespace qe {

constexpr int PF_THREADS = 256;

template <int D>
struct PfShape {
  static constexpr int N = PAGES_FEW_ROWS;
  static constexpr int CB = D / 64;
  static constexpr int TILE = 128 * D * 2;                        // a slot
  static constexpr int Q_CB = N * 128, Q_BUF = CB * Q_CB;          // a query buffer's column block, and the buffer
  static constexpr int P_BUF = 128 * 128;                         // 128 keys, two times 2 N columns
  static constexpr int ALL = 7 * 32768;
  static constexpr int SLOTS = (ALL - 2 * Q_BUF - P_BUF) / (2 * TILE) * 2;
  // Keys and values sent by a warp each: what a lane's copies cost, some 100 cycles each, and what it looks up is what bounds 64 channels
  // (decode step with pages of 16, 32, 64 tokens 218, 172, 151 us with one warp, 152, 148, 146 with two).  With 128 channels memory bounds,
  // and one warp sends them in the order they are used (16 sequences of up to 32K tokens 275 us with one, 282 with two).
  static constexpr bool SPLIT = D == 64;
  static constexpr int SMEM = ALL + 1024;
  static constexpr int TM_O = 2 * N, TM_COLS = 4 * N;             // tensor memory: S 0, S 1 (N columns each), O (2 N)
};

// Reduces v[0 .. N) over the warp's lanes; returns the column whose result v[0] then is (of 16, lanes 2 i and 2 i + 1 both have column i).
// Each step halves the columns a lane keeps: for 16, 16 exchanges instead of 80.
template <int N, class Op>
__device__ __forceinline__ int pf_reduce(float (&v)[N], Op op) {
  const int lane = threadIdx.x & 31;
  int first = 0;
#pragma unroll
  for (int s = 16, len = N; s >= 1; s >>= 1) {
    const bool up = lane & s;
    if (len > 1) {
      len >>= 1;
#pragma unroll
      for (int i = 0; i < len; ++i) {
        const float got = __shfl_xor_sync(~0u, up ? v[i] : v[i + len], s);
        v[i] = op(up ? v[i + len] : v[i], got);
      }
      first += up ? len : 0;
    } else {
      v[0] = op(v[0], __shfl_xor_sync(~0u, v[0], s));
    }
  }
  return first;
}

// Zeros in the rows of a slot that the lanes of a warp name, lane l row `first` + l.  All lanes write side by side, 512 bytes a time (a
// row each, 128 bytes apart, the stores take their turns in the same banks: 256 sequences under a window of 512 tokens 129 -> 123.5 us.  The
// kernel with halves writes a row each: there this made the whole of its softmax slower, by 2 to 6 %, in either form of the loop).
template <int CB>
__device__ __forceinline__ void pa_zero_rows(unsigned slot, int first, bool mine) {
  const unsigned rows = __ballot_sync(~0u, mine), lane = threadIdx.x & 31;
  constexpr int PER = 4 / CB;                                     // rows at a time
  const int sub = lane / (8 * CB), cb = lane / 8 % CB;
  const unsigned at = slot + (first >> 3) * (CB * PA_CELL) + cb * PA_CELL + (lane & 7) * 16;
#pragma unroll
  for (int i = 0; i < 32; i += PER) {
    const int r = i + sub;
    if (rows >> r & 1)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + pa_slot_row<CB>(r)), "r"(0) : "memory");
  }
}

// the softmax warps: barrier, and barrier with the OR of a truth value
__device__ __forceinline__ void pf_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool pf_or(bool v) {
  unsigned r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbar.red.or.pred p, 1, 128, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((unsigned)v)
      : "memory");
  return r != 0;
}

// R columns of this thread's tensor-memory lane, and back
template <int R>
__device__ __forceinline__ void pf_ld(unsigned t, unsigned* r) {
  if constexpr (R == 16) pa_ld16(t, r);
  else if constexpr (R == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(t) : "memory");
}
template <int R>
__device__ __forceinline__ void pf_st(unsigned t, const unsigned* r) {
  if constexpr (R == 16) pa_st16(t, r);
  else if constexpr (R == 8) pa_st8(t, r);
  else asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

template <int D, int R, bool FP16, int MODE>
__global__ void __launch_bounds__(PF_THREADS, 1)
    pages_few_kernel(const __grid_constant__ PaParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv) {
  using Sh = PfShape<D>;
  using Cursor = typename PaWalk<1, MODE>::Cursor;
  constexpr int NS = Sh::SLOTS, N = Sh::N;
  constexpr bool SPLIT = Sh::SPLIT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long b_kfull[NS], b_kempty[NS], b_qfull[2], b_qempty[2], b_s[2], b_p[2], b_o[2], b_end;
  __shared__ unsigned s_tmem;
  __shared__ int s_abort;
  __shared__ typename PaWalk<1, MODE>::Place s_place[PaWalk<1, MODE>::PLACES];
  __shared__ long long s_w[PF_THREADS / 32];
  __shared__ __align__(16) float s_red[R][4];      // a column's value of each softmax warp
  __shared__ float s_inv[R];
  __shared__ PaValid<MODE, NS> s_valid;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0), aux = warp - 4;   // aux: TMA, tensor cores, queries, tensor memory
  const unsigned sm = (smem_u32(smem_raw) + 1023) & ~1023u;
  const unsigned sm_q = sm, sm_p = sm + 2 * Sh::Q_BUF, sm_kv = sm_p + Sh::P_BUF;
  const PaWait wait{&p.pg, &s_abort};

  if (aux == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(Sh::TM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&b_kfull[i]), 1);
      mbar_init(smem_u32(&b_kempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b_qfull[i]), 1);
      mbar_init(smem_u32(&b_qempty[i]), 1);
      mbar_init(smem_u32(&b_s[i]), 1);
      mbar_init(smem_u32(&b_p[i]), 4);
      mbar_init(smem_u32(&b_o[i]), 1);
    }
    mbar_init(smem_u32(&b_end), 1);
    mbar_fence_init();
    s_abort = 0;
  }
  // columns behind the tile's rows are zero queries
  for (int i = tid; i < 2 * Sh::Q_BUF / 16; i += PF_THREADS)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sm_q + i * 16), "r"(0) : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  pa_fence_before();
  griddep_wait();
  griddep_launch_dependents();   // (what follows may then rely on all that ran before this launch)
  static_assert(2 * Sh::Q_BUF + 4 * pa_find_ints(PF_THREADS) <= Sh::ALL, "the cuts' space is behind the query buffers");
  const bool work = PaWalk<1, MODE>::template find<PF_THREADS>(p, s_place, s_w, reinterpret_cast<int*>(smem_raw + 1024 + 2 * Sh::Q_BUF));   // ends with a barrier
  pa_fence_after();
  const unsigned tm = s_tmem;

  if (work && (aux == 0 || (SPLIT && aux == 3))) {
    // ============================== keys and values, or one of them
    const int kv0 = SPLIT && aux == 3;
    constexpr int STEP = SPLIT ? 2 : 1;
    static_assert(!SPLIT || NS % 2 == 0, "keys and values have slots of their own");
    Cursor cur;
    cur.set(p, s_place);
    const PaCopy<Sh::CB> copy(p);
    // this lane's piece, its entry loaded a block before it is looked at
    typename PaWalk<1, MODE>::Keys keys;
    int slot = kv0, ph = 1, issued = 0, left = cur.count();
    PaPiece next = keys.at(p, cur, cur.b, copy.piece * copy.rows);
    int till = PaWait::counted(p, PaWait::KEYS);
    bool ok = true;
#pragma unroll 1
    while (left > 0 && ok) {
      const int tk = next.tok, h = cur.h, now = next.entry;
      const bool there = next.entry >= 0 && next.entry < p.pg.P;
      if (!there && next.valid != PA_NO_KEYS) pages_report(p.pg, QE_PAGES_ERR_PAGE);
      const int valid = there ? next.valid : 255;
      ++cur.b;
      if (--left == 0) {
        cur.next_tile(p);
        left = cur.count();
      }
      if (left > 0) next = keys.at(p, cur, cur.b, copy.piece * copy.rows);
#pragma unroll 1
      for (int kv = kv0; kv < (SPLIT ? kv0 + 1 : 2); ++kv) {
        ok = ok && wait.count(till, smem_u32(&b_kempty[slot]), ph);
        if (!__all_sync(~0u, ok)) {
          ok = false;
          break;
        }
        const unsigned full = smem_u32(&b_kfull[slot]);
        if constexpr (MODE == PA_SHARED) {   // (told by the values' arrival)
          if (kv && lane < copy.pieces) s_valid.set(slot, lane, valid);
          __syncwarp();
        }
        if (lane == 0) mbar_expect_tx(full, Sh::TILE);
        __syncwarp();
        if (copy.mine) copy.send(p, kv ? &mv : &mk, sm_kv + slot * Sh::TILE, there, now, h, tk, full);
        ++issued;
        if ((slot += STEP) >= NS) {
          slot -= NS;
          ph ^= 1;
        }
      }
    }
    if (lane == 0)   // the copies land before the CTA leaves (early, it may be, and for another warp's wait)
      for (int i = max(0, issued - NS / STEP); i < issued; ++i) {
        const int place = STEP * i + kv0;
        wait.drain(smem_u32(&b_kfull[place % NS]), (place / NS) & 1);
      }
  } else if (work && aux == 1) {
    // ============================== tensor cores (the whole warp walks the loop, one lane issues)
    constexpr unsigned FMT = FP16 ? 0u : (1u << 7) | (1u << 10);
    constexpr unsigned ID_S = (1u << 4) | FMT | (((unsigned)N >> 3) << 17) | ((128u >> 4) << 24);
    constexpr unsigned ID_O = (1u << 4) | FMT | (1u << 15) | (1u << 16) | ((2u * N >> 3) << 17) | (((unsigned)D >> 4) << 24);
    Cursor cur;
    cur.set(p, s_place);
    // The ring is consumed in its order (K 0, V 0, K 1, ...), but S runs a block ahead: K n is used before V n - 1.
    int slot = 0, ph = 0, pp = 0, qp = 0, tile = 0, left = 0;   // (bit i of pp, qp: the parity of p[i], qfull[i])
    int till = PaWait::counted(p, PaWait::PRODUCTS);
    bool was_first = false, ok = true, more = true;
    auto step = [&]() {
      if (++slot == NS) {
        slot = 0;
        ph ^= 1;
      }
    };
#pragma unroll 1
    for (int n = 0; more; ++n) {
      const bool first = left == 0;
      if (first) {
        if (n > 0) cur.next_tile(p);
        left = cur.count();
        more = left > 0;      // one more round for the last P V
      }
      const bool last = left == 1;
      if (more) {
        const int kslot = n == 0 ? slot : (slot + 1 == NS ? 0 : slot + 1), kph = n > 0 && slot + 1 == NS ? ph ^ 1 : ph;
        const int qb = tile & 1;
        if (first) {
          ok = ok && wait(smem_u32(&b_qfull[qb]), qp >> qb & 1);
          qp ^= 1 << qb;
        }
        ok = ok && wait.count(till, smem_u32(&b_kfull[kslot]), kph);
        if (!__all_sync(~0u, ok)) break;
        pa_fence_after();
        if (pa_elect()) {   // S n = K Q^T
          const unsigned long long a = PA_DESC_K<Sh::CB> | ((sm_kv + kslot * Sh::TILE) >> 4), b = PA_DESC_Q | ((sm_q + qb * Sh::Q_BUF) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            pa_mma_ss(tm + (n & 1) * N, a + (((k >> 2) * PA_CELL + (k & 3) * 32) >> 4), b + (((k >> 2) * Sh::Q_CB + (k & 3) * 32) >> 4), ID_S,
                      k > 0);
          pa_commit(smem_u32(&b_s[n & 1]));
          pa_commit(smem_u32(&b_kempty[kslot]));
          if (last) pa_commit(smem_u32(&b_qempty[qb]));
        }
        __syncwarp();
        if (last) ++tile;
      }
      if (n > 0) {
        ok = ok && wait(smem_u32(&b_kfull[slot]), ph);
        const int pb = (n - 1) & 1;
        ok = ok && wait(smem_u32(&b_p[pb]), pp >> pb & 1);
        pp ^= 1 << pb;
        if (!__all_sync(~0u, ok)) break;
        pa_fence_after();
        if (pa_elect()) {   // O += V^T P^T
          const unsigned long long a = PA_DESC_V<Sh::CB> | ((sm_kv + slot * Sh::TILE) >> 4), b = PA_DESC_P | ((sm_p + pb * 64) >> 4);
#pragma unroll
          for (int k = 0; k < PA_BN / 16; ++k) pa_mma_ss(tm + Sh::TM_O, a + k * 128 * Sh::CB, b + k * 128, ID_O, !was_first || k > 0);
          pa_commit(smem_u32(&b_kempty[slot]));
          pa_commit(smem_u32(&b_o[pb]));
        }
        __syncwarp();
        step();
      }
      if (more) step();
      was_first = first;
      --left;
    }
    if (pa_elect()) pa_commit(smem_u32(&b_end));   // everything issued is complete before tensor memory goes
    __syncwarp();
    wait.drain(smem_u32(&b_end), 0);
  } else if (work && aux == 2) {
    // ============================== queries (one lane; the walk over groups takes the warp)
    Cursor cur;
    cur.set(p, s_place);
    PaFill fill[2];
    int tile = 0, blocks = 0, till = PaWait::counted(p, PaWait::QUERIES);   // (blocks: of the tiles before)
    bool ok = true;
    auto send = [&]() {
      const int qb = tile & 1;
      ok = wait.count(till, smem_u32(&b_qempty[qb]), fill[qb].empty(), blocks);
      if (!ok) return;
      const unsigned full = smem_u32(&b_qfull[qb]);
      mbar_expect_tx(full, p.T * p.G * 128 * Sh::CB);
      for (int cb = 0; cb < Sh::CB; ++cb)
        pa_tma3(sm_q + qb * Sh::Q_BUF + cb * Sh::Q_CB, &mq, cb * 64, cur.head() * p.G, cur.tok(p), full);
      ++fill[qb].sent;
      ++tile;
      blocks += cur.count();
    };
    auto drain = [&]() {
      for (int qb = 0; qb < 2; ++qb)
        if (fill[qb].sent > 0) wait.drain(smem_u32(&b_qfull[qb]), fill[qb].landed());
    };
    if constexpr (MODE == PA_SHARED) {
#pragma unroll 1
      for (; cur.count() > 0; cur.next_tile(p)) {
        if (lane == 0) send();
        if (!__shfl_sync(~0u, ok, 0)) break;
      }
      if (lane == 0) drain();
    } else if (lane == 0) {
#pragma unroll 1
      for (; ok && cur.count() > 0; cur.next_tile(p)) send();
      drain();
    }
  } else if (work && aux < 0) {
    // ============================== softmax: a key of every block, all rows
    const int kl = tid;
    const unsigned lane_off = (unsigned)(warp * 32) << 16;
    const unsigned prow = sm_p + kl * 128, x7 = kl & 7;   // this key's probabilities, in chunks of 16 bytes swizzled by the key
    Cursor cur;
    cur.set(p, s_place);
    int sp = 0, n = 0;   // (bit i of sp: the parity of s[i])
    auto larger = [](float a, float b) { return fmaxf(a, b); };
    auto plus = [](float a, float b) { return a + b; };
    // A wait that fails (the CTA is leaving) lets the loops run out without waiting, so that the warps' barriers stay in step.
#pragma unroll 1
    for (int cnt; (cnt = cur.count()) > 0; cur.next_tile(p)) {
      const PaFewSight<R, MODE> sight(p, cur);
      unsigned unset = 0;                                           // rows that have seen no key: they have no reference yet
      constexpr float UP = PA_UP<FP16>;
      float base[R], sum[R];                                        // UP - reference (log2 units), and this key's part of the sum
#pragma unroll
      for (int c = 0; c < R; ++c) sum[c] = 0.f;
#pragma unroll 1
      for (int k = 0; k < cnt; ++k, ++n) {
        const int key = (cur.b + k) * PA_BN + kl;
        wait(smem_u32(&b_s[n & 1]), sp >> (n & 1) & 1);
        sp ^= 1 << (n & 1);
        __syncwarp();
        pa_fence_after();
        unsigned s[R];
        pf_ld<R>(tm + (n & 1) * N + lane_off, s);
        pa_wait_ld<R>(s);
        if (__builtin_expect(sight.partly((cur.b + k) * PA_BN), 0)) {
          sight.mask(p, key, s);
          if (sight.strange((cur.b + k) * PA_BN)) {
            // the values that nobody sees may be anything: zeros, so that 0 x NaN does not reach the sum
            const int place = 2 * n + 1, slot = place % NS;
            wait(smem_u32(&b_kfull[slot]), (place / NS) & 1);
            pa_zero_rows<Sh::CB>(sm_kv + slot * Sh::TILE, warp * 32, MODE == PA_SHARED ? s_valid.none(slot, kl, p) : sight.none(key));
            __syncwarp();
          }
        }
        bool over = false;
        if (k > 0) {
#pragma unroll
          for (int c = 0; c < R; ++c) over |= fmaf(__uint_as_float(s[c]), p.scale2, base[c]) > PA_LAZY + UP;
          if (MODE != PA_PLAIN && unset) {   // (the first logit that such a row sees is its reference, however far below zero)
#pragma unroll
            for (int c = 0; c < R; ++c) over |= (unset >> c & 1) && s[c] != 0xFF800000u;
          }
        }
        if (__builtin_expect(k == 0 || pf_or(over), 0)) {
          float m[R], f[R];
#pragma unroll
          for (int c = 0; c < R; ++c) m[c] = __uint_as_float(s[c]);
          const int col = pf_reduce<R>(m, larger);
          s_red[col][warp] = m[0];
          pf_sync();
#pragma unroll
          for (int c = 0; c < R; ++c) {
            const float4 w = *reinterpret_cast<const float4*>(s_red[c]);
            const float top = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) * p.scale2;
            // (a row that sees none of these keys keeps its reference; of a first block, any)
            const float nb = top == -INFINITY ? (k == 0 ? UP : base[c]) : UP - top;
            float use = k == 0 ? nb : fminf(base[c], nb);
            f[c] = k == 0 ? 1.f : ex2(use - base[c]);
            if constexpr (MODE != PA_PLAIN) {
              if (unset >> c & 1) {   // (its sums are zero)
                use = nb;
                f[c] = 1.f;
              }
              unset = top == -INFINITY ? (k == 0 ? unset | 1u << c : unset) : unset & ~(1u << c);
            }
            base[c] = use;
            sum[c] *= f[c];
          }
          if (k > 0) {
            wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);   // the P V before this block's
            __syncwarp();
            pa_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              unsigned o[R];
              const unsigned at = tm + Sh::TM_O + part * N + lane_off;
              pf_ld<R>(at, o);
              pa_wait_ld<R>(o);
#pragma unroll
              for (int c = 0; c < R; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              pf_st<R>(at, o);
            }
            pa_wait_st();
          }
          pf_sync();   // s_red may be written again
        }
        // (this S says that the P V two blocks ago is complete: its P may be overwritten)
        const int pb = n & 1;
        const unsigned long long sc2 = f2_pack(p.scale2, p.scale2);
#pragma unroll
        for (int c = 0; c < R; c += 8) {
          unsigned hi[4] = {}, lo[4] = {};
#pragma unroll
          for (int i = 0; i < (R < 8 ? R / 2 : 4); ++i) {
            const int a = c + 2 * i;
            const unsigned long long x =
                f2_fma((unsigned long long)s[a] | ((unsigned long long)s[a + 1] << 32), sc2, f2_pack(base[a], base[a + 1]));
            const float e0 = ex2(f2_lo(x)), e1 = ex2(f2_hi(x));
            sum[a] += e0;
            sum[a + 1] += e1;
            hi[i] = pa_pack<FP16>(e0, e1);
            const float2 r = pa_unpack<FP16>(hi[i]);
            lo[i] = pa_pack<FP16>(e0 - r.x, e1 - r.y);
          }
          // columns c .. c + 7 and N more of this key's row
          const unsigned h = pb * 4 + c / 8, l = h + N / 8;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + ((h ^ x7) << 4)), "r"(hi[0]), "r"(hi[1]),
                       "r"(hi[2]), "r"(hi[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + ((l ^ x7) << 4)), "r"(lo[0]), "r"(lo[1]),
                       "r"(lo[2]), "r"(lo[3])
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        pa_fence_before();
        __syncwarp();
        if (lane == 0) pa_arrive(smem_u32(&b_p[pb]));
      }

      // ------------------------------ the tile's end in this piece
      const int col = pf_reduce<R>(sum, plus);
      s_red[col][warp] = sum[0];
      pf_sync();
      const bool whole = cnt == cur.nb;
      const int ntok = cur.tokens(p), rows = ntok * p.G;
      const long long part = (long long)blockIdx.x * 2 + (cur.b == 0 ? 1 : 0);
      if (kl < rows) {   // a thread per row
        const int row = kl;
        float ref = 0.f;   // (of the sums: UP below the reference)
#pragma unroll
        for (int c = 0; c < R; ++c)
          if (c == kl) ref = -base[c];
        const float4 w = *reinterpret_cast<const float4*>(s_red[row]);
        const float all = w.x + w.y + w.z + w.w;
        s_inv[row] = all == 0.f ? 0.f : 1.f / all;
        if (!whole) {
          p.part_ml[part * 128 + row] = make_float2(all == 0.f ? -INFINITY : ref, all);
        } else if (p.lse) {
          const int t = row / p.G;
          p.lse[(long long)(cur.tok(p) + t) * p.Hq + cur.head() * p.G + (row - t * p.G)] =
              all == 0.f ? -INFINITY : (ref + UP + log2f(all * PA_DOWN<FP16>)) * 0.69314718055994531f;
        }
      }
      pf_sync();
      wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);
      __syncwarp();
      pa_fence_after();
      // a thread has a channel: lane of O (64 channels: sixteen to a warp)
      const int chan = D == 128 ? kl : warp * 16 + lane;
      const bool have = D == 128 || lane < 16;
      unsigned o[R], l[R];
      pf_ld<R>(tm + Sh::TM_O + lane_off, o);
      pf_ld<R>(tm + Sh::TM_O + N + lane_off, l);
      pa_wait_ld<R>(o);
      pa_wait_ld<R>(l);
      uint16_t* dst = p.out + (long long)cur.tok(p) * p.ots + (long long)cur.head() * p.G * p.ohs + chan;
      float* po = p.part_o + (part * (D / 4) + chan / 4) * 512 + chan % 4;
      int g = 0;
      unsigned strange = 0;
#pragma unroll
      for (int c = 0; c < R; ++c)
        if (c < rows) {
          const float x = __uint_as_float(o[c]) + __uint_as_float(l[c]);
          if (have && whole) {
            const unsigned y = pa_pack<FP16>(x * s_inv[c], 0.f);
            *dst = (uint16_t)y;
            if (MODE == PA_SHARED) strange |= pa_strange<FP16, 1>(&y);
          }
          if (have && !whole) po[c * 4] = x;
          dst += p.ohs;
          if (++g == p.G) {
            g = 0;
            dst += p.ots - p.G * p.ohs;
          }
        }
      if (MODE == PA_SHARED && strange) pages_report(p.pg, QE_PAGES_ERR_VALUE);
      pa_fence_before();
      pf_sync();   // O and the sums are read whole before the next tile's
    }
  }
  if constexpr (MODE == PA_SHARED)
    if (aux == 2 && pa_checks_shared(p)) pa_check_shared(p);
  __syncthreads();
  if (aux == 3) {
    pa_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(Sh::TM_COLS) : "memory");
  }
}

}  // namespace qe
