// qe_pages_halves.cuh -- attention of a chunk of new tokens over the cached pages, on the 5th-generation
// tensor cores (tcgen05.mma, operands by TMA, accumulators and probabilities in tensor memory).
//
// For the row of token t (of a chunk of m) and query head h, with V visible keys (causal: kv_len - m + t + 1):
//   out = sum_i 2^(x_i - M) v_i / sum_i 2^(x_i - M),   x_i = scale log2(e) q . k_i,
// in one pass over the keys in blocks of 128 with a running reference M, sum and accumulator in float32.
//
// Tiles.  A tile is NH halves of 128 rows: T tokens x the G query heads of one KV head per half (row t G + g,
// T = floor(128 / G)), so a block's keys and values are read once for all of them.  NH = 2 for chunks: while one half's
// softmax runs, the other half's products keep the tensor cores busy.  NH = 1 where a chunk's rows fit one half (drafts): bound by
// the memory the cache is read from, so one half and the S buffers of both to run ahead.  (At most 16 rows: qe_pages_few.cuh.)
//
// Split.  All (tile, block) pairs of the call form one line, cut into equal pieces, one per CTA (one CTA per SM): long
// caches with few rows are split along the keys, prompts are balanced whatever their causal shape.  A tile inside a piece is
// finished by its CTA; one that is cut leaves (M, sum, accumulator) parts that the join kernel merges.  The line is computed
// from the lengths on the device by every CTA alike (a sum of floors in closed form per sequence).
//
// CTA: 8 softmax warps per half, two threads per row (one for each 64 keys of a block: the softmax of a half has to fit under
// the products of the other), then a warp each for TMA of keys and values (page by page, into a ring of slots), tensor-core
// issue of half 0 and of half 1, and TMA of the queries.
//  * S = Q K^T (M 128, N 128): both operands in shared memory, 128-byte swizzle, K-major.
//  * P overwrites its S in tensor memory in the pool's type; O += P V (N = head_dim) takes P from there and V as the
//    MN-major operand (its rows are tokens).
//  * The reference M is raised only when a row's maximum passes it by 2^8 (then the softmax warps rescale O in tensor
//    memory); up to that P and the sums are larger than 1, exactly as precise.
//  * P is rounded to the pool's type (the tensor cores' operand): off by half a step at most, as the result itself is, but for fp16 by
//    2^-32 of the reference's weight where that is more (P is taken 2^7 times as large, or it would be 2^-25); the sum is of the
//    unrounded ones.  With NH = 1, where the tensor cores wait for memory anyway, what the rounding leaves is kept as
//    a second operand and multiplied too: error against 64 bits 1.45 -> 1.0 times that of the result's own rounding.
//    REST: with two halves of shared prefixes too, where the caller says that the chunks are short (a block of both halves then has one and a
//    half times the products and takes 2.0 us where reading it takes 1.4: 64 sequences behind a 32K prefix 69 -> 79 us, error 2.2e-3 -> 1.7e-3).
// mbarriers.  Every wait is bounded, by 0.2 s and 10 us for each block that it may sit out; one that expires sets QE_PAGES_ERR_TIMEOUT
// and an abort flag that ends all loops, and the CTA leaves after what it issued has landed: each warp that issues waits for its own
// last, whether it or another warp gave up.
//  * kfull / kempty per slot, qfull / qempty per query buffer, s[i]: S i complete (tensor-core commit);
//  * p[i][c]: part c of P i written (so many of each 64 keys), one arrival per softmax warp (the products of the first part start while
//    the softmax is at the others: 32K chunk 705 -> 682 us with two parts);
//  * o[h]: half h's O of a tile complete; with NH = 1 o[i]: the P V of an even or odd block complete (an S tells only that the P V two
//    blocks before is, so one barrier's parity could mean the last P V or the one before);
//  * turn[h]: half h may issue.
#pragma once
#include "qe_pages_walk.cuh"

namespace qe {

// Parts that a block's probabilities are handed over in.  Four with two halves (512 tokens over 8K 54.7 -> 53.1 us against two, 64-channel
// chunk 491 -> 485); with one half, where a part more is a wait more for two stores, 64-channel drafts take 105 us with four and 92 with two.
template <int NH>
constexpr int PA_PARTS = NH == 2 ? 4 : 2;

// Keys and values sent by a warp each: with 64 channels, where what copies cost bounds small pages (PfShape), if one of the 4 warps
// is free for it (a fifth would leave the softmax of two halves 80 registers).
template <int D, int NH>
constexpr bool PA_SPLIT = D == 64 && NH == 1;
// threads: 8 softmax warps per half, 4 more warps
template <int NH>
constexpr int PA_THREADS = 256 * NH + 128;

template <int D>
struct PaShape {
  static constexpr int CB = D / 64;              // column blocks of 128 bytes
  static constexpr int TILE = 128 * D * 2;       // a query buffer, or a slot: 128 rows
  static constexpr int ALL = 7 * 32768;          // query buffers and slots together
  static constexpr int MOST = (ALL - TILE) / TILE;
  static constexpr int SMEM = ALL + 1024;
  // Slots beside two query buffers of `rows` rows (64 where a tile has no more, else 128; the products of rows behind read what
  // lies there and are not used): bound by memory, the ring's depth is what counts.
  // (with 64 channels an even number, for keys and values with slots of their own)
  static constexpr int slots(int rows) { return (ALL - 2 * CB * rows * 128) / (TILE * (3 - CB)) * (3 - CB); }
  static constexpr int TM_O = 256;               // tensor memory: S0 at column 0, S1 at 128, O0 here, O1 at + D
};

// the two warps of a row: barrier, and barrier with the OR of a truth value
__device__ __forceinline__ void pa_pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pa_pair_or(int id, bool v) {
  unsigned r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbar.red.or.pred p, %2, 64, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((unsigned)v), "r"(id)
      : "memory");
  return r != 0;
}

// D / 2 columns of 16 lanes: register 4 j + e is (lane T / 4, column 8 j + 2 (T mod 4) + e), 4 j + 2 + e the same of lane 8 + T / 4
template <int D>
__device__ __forceinline__ void pa_ld_rows(unsigned t, unsigned* r) {
  if constexpr (D == 128)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
// Among four lanes: u[K q + k] of lane t (q, t < 4, k < K) becomes u[4 k + t] of lane q.
template <int K>
__device__ __forceinline__ void pa_quad_transpose(unsigned* u) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    const bool odd = lane & s;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (!(q & s))
#pragma unroll
        for (int k = 0; k < K; ++k) {
          unsigned &a = u[K * q + k], &b = u[K * (q + s) + k];
          const unsigned got = __shfl_xor_sync(~0u, odd ? a : b, s);
          if (odd) a = got;
          else b = got;
        }
  }
  if constexpr (K == 2) {   // (lane, k) -> (k, lane)
    const unsigned x[8] = {u[0], u[2], u[4], u[6], u[1], u[3], u[5], u[7]};
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = x[i];
  }
}
// ---------------------------------------------------------------------------- the kernel

template <int D, int NH, bool FP16, int MODE, bool REST>
__global__ void __launch_bounds__(PA_THREADS<NH>, 1)
    pages_attend_kernel(const __grid_constant__ PaParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv) {
  using Sh = PaShape<D>;
  using Cursor = typename PaWalk<NH, MODE>::Cursor;
  constexpr int PARTS = PA_PARTS<NH>;
  const int NS = NH == 1 && p.q_rows == 64 ? Sh::slots(64) : Sh::slots(128);
  const int q_cb = (NH == 1 ? p.q_rows : 128) * 128, q_buf = Sh::CB * q_cb;   // bytes of a query buffer's column block, and of the buffer
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long b_kfull[Sh::MOST], b_kempty[Sh::MOST], b_qfull[2], b_qempty[2], b_s[2], b_p[2][PARTS], b_o[2], b_turn[2], b_end;
  __shared__ unsigned s_tmem;
  __shared__ int s_abort;
  __shared__ typename PaWalk<NH, MODE>::Place s_place[PaWalk<NH, MODE>::PLACES];
  __shared__ long long s_w[PA_THREADS<NH> / 32];
  __shared__ float s_x[NH][128];      // what the two threads of a row tell each other
  __shared__ PaValid<MODE, Sh::MOST> s_valid;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0), aux = warp - 8 * NH;   // aux: TMA, tensor cores of half 0 and 1, queries
  const unsigned sm = (smem_u32(smem_raw) + 1023) & ~1023u;
  const unsigned sm_q = sm, sm_kv = sm + 2 * q_buf;
  const PaWait wait{&p.pg, &s_abort};

  if (aux == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&b_kfull[i]), 1);
      mbar_init(smem_u32(&b_kempty[i]), NH);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&b_qfull[i]), 1);
      mbar_init(smem_u32(&b_qempty[i]), 1);
      mbar_init(smem_u32(&b_s[i]), 1);
      for (int c = 0; c < PARTS; ++c) mbar_init(smem_u32(&b_p[i][c]), 8);
      mbar_init(smem_u32(&b_o[i]), 1);
      mbar_init(smem_u32(&b_turn[i]), 1);
    }
    mbar_init(smem_u32(&b_end), NH);
    mbar_fence_init();
    s_abort = 0;
  }
  pa_fence_before();
  griddep_wait();
  griddep_launch_dependents();   // (what follows may then rely on all that ran before this launch)
  static_assert(1024 + 4 * pa_find_ints(PA_THREADS<NH>) <= Sh::ALL, "the cuts' space is in the ring");
  const bool work = PaWalk<NH, MODE>::template find<PA_THREADS<NH>>(p, s_place, s_w, reinterpret_cast<int*>(smem_raw) + 256);   // ends with a barrier
  pa_fence_after();
  const unsigned tm = s_tmem;

  if (aux >= 0) {
    if (NH == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    constexpr bool SPLIT = PA_SPLIT<D, NH>;
    if (work && (aux == 0 || (SPLIT && aux == 2))) {
      // ============================== keys and values, or one of them
      const int kv0 = SPLIT && aux != 0;
      constexpr int STEP = SPLIT ? 2 : 1;
      Cursor cur;
      cur.set(p, s_place);
      const PaCopy<Sh::CB> copy(p);
      // this lane's piece, its entry loaded a block before it is looked at
      typename PaWalk<NH, MODE>::Keys keys;
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
    } else if (work && aux - 1 < NH) {
      // ============================== tensor cores: a warp per half, so that the waits and the issue of one half pass while
      // the products of the other run.  The whole warp walks the loop (addresses and descriptors stay uniform), one lane issues.
      const int h = aux - 1;
      constexpr unsigned FMT = FP16 ? 0u : (1u << 7) | (1u << 10);
      constexpr unsigned ID_S = (1u << 4) | FMT | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      constexpr unsigned ID_O = (1u << 4) | FMT | (1u << 16) | (((unsigned)D >> 3) << 17) | ((128u >> 4) << 24);
      Cursor cur;
      cur.set(p, s_place);
      // The ring is consumed in its order: K 0, then V n - 1 and K n in turn.
      int slot = 0, ph = 0, pp = 0, qp = 0, tile = 0, left = 0;   // (bit i of pp, qp: the parity of p[i], qfull[i])
      int till = PaWait::counted(p, PaWait::PRODUCTS);
      int at = 0, all = 0, done = 0;   // (shared: the block; how many of the tile's are for this half, and how many of them were before)
      bool was_first = false, was_last = false, was_mine = false, mine = false, ok = true, more = true;
      auto step = [&]() {
        if (++slot == NS) {
          slot = 0;
          ph ^= 1;
        }
      };
      const unsigned t_o = tm + Sh::TM_O + h * D;
      auto qk = [&](int qb, int sb, int kslot, bool q_done) {   // S sb = Q qb K^T (by one lane)
        const unsigned long long a = PA_DESC_Q | ((sm_q + qb * q_buf) >> 4), b = PA_DESC_K<Sh::CB> | ((sm_kv + kslot * Sh::TILE) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const unsigned o = ((k >> 2) * PA_CELL + (k & 3) * 32) >> 4, oq = ((k >> 2) * q_cb + (k & 3) * 32) >> 4;
          if (NH == 2 && k == D / 16 - 2) pa_arrive(smem_u32(&b_turn[h ^ 1]));   // (its first product is issued by when these are done)
          pa_mma_ss(tm + sb * 128, a + oq, b + o, ID_S, k > 0);
        }
        pa_commit(smem_u32(&b_s[sb]));
        pa_commit(smem_u32(&b_kempty[kslot]));
        if (q_done) pa_commit(smem_u32(&b_qempty[qb]));
      };
      // O += P sb V over one part of each 64 keys (by one lane)
      auto pv = [&](int part, int sb, int vslot, bool acc) {
        const unsigned long long b = PA_DESC_V<Sh::CB> | ((sm_kv + vslot * Sh::TILE) >> 4);
        constexpr int KS = 4 / PARTS;   // steps of 16 keys of a part of 64
#pragma unroll
        for (int rest = 0; rest < (REST ? 2 : 1); ++rest)   // (with the remainders of P)
#pragma unroll
          for (int i = 0; i < 2 * KS; ++i) {
            const int k = i / KS * 4 + part * KS + i % KS;
            pa_mma_ts(t_o, tm + sb * 128 + rest * 64 + k * 8, b + k * 128 * Sh::CB, ID_O, acc || rest > 0 || i > 0);
          }
      };
#pragma unroll 1
      for (int n = 0; more; ++n) {
        bool first = left == 0;
        if (first) {
          if (n > 0) cur.next_tile(p);
          left = cur.count();
          more = left > 0;      // one more round for the last P V
          mine = h == 0 || cur.second_half(p);
          if constexpr (MODE == PA_SHARED && NH == 2) {
            at = cur.b;
            all = more && mine ? cur.count_for(h) : 0;
            done = 0;
          }
        }
        bool last = left == 1;
        if constexpr (MODE == PA_SHARED && NH == 2) {   // of the blocks that are for this half
          mine = more && all > 0 && cur.is_for(h, at++);
          first = mine && done == 0;
          done += mine;
          last = mine && done == all;
        }
        const int vslot = slot;
        if constexpr (NH == 2) {
          // what has to be there: values, keys and queries, long before the probabilities
          if (n > 0) {
            ok = ok && wait(smem_u32(&b_kfull[slot]), ph);
            step();
          }
          if (more) {
            ok = ok && wait.count(till, smem_u32(&b_kfull[slot]), ph);
            if (first && mine) {
              ok = ok && wait(smem_u32(&b_qfull[h]), qp & 1);
              qp ^= 1;
            }
          }
          if (!__all_sync(~0u, ok)) break;
          const bool do_pv = n > 0 && was_mine, do_qk = more && mine;
          // The halves take turns, products of a half in one go: one half's softmax runs under the other's products.  (Left
          // to themselves they interleave, and both softmaxes and then both halves' products run at the same time.)
          ok = wait(smem_u32(&b_turn[h]), (n & 1) ^ h ^ 1);
          if (do_pv) {
#pragma unroll
            for (int c = 0; c < PARTS - 1; ++c) {
              ok = wait(smem_u32(&b_p[h][c]), pp) && ok;
              pa_fence_after();
              if (pa_elect()) pv(c, h, vslot, c > 0 || !was_first);
              __syncwarp();
            }
            ok = wait(smem_u32(&b_p[h][PARTS - 1]), pp) && ok;
            pp ^= 1;
          }
          pa_fence_after();
          if (pa_elect()) {
            if (do_pv) {
              pv(PARTS - 1, h, vslot, true);
              if (was_last) pa_commit(smem_u32(&b_o[h]));
              pa_commit(smem_u32(&b_kempty[vslot]));
            } else if (n > 0) {
              pa_arrive(smem_u32(&b_kempty[vslot]));
            }
            if (do_qk) qk(h, h, slot, last);
            else if (more) pa_arrive(smem_u32(&b_kempty[slot]));
            if (!do_qk) pa_arrive(smem_u32(&b_turn[h ^ 1]));
          }
          __syncwarp();
          if (more) step();
        } else {
          // S runs a block ahead: K n before V n - 1 and P n - 1
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
            if (pa_elect()) qk(qb, n & 1, kslot, last);
            __syncwarp();
            if (last) ++tile;
          }
          if (n > 0) {
            const int sb = (n - 1) & 1;
            ok = ok && wait(smem_u32(&b_kfull[vslot]), ph);
            ok = ok && wait(smem_u32(&b_p[sb][0]), pp >> sb & 1);
            if (!__all_sync(~0u, ok)) break;
#pragma unroll
            for (int c = 0; c < PARTS - 1; ++c) {
              if (c > 0) ok = wait(smem_u32(&b_p[sb][c]), pp >> sb & 1) && ok;
              pa_fence_after();
              if (pa_elect()) pv(c, sb, vslot, c > 0 || !was_first);
              __syncwarp();
            }
            ok = wait(smem_u32(&b_p[sb][PARTS - 1]), pp >> sb & 1) && ok;
            pp ^= 1 << sb;
            pa_fence_after();
            if (pa_elect()) {
              pv(PARTS - 1, sb, vslot, true);
              pa_commit(smem_u32(&b_kempty[vslot]));
              pa_commit(smem_u32(&b_o[sb]));
            }
            __syncwarp();
            step();
          }
          if (more) step();
        }
        was_first = first;
        was_last = last;
        was_mine = mine;
        --left;
      }
      if (pa_elect()) pa_commit(smem_u32(&b_end));   // everything issued is complete before tensor memory goes
      __syncwarp();
      wait.drain(smem_u32(&b_end), 0);
    } else if (work && aux == 3) {
      // ============================== queries (one lane; the walk over groups takes the warp)
      Cursor cur;
      cur.set(p, s_place);
      PaFill fill[2];
      int tile = 0, blocks = 0, till = PaWait::counted(p, PaWait::QUERIES);   // (blocks: of the tiles before)
      bool ok = true;
      auto send = [&]() {
        const int halves = cur.second_half(p) ? 2 : 1;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          if constexpr (MODE == PA_SHARED && NH == 2)
            if (cur.count_for(h) == 0) continue;
          const int qb = NH == 2 ? h : tile & 1;
          ok = wait.count(till, smem_u32(&b_qempty[qb]), fill[qb].empty(), blocks);
          if (!ok) break;
          const unsigned full = smem_u32(&b_qfull[qb]);
          mbar_expect_tx(full, p.T * p.G * 128 * Sh::CB);
          for (int cb = 0; cb < Sh::CB; ++cb)
            pa_tma3(sm_q + qb * q_buf + cb * q_cb, &mq, cb * 64, cur.head() * p.G, cur.tok(p) + h * p.T, full);
          ++fill[qb].sent;
        }
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
    }
  } else {
    if (NH == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int half = warp >> 3;
    if (work) {
      // ============================== softmax: a row of the half and one half of a block's keys
      const int w4 = warp & 3, ch = (warp >> 2) & 1, r = w4 * 32 + lane;
      const unsigned lane_off = (unsigned)(w4 * 32) << 16;
      const unsigned t_o = tm + Sh::TM_O + half * D + ch * (D / 2) + lane_off;   // this thread's half of O's columns
      const int pair = 1 + half * 4 + w4;                 // named barrier of the two warps of these rows
      Cursor cur;
      cur.set(p, s_place);
      const int rt = r / p.G, rg = r - rt * p.G;
      int sp = 0, tiles = 0, n = 0;   // (bit i of sp: the parity of s[i])
      auto together = [&](float x, auto op) {   // op of the row's two values, the same for both threads
        if (ch) s_x[half][r] = x;
        pa_pair_sync(pair);
        if (!ch) s_x[half][r] = x = op(x, s_x[half][r]);
        pa_pair_sync(pair);
        return ch ? s_x[half][r] : x;
      };
      // A wait that fails (the CTA is leaving) lets the loops run out without waiting, so that the pairs' barriers stay in step.
#pragma unroll 1
      for (int cnt; (cnt = cur.count()) > 0;) {
        if (NH == 2 && half == 1 && !cur.second_half(p)) {
          n += cnt;
          cur.next_tile(p);
          continue;
        }
        const int t = half * p.T + rt;                    // token of the tile
        const bool live = rt < p.T && t < cur.tokens(p);
        const bool any_live = __any_sync(~0u, live);
        const bool whole = cnt == cur.nb;
        const long long part = ((long long)blockIdx.x * 2 + (cur.b == 0 ? 1 : 0)) * NH + half;
        if constexpr (MODE == PA_SHARED && NH == 2)
          if (cur.count_for(half) == 0) {   // (whole tiles have blocks for both)
            if (live && ch == 0) p.part_ml[part * 128 + r] = make_float2(-INFINITY, 0.f);
            n += cnt;
            cur.next_tile(p);
            continue;
          }
        // from this thread's half of the first block on (shared: of the stream)
        const PaSight<NH, MODE> sight(p, cur, half, t, live, any_live, (MODE == PA_SHARED ? 0 : cur.b * PA_BN) + ch * 64);
        bool begun = false;
        float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int k = 0; k < cnt; ++k, ++n) {
          int at = k * PA_BN;
          if constexpr (MODE == PA_SHARED)
            if (const int z = cur.block(cur.b + k, at); NH == 2 && cur.b + k >= cur.np && z != half) continue;
          const bool begin = MODE == PA_SHARED ? !begun : k == 0;
          begun = true;
          const int sb = NH == 2 ? half : n & 1;
          wait(smem_u32(&b_s[sb]), sp >> sb & 1, NH == 2 ? n : 0);   // (half 1 may have sat out tiles before)
          sp ^= 1 << sb;
          __syncwarp();
          pa_fence_after();
          const unsigned t_s = tm + sb * 128 + lane_off;
          if (__builtin_expect(sight.strange(at) && ch == 0, 0)) {
            // the values that nobody sees may be anything: zeros, so that 0 x NaN does not reach the sum
            const int place = 2 * n + 1, slot = place % NS;
            wait(smem_u32(&b_kfull[slot]), (place / NS) & 1);
            if (MODE == PA_SHARED ? s_valid.none(slot, r, p) : sight.none(at + r)) {
              const unsigned row = sm_kv + slot * Sh::TILE + pa_slot_row<Sh::CB>(r);
#pragma unroll 1
              for (int cb = 0; cb < Sh::CB; ++cb)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + cb * PA_CELL + e * 16), "r"(0) : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          if (MODE == PA_SHARED && any_live && sight.nothing(at, ch * 64)) {
            // nothing of the block is for these rows (both warps of a row say so): probabilities of zero
            unsigned z[16] = {};
            pa_st16(t_s + ch * 32, z);
            pa_st16(t_s + ch * 32 + 16, z);
            if (REST) {
              pa_st16(t_s + 64 + ch * 32, z);
              pa_st16(t_s + 64 + ch * 32 + 16, z);
            }
            pa_wait_st();
            pa_fence_before();
            __syncwarp();
            if (lane == 0)
              for (int c = 0; c < PARTS - 1; ++c) pa_arrive(smem_u32(&b_p[sb][c]));
          } else if (any_live) {
            unsigned s[64];
            pa_ld32(t_s + ch * 64, s);
            pa_ld32(t_s + ch * 64 + 32, s + 32);
            pa_wait_ld<64>(s);
            if (__builtin_expect(sight.partly(at), 0)) sight.mask(at, s);
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4]));
#pragma unroll
            for (int c = 8; c < 64; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[c + e])), __uint_as_float(s[c + 4 + e]));
            float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (__builtin_expect(begin || pa_pair_or(pair, live && (m - ref) * p.scale2 > PA_LAZY), 0)) {
              m = together(fmaxf(m, ref), [](float a, float b) { return fmaxf(a, b); });
              const float f = m == -INFINITY ? 1.f : ex2((ref - m) * p.scale2);
              ref = m;
              if (!begin) {
                sum *= f;
                if constexpr (NH == 1) {   // the P V before this block's may still be running
                  wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);
                  __syncwarp();
                  pa_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 16) {
                  unsigned o[16];
                  pa_ld16(t_o + c, o);
                  pa_wait_ld<16>(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  pa_st16(t_o + c, o);
                }
                pa_wait_st();
                pa_fence_before();
                pa_pair_sync(pair);   // O is scaled whole before either half of the keys is handed over
              }
            }
            const float base = PA_UP<FP16> - (ref == -INFINITY ? 0.f : ref * p.scale2);
            const unsigned long long sc2 = f2_pack(p.scale2, p.scale2), ba2 = f2_pack(base, base);
            unsigned long long acc[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < PARTS; ++c) {
              constexpr int N = 32 / PARTS;   // pairs of keys
              unsigned pk[N], rest[N];
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const unsigned long long x =
                    f2_fma((unsigned long long)s[2 * (c * N + e)] | ((unsigned long long)s[2 * (c * N + e) + 1] << 32), sc2, ba2);
                const float e0 = ex2(f2_lo(x)), e1 = ex2(f2_hi(x));
                acc[e & 1] = f2_add(acc[e & 1], f2_pack(e0, e1));
                pk[e] = pa_pack<FP16>(e0, e1);
                if (REST) {
                  const float2 r = pa_unpack<FP16>(pk[e]);
                  const unsigned long long d = f2_sub(f2_pack(e0, e1), f2_pack(r.x, r.y));
                  rest[e] = pa_pack<FP16>(f2_lo(d), f2_hi(d));
                }
              }
              if constexpr (NH == 1) {
                pa_st16(t_s + ch * 32 + c * N, pk);
                pa_st16(t_s + 64 + ch * 32 + c * N, rest);
              } else {
                pa_st8(t_s + ch * 32 + c * N, pk);
                if (REST) pa_st8(t_s + 64 + ch * 32 + c * N, rest);
              }
              if (c < PARTS - 1) {   // the products of these may start
                pa_wait_st();
                pa_fence_before();
                __syncwarp();
                if (lane == 0) pa_arrive(smem_u32(&b_p[sb][c]));
              }
            }
            const unsigned long long a = f2_add(acc[0], acc[1]);
            sum += f2_lo(a) + f2_hi(a);
            pa_wait_st();
          } else {
            if (lane == 0)
              for (int c = 0; c < PARTS - 1; ++c) pa_arrive(smem_u32(&b_p[sb][c]));
          }
          pa_fence_before();
          __syncwarp();
          if (lane == 0) pa_arrive(smem_u32(&b_p[sb][PARTS - 1]));
        }

        // ------------------------------ the tile's end in this piece
        const int tok = cur.tok(p) + t, head = cur.head() * p.G + rg;
        cur.next_tile(p);   // (while the last products run: 256 samples 66.5 -> 64.3 us, 2048 tokens over 32K 617 -> 606, prompts under a window 217 -> 219)
        if (NH == 2) wait(smem_u32(&b_o[half]), tiles & 1);
        else wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);
        ++tiles;
        __syncwarp();
        pa_fence_after();
        if (any_live) {
          sum = together(sum, [](float a, float b) { return a + b; });
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          if (whole) {
            // four lanes write a row's 128 (64) bytes side by side, eight rows a store: with a row per lane a store touches 32
            // lines, and what follows queues behind it (prompts 132 -> 129 us)
            const unsigned long long at = live ? reinterpret_cast<unsigned long long>(p.out + tok * p.ots + head * p.ohs + ch * (D / 2)) : 0ull;
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              unsigned o[D / 4];
              pa_ld_rows<D>(t_o + ((unsigned)(16 * g) << 16), o);
              pa_wait_ld<D / 4>(o);
#pragma unroll
              for (int up = 0; up < 2; ++up) {
                const int from = 16 * g + 8 * up + (lane >> 2);
                const float f = __shfl_sync(~0u, inv, from);
                const unsigned long long to = __shfl_sync(~0u, at, from);
                unsigned u[D / 16];                       // unit j: channels 8 j + 2 (lane mod 4), + 1
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                  u[j] = pa_pack<FP16>(__uint_as_float(o[4 * j + 2 * up]) * f, __uint_as_float(o[4 * j + 2 * up + 1]) * f);
                if (MODE == PA_SHARED && to && pa_strange<FP16, D / 16>(u)) pages_report(p.pg, QE_PAGES_ERR_VALUE);
                pa_quad_transpose<D / 64>(u);
                if (to) {
                  uint16_t* dst = reinterpret_cast<uint16_t*>(to) + (lane & 3) * (D / 8);
                  if constexpr (D == 128) pa_store32(dst, u);
                  else *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
                }
              }
            }
          } else {
            float* po = p.part_o + (part * (D / 4) + ch * (D / 8)) * 512 + r * 4;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
              unsigned o[32];
              pa_ld32(t_o + c, o);
              pa_wait_ld<32>(o);
              if (live && (MODE != PA_SHARED || sum != 0.f))   // (the join leaves out a part without a sum)
#pragma unroll
                for (int e = 0; e < 8; ++e)       // four channels of 32 rows side by side
                  *reinterpret_cast<uint4*>(po + (c / 4 + e) * 512) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          if (live && whole && p.lse && ch == 0) p.lse[(long long)tok * p.Hq + head] = sum == 0.f ? -INFINITY : ref * p.scale + logf(sum * PA_DOWN<FP16>);
          if (live && !whole && ch == 0) p.part_ml[part * 128 + r] = make_float2(sum == 0.f ? -INFINITY : ref * p.scale2 - PA_UP<FP16>, sum);
          pa_fence_before();
          pa_pair_sync(pair);   // O is read whole before the next tile's first P is handed over
        }
      }
    }
  }
  if constexpr (MODE == PA_SHARED)
    if (aux == 3 && pa_checks_shared(p)) pa_check_shared(p);
  __syncthreads();
  if (aux == 3) {
    pa_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

}  // namespace qe
