// qe_pages_attn.cu -- attention of a chunk of new tokens over the cached pages, on the 5th-generation
// tensor cores (tcgen05.mma, operands by TMA, accumulators and probabilities in tensor memory).
//
// For the row of token t (of a chunk of m) and query head h, with V visible keys (causal: kv_len - m + t + 1):
//   out = sum_i 2^(x_i - M) v_i / sum_i 2^(x_i - M),   x_i = scale log2(e) q . k_i,
// in one pass over the keys in blocks of 128 with a running reference M, sum and accumulator in float32.
//
// Tiles.  A tile is NH halves of 128 rows: T tokens x the G query heads of one KV head per half (row t G + g,
// T = floor(128 / G)), so a block's keys and values are read once for all of them.  NH = 2 for chunks: while one half's
// softmax runs, the other half's products keep the tensor cores busy.  NH = 1 where a chunk's rows fit one half (drafts): bound by
// the memory the cache is read from, so one half and the S buffers of both to run ahead.  (At most 16 rows: qe_pages_few.cu.)
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
// mbarriers.  Every wait is bounded, by 0.2 s and 10 us for each block that it may sit out; one that expires sets QE_PAGES_ERR_TIMEOUT
// and an abort flag that ends all loops, and the CTA leaves after what it issued has landed: each warp that issues waits for its own
// last, whether it or another warp gave up.
//  * kfull / kempty per slot, qfull / qempty per query buffer, s[i]: S i complete (tensor-core commit);
//  * p[i][c]: part c of P i written (so many of each 64 keys), one arrival per softmax warp (the products of the first part start while
//    the softmax is at the others: 32K chunk 705 -> 682 us with two parts);
//  * o[h]: half h's O of a tile complete; with NH = 1 o[i]: the P V of an even or odd block complete (an S tells only that the P V two
//    blocks before is, so one barrier's parity could mean the last P V or the one before);
//  * turn[h]: half h may issue.
#include <atomic>

#include "qe_pages_attn.cuh"

namespace qe {

// Parts that a block's probabilities are handed over in.  Four with two halves (512 tokens over 8K 54.7 -> 53.1 us against two, 64-channel
// chunk 491 -> 485); with one half, where a part more is a wait more for two stores, 64-channel drafts take 105 us with four and 92 with two.
template <int NH>
constexpr int PA_PARTS = NH == 2 ? 4 : 2;

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
  static constexpr int slots(int rows) { return (ALL - 2 * CB * rows * 128) / TILE; }
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

template <int D, int NH, bool FP16>
__global__ void __launch_bounds__(PA_THREADS<NH>, 1)
    pages_attend_kernel(const __grid_constant__ PaParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv) {
  using Sh = PaShape<D>;
  constexpr int PARTS = PA_PARTS<NH>;
  const int NS = NH == 1 && p.q_rows == 64 ? Sh::slots(64) : Sh::slots(128);
  const int q_cb = (NH == 1 ? p.q_rows : 128) * 128, q_buf = Sh::CB * q_cb;   // bytes of a query buffer's column block, and of the buffer
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long b_kfull[Sh::MOST], b_kempty[Sh::MOST], b_qfull[2], b_qempty[2], b_s[2], b_p[2][PARTS], b_o[2], b_turn[2], b_end;
  __shared__ unsigned s_tmem;
  __shared__ int s_abort;
  __shared__ PaPlace s_place[2];
  __shared__ long long s_w[PA_THREADS<NH> / 32];
  __shared__ float s_x[NH][128];      // what the two threads of a row tell each other

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
  pa_find<NH, PA_THREADS<NH>>(p, s_place, s_w);   // ends with a barrier
  pa_fence_after();
  const unsigned tm = s_tmem;
  // (two cuts that fall into the same place leave an empty piece)
  const bool work = s_place[0].i < p.c.n && (s_place[0].i != s_place[1].i || s_place[0].h != s_place[1].h || s_place[0].j != s_place[1].j ||
                                             s_place[0].b != s_place[1].b);

  if (aux >= 0) {
    if (NH == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (work && aux == 0) {
      // ============================== keys and values
      PaCursor<NH> cur;
      cur.set(p, s_place);
      const int rows = min(p.pg.S, PA_BN);               // tokens of a piece: a page, or a block's part of one
      const int np = PA_BN / rows;
      const int piece = lane % np, cb = lane / np;       // lane -> (page of the block, column block)
      const bool mine = cb < Sh::CB;
      // the table's entry for this lane's piece (INT_MIN behind the sequence's end), loaded a block before it is looked at
      auto entry = [&]() {
        const int key = cur.b * PA_BN + piece * rows;
        return key < cur.q.s.len ? p.t.table[(long long)cur.q.s.row * p.t.stride + (key >> p.pg.lgS)] : INT_MIN;
      };
      int slot = 0, ph = 1, issued = 0, left = cur.count();
      int next = entry(), till = PaWait::counted(p, PaWait::KEYS);
      bool ok = true;
#pragma unroll 1
      while (left > 0 && ok) {
        const int tk = (cur.b * PA_BN) & (p.pg.S - 1), h = cur.h;
        const bool there = next >= 0 && next < p.pg.P;
        const int now = there ? next : p.pg.P;             // out of the pool: the copy fills zeros
        if (!there && next != INT_MIN) pages_report(p.pg, QE_PAGES_ERR_PAGE);
        ++cur.b;
        if (--left == 0) {
          cur.next_tile(p);
          left = cur.count();
        }
        if (left > 0) next = entry();
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && wait.count(till, smem_u32(&b_kempty[slot]), ph);
          if (!__all_sync(~0u, ok)) {
            ok = false;
            break;
          }
          const unsigned full = smem_u32(&b_kfull[slot]);
          if (lane == 0) mbar_expect_tx(full, Sh::TILE);
          __syncwarp();
          if (mine) pa_tma4(sm_kv + slot * Sh::TILE + cb * 16384 + piece * rows * 128, kv ? &mv : &mk, cb * 64, tk, h, now, full);
          ++issued;
          if (++slot == NS) {
            slot = 0;
            ph ^= 1;
          }
        }
      }
      if (lane == 0)   // the copies land before the CTA leaves (early, it may be, and for another warp's wait)
        for (int i = max(0, issued - NS); i < issued; ++i) wait.drain(smem_u32(&b_kfull[i % NS]), (i / NS) & 1);
    } else if (work && aux - 1 < NH) {
      // ============================== tensor cores: a warp per half, so that the waits and the issue of one half pass while
      // the products of the other run.  The whole warp walks the loop (addresses and descriptors stay uniform), one lane issues.
      const int h = aux - 1;
      constexpr unsigned FMT = FP16 ? 0u : (1u << 7) | (1u << 10);
      constexpr unsigned ID_S = (1u << 4) | FMT | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      constexpr unsigned ID_O = (1u << 4) | FMT | (1u << 16) | (((unsigned)D >> 3) << 17) | ((128u >> 4) << 24);
      PaCursor<NH> cur;
      cur.set(p, s_place);
      // The ring is consumed in its order: K 0, then V n - 1 and K n in turn.
      int slot = 0, ph = 0, pp = 0, qp = 0, tile = 0, left = 0;   // (bit i of pp, qp: the parity of p[i], qfull[i])
      int till = PaWait::counted(p, PaWait::PRODUCTS);
      bool was_first = false, was_last = false, was_mine = false, mine = false, ok = true, more = true;
      auto step = [&]() {
        if (++slot == NS) {
          slot = 0;
          ph ^= 1;
        }
      };
      const unsigned t_o = tm + Sh::TM_O + h * D;
      auto qk = [&](int qb, int sb, int kslot, bool q_done) {   // S sb = Q qb K^T (by one lane)
        const unsigned long long a = PA_DESC_K | ((sm_q + qb * q_buf) >> 4), b = PA_DESC_K | ((sm_kv + kslot * Sh::TILE) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const unsigned o = ((k >> 2) * 16384 + (k & 3) * 32) >> 4, oq = ((k >> 2) * q_cb + (k & 3) * 32) >> 4;
          if (NH == 2 && k == D / 16 - 2) pa_arrive(smem_u32(&b_turn[h ^ 1]));   // (its first product is issued by when these are done)
          pa_mma_ss(tm + sb * 128, a + oq, b + o, ID_S, k > 0);
        }
        pa_commit(smem_u32(&b_s[sb]));
        pa_commit(smem_u32(&b_kempty[kslot]));
        if (q_done) pa_commit(smem_u32(&b_qempty[qb]));
      };
      // O += P sb V over one part of each 64 keys (by one lane)
      auto pv = [&](int part, int sb, int vslot, bool acc) {
        const unsigned long long b = PA_DESC_V | ((sm_kv + vslot * Sh::TILE) >> 4);
        constexpr int KS = 4 / PARTS;   // steps of 16 keys of a part of 64
#pragma unroll
        for (int rest = 0; rest < (NH == 1 ? 2 : 1); ++rest)   // (with the remainders of P)
#pragma unroll
          for (int i = 0; i < 2 * KS; ++i) {
            const int k = i / KS * 4 + part * KS + i % KS;
            pa_mma_ts(t_o, tm + sb * 128 + rest * 64 + k * 8, b + k * 128, ID_O, acc || rest > 0 || i > 0);
          }
      };
#pragma unroll 1
      for (int n = 0; more; ++n) {
        const bool first = left == 0;
        if (first) {
          if (n > 0) cur.next_tile(p);
          left = cur.count();
          more = left > 0;      // one more round for the last P V
          mine = h == 0 || cur.second_half(p);
        }
        const bool last = left == 1;
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
      // ============================== queries
      if (lane == 0) {
        PaCursor<NH> cur;
        cur.set(p, s_place);
        PaFill fill[2];
        int tile = 0, blocks = 0, till = PaWait::counted(p, PaWait::QUERIES);   // (blocks: of the tiles before)
        bool ok = true;
#pragma unroll 1
        for (; ok && cur.count() > 0; cur.next_tile(p)) {
          const int halves = cur.second_half(p) ? 2 : 1;
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {
            const int qb = NH == 2 ? h : tile & 1;
            ok = wait.count(till, smem_u32(&b_qempty[qb]), fill[qb].empty(), blocks);
            if (!ok) break;
            const unsigned full = smem_u32(&b_qfull[qb]);
            mbar_expect_tx(full, p.T * p.G * 128 * Sh::CB);
            for (int cb = 0; cb < Sh::CB; ++cb)
              pa_tma3(sm_q + qb * q_buf + cb * q_cb, &mq, cb * 64, cur.h * p.G, cur.q.s.q0 + (cur.j * NH + h) * p.T, full);
            ++fill[qb].sent;
          }
          ++tile;
          blocks += cur.count();
        }
        for (int qb = 0; qb < 2; ++qb)
          if (fill[qb].sent > 0) wait.drain(smem_u32(&b_qfull[qb]), fill[qb].landed());
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
      PaCursor<NH> cur;
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
      for (int cnt; (cnt = cur.count()) > 0; cur.next_tile(p)) {
        if (NH == 2 && half == 1 && !cur.second_half(p)) {
          n += cnt;
          continue;
        }
        const int t = (cur.j * NH + half) * p.T + rt;
        const bool live = rt < p.T && t < cur.q.s.m;
        const bool any_live = __any_sync(~0u, live);
        const int len = cur.q.s.len - cur.b * PA_BN;      // keys from the first block on
        // and visible ones, from this thread's half on (a lane without a row computes whatever it finds, and nobody reads it)
        const int vis = !live ? 1 << 30 : (p.causal ? cur.q.s.len - cur.q.s.m + t + 1 : cur.q.s.len) - cur.b * PA_BN - ch * 64;
        const int all_vis = __reduce_min_sync(~0u, vis);
        float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int k = 0; k < cnt; ++k, ++n) {
          const int sb = NH == 2 ? half : n & 1;
          wait(smem_u32(&b_s[sb]), sp >> sb & 1, NH == 2 ? n : 0);   // (half 1 may have sat out tiles before)
          sp ^= 1 << sb;
          __syncwarp();
          pa_fence_after();
          const unsigned t_s = tm + sb * 128 + lane_off;
          if (__builtin_expect((k + 1) * PA_BN > len && ch == 0, 0)) {
            // the values behind the sequence's end may be anything: zeros, so that 0 x NaN does not reach the sum
            const int place = 2 * n + 1, slot = place % NS;
            wait(smem_u32(&b_kfull[slot]), (place / NS) & 1);
            if (k * PA_BN + r >= len) {
              const unsigned row = sm_kv + slot * Sh::TILE + r * 128;
#pragma unroll 1
              for (int cb = 0; cb < Sh::CB; ++cb)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + cb * 16384 + e * 16), "r"(0) : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          if (any_live) {
            unsigned s[64];
            pa_ld32(t_s + ch * 64, s);
            pa_ld32(t_s + ch * 64 + 32, s + 32);
            pa_wait_ld<64>(s);
            if (__builtin_expect(k * PA_BN + 64 > all_vis, 0)) {
              const int left = vis - k * PA_BN;           // visible keys of these
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c >= left) s[c] = 0xFF800000u;        // -inf, whatever lies there
            }
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4]));
#pragma unroll
            for (int c = 8; c < 64; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[c + e])), __uint_as_float(s[c + 4 + e]));
            float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (__builtin_expect(k == 0 || pa_pair_or(pair, live && (m - ref) * p.scale2 > PA_LAZY), 0)) {
              m = together(fmaxf(m, ref), [](float a, float b) { return fmaxf(a, b); });
              const float f = m == -INFINITY ? 1.f : ex2((ref - m) * p.scale2);
              ref = m;
              if (k > 0) {
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
                if (NH == 1) {
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
        if (NH == 2) wait(smem_u32(&b_o[half]), tiles & 1);
        else wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);
        ++tiles;
        __syncwarp();
        pa_fence_after();
        if (any_live) {
          sum = together(sum, [](float a, float b) { return a + b; });
          const bool whole = cnt == cur.nb;
          const int tok = cur.q.s.q0 + t;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int head = cur.h * p.G + rg;
          const long long part = ((long long)blockIdx.x * 2 + (cur.b == 0 ? 1 : 0)) * NH + half;
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
              if (live)
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
  __syncthreads();
  if (aux == 3) {
    pa_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

// Joins the parts of the tiles that were cut: block (x, y) takes one of them, and of it half y / (D / CH) and CH channels.  A thread
// per row; where there are fewer rows than threads, several threads share a row's parts.  A call of few tiles, which are then cut
// into many parts, has blocks of 512 threads for each of its tiles, of as few channels as let all run at once (180 rows over 30K tokens,
// two tiles of 64 channels: 74 -> 21 us with the attention itself; with 8 channels always 23.5); one of many tiles 128 threads for each
// piece, most of which leave at once: looking for the tiles first costs 1.5 us more.
template <int D, int NH, bool FP16, int NT, int CH>
__global__ void __launch_bounds__(NT) pages_join_kernel(const __grid_constant__ PaParams p) {
  __shared__ float s_m[NT], s_sum[NT], s_o[CH][NT];
  __shared__ uint2 s_piece[NT == 128 ? 1 : PA_MAX_CTAS / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.y / (D / CH), ch = blockIdx.y % (D / CH) * CH;
  // the tile's pieces but its first: [c, end)
  int c = blockIdx.x, end, rows;
  PaRec r;
  if constexpr (NT == 128) {   // piece x, if it is the first that starts inside of its tile
    if (c == 0) return;
    r = p.rec[c];
    const long long last = p.rec[c - 1].begin, next = c + 1 < p.ctas ? p.rec[c + 1].begin : -1;   // (all loads at once)
    const int last_b = p.rec[c - 1].b;
    if (r.begin < 0 || r.b == 0 || (last == r.begin && last_b > 0)) return;
    rows = (min(r.ntok, (h + 1) * p.T) - h * p.T) * p.G;
    if (rows <= 0) return;
    end = c + 1;
    for (int in = NT; in == NT && next == r.begin && end < r.pieces; end += in) {
      const int q = end + threadIdx.x;
      in = __syncthreads_count(q < r.pieces && p.rec[q].begin == r.begin);
    }
  } else {   // the x-th of the tiles that are cut
    const int words = (p.ctas + 31) >> 5;
    for (int i = threadIdx.x; i < words * 32; i += NT) {
      bool first = false, more = false;   // piece i is the first that starts inside of its tile, or another one
      if (i > 0 && i < p.ctas) {
        const long long at = p.rec[i].begin, last = p.rec[i - 1].begin;
        const int b = p.rec[i].b, last_b = p.rec[i - 1].b;
        more = (at >= 0) & (b > 0) & (last == at) & (last_b > 0);
        first = (at >= 0) & (b > 0) & !more;
      }
      const unsigned f = __ballot_sync(~0u, first), m = __ballot_sync(~0u, more);
      if ((threadIdx.x & 31) == 0) s_piece[i >> 5] = make_uint2(f, m);
    }
    __syncthreads();
    int w = 0;
    while (w < words && __popc(s_piece[w].x) <= c) c -= __popc(s_piece[w++].x);
    if (w == words) return;
    unsigned x = s_piece[w].x;
    for (; c > 0; --c) x &= x - 1;
    c = w * 32 + __ffs(x) - 1;
    r = p.rec[c];
    end = c + 1;
    w = end >> 5;
    x = w < words ? ~s_piece[w].y & ~0u << (end & 31) : 0;
    while (x == 0 && ++w < words) x = ~s_piece[w].y;
    end = w < words ? w * 32 + __ffs(x) - 1 : p.ctas;
    rows = (min(r.ntok, (h + 1) * p.T) - h * p.T) * p.G;
    if (rows <= 0) return;
  }
  int lg = 0;
  while ((1 << lg) < rows) ++lg;
  const int row = threadIdx.x & ((1 << lg) - 1), grp = threadIdx.x >> lg;
  // groups of threads that share a row's parts, so that a group has AT parts (whose loads are all under way before the first is used)
  constexpr int AT = NT == 512 ? 4 : 2;
  const int grps = min(NT >> lg, (end - c + AT) / AT);
  float m = -INFINITY, sum = 0.f, o[CH] = {};
  if (grp < grps)
#pragma unroll 1
    for (int q0 = c - 1 + grp; q0 < end; q0 += AT * grps) {
      float2 ml[AT];
      float4 x[AT][CH / 4];
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        const int q = q0 + a * grps;
        ml[a] = make_float2(-INFINITY, 0.f);
        if (q < end) {
          const long long part = ((long long)q * 2 + (q < c ? 1 : 0)) * NH + h;
          ml[a] = p.part_ml[part * 128 + row];
          const float4* po = reinterpret_cast<const float4*>(p.part_o + (part * (D / 4) + ch / 4) * 512) + row;
#pragma unroll
          for (int e = 0; e < CH / 4; ++e) x[a][e] = po[e * 128];
        }
      }
      float top = m;
#pragma unroll
      for (int a = 0; a < AT; ++a) top = fmaxf(top, ml[a].x);
      const float base = top == -INFINITY ? 0.f : top, f0 = ex2(m - base);
      m = top;
      sum *= f0;
#pragma unroll
      for (int e = 0; e < CH; ++e) o[e] *= f0;
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        const float f = ex2(ml[a].x - base);
        sum += ml[a].y * f;
        if (f != 0.f)   // (a part without keys may hold anything)
#pragma unroll
          for (int e = 0; e < CH / 4; ++e) {
            o[4 * e] += x[a][e].x * f;
            o[4 * e + 1] += x[a][e].y * f;
            o[4 * e + 2] += x[a][e].z * f;
            o[4 * e + 3] += x[a][e].w * f;
          }
      }
    }
  if (grps > 1) {
    s_m[threadIdx.x] = m;
    __syncthreads();
    for (int g = 0; g < grps; ++g) m = fmaxf(m, s_m[(g << lg) + row]);
    const float mine = s_m[threadIdx.x], f = mine == -INFINITY ? 0.f : ex2(mine - m);
    s_sum[threadIdx.x] = sum * f;
#pragma unroll
    for (int e = 0; e < CH; ++e) s_o[e][threadIdx.x] = o[e] * f;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < CH; ++e) o[e] = 0.f;
    if (grp == 0)
      for (int g = 0; g < grps; ++g) {
        sum += s_sum[(g << lg) + row];
#pragma unroll
        for (int e = 0; e < CH; ++e) o[e] += s_o[e][(g << lg) + row];
      }
  }
  if (grp != 0 || row >= rows) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int t = row / p.G, head = r.kvh * p.G + (row - t * p.G);
  const long long tok = r.tok + h * p.T + t;
  unsigned x[CH / 2];
#pragma unroll
  for (int e = 0; e < CH / 2; ++e) x[e] = pa_pack<FP16>(o[2 * e] * inv, o[2 * e + 1] * inv);
  uint16_t* dst = p.out + tok * p.ots + head * p.ohs + ch;
  if constexpr (CH == 16) pa_store32(dst, x);
  else if constexpr (CH == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(x[0], x[1]);
  if (p.lse && ch == 0) p.lse[tok * p.Hq + head] = sum == 0.f ? -INFINITY : (m + PA_UP<FP16> + log2f(sum * PA_DOWN<FP16>)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------------------- launch

bool pages_attend_cuts(const PagesView& pg, const TableView& t) { return ((long long)t.cols << pg.lgS) > PA_WHOLE * PA_BN; }

// parts of NH halves of 128 rows, two per CTA; records
size_t pages_attend_bytes(int n_sm, int D) {
  return (size_t)n_sm * (sizeof(PaRec) + 2 * 2 * 128 * (sizeof(float2) + sizeof(float) * D)) + 64;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(p);
  fn.store(f);
  return f;
}

template <int D, int NH, bool FP16>
static cudaError_t launch_t(const PaParams& p, const CUtensorMap* maps, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};   // devices whose copy of the kernel has its attribute
  if (device >= 64 || !(ready.load() >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(pages_attend_kernel<D, NH, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, PaShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (device < 64) ready.fetch_or(1ull << device);
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(PA_THREADS<NH>);
  cfg.dynamicSmemBytes = PaShape<D>::SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, pages_attend_kernel<D, NH, FP16>, p, maps[0], maps[1], maps[2]);
  return e != cudaSuccess || !p.rec ? e : launch_pages_join(p, NH, FP16, st);   // (no rec: no tile is cut)
}

template <int D, int NH, bool FP16>
static cudaError_t join_t(const PaParams& p, cudaStream_t st) {
  // at most so many tiles; few: the blocks for them all run at once, two to an SM
  const long long tt = (long long)NH * p.T, tiles = (p.c.n + (p.c.total > p.c.n ? (p.c.total - p.c.n) / tt : 0)) * p.pg.H;
  auto few = [&](int ch) { return tiles * NH * (D / ch) <= 2 * p.ctas; };
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  auto launch = [&](auto kernel, long long x, int ch, int threads) {
    cfg.gridDim = dim3((unsigned)x, NH * (D / ch));
    cfg.blockDim = dim3(threads);
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  if (few(4)) return launch(pages_join_kernel<D, NH, FP16, 512, 4>, tiles, 4, 512);
  if (few(8)) return launch(pages_join_kernel<D, NH, FP16, 512, 8>, tiles, 8, 512);
  return launch(pages_join_kernel<D, NH, FP16, 128, 16>, p.ctas, 16, 128);
}
cudaError_t launch_pages_join(const PaParams& p, int nh, int fp16, cudaStream_t st) {
  if (p.pg.D == 128) {
    if (nh == 1) return fp16 ? join_t<128, 1, true>(p, st) : join_t<128, 1, false>(p, st);
    return fp16 ? join_t<128, 2, true>(p, st) : join_t<128, 2, false>(p, st);
  }
  if (nh == 1) return fp16 ? join_t<64, 1, true>(p, st) : join_t<64, 1, false>(p, st);
  return fp16 ? join_t<64, 2, true>(p, st) : join_t<64, 2, false>(p, st);
}

cudaError_t launch_pages_attend(const PagesAttendParams& a, int fp16, int device, int n_sm, void* ws, cudaStream_t st) {
  const EncodeFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const PagesView& g = a.pg;
  PaParams p{};
  p.pg = g;
  p.t = a.t;
  p.c = a.c;
  p.out = a.out;
  p.lse = a.lse;
  p.ots = a.ots;
  p.ohs = a.ohs;
  p.Hq = a.Hq;
  p.G = a.Hq / g.H;
  p.causal = a.causal;
  p.ctas = n_sm < PA_MAX_CTAS ? n_sm : PA_MAX_CTAS;
  p.scale = a.scale;
  p.expire = a.expire;
  p.scale2 = a.scale * 1.44269504088896341f;
  // One half where the longest chunk's rows fit it (bound by reading the cache), else two.  The tile takes no more
  // tokens than the longest chunk, so that its query copy does not read the next sequences' rows.
  const int fit = 128 / p.G;
  const bool one = a.max_q_len > 0 && a.max_q_len <= fit;
  p.T = one ? a.max_q_len : fit;
  p.q_rows = one && p.T * p.G <= 64 ? 64 : 128;
  const int nh = one ? 1 : 2;
  if (pages_attend_cuts(g, a.t)) {
    char* at = static_cast<char*>(ws);
    p.part_o = reinterpret_cast<float*>(at);
    at += (size_t)n_sm * 2 * nh * 128 * g.D * sizeof(float);
    p.part_ml = reinterpret_cast<float2*>(at);
    at += (size_t)n_sm * 2 * nh * 128 * sizeof(float2);
    p.rec = reinterpret_cast<PaRec*>(at);
  }

  CUtensorMap maps[3];
  const CUtensorMapDataType ty = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  // (a driver call: a thread that has made none of the runtime's has no context yet, which cudaSetDevice gives it)
  auto encode = [&](CUtensorMap* map, int rank, uint16_t* base, const cuuint64_t* dim, const cuuint64_t* str, const cuuint32_t* box) {
    auto call = [&] {
      return enc(map, ty, rank, base, dim, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if ((r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) && cudaSetDevice(device) == cudaSuccess) r = call();
    return r == CUDA_SUCCESS;
  };
  auto bytes = [&](long long stride) { return (cuuint64_t)(stride > 0 ? stride * 2 : g.D * 2); };   // (an axis of one entry: any)
  {
    const cuuint64_t dim[3] = {(cuuint64_t)g.D, (cuuint64_t)a.Hq, (cuuint64_t)a.c.total};
    const cuuint64_t str[2] = {bytes(a.Hq > 1 ? a.qhs : 0), bytes(a.c.total > 1 ? a.qts : 0)};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.T};
    if (!encode(&maps[0], 3, const_cast<uint16_t*>(a.q), dim, str, box)) return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dim[4] = {(cuuint64_t)g.D, (cuuint64_t)g.S, (cuuint64_t)g.H, (cuuint64_t)g.P};
    const cuuint64_t str[3] = {bytes(g.ts), bytes(g.hs), bytes(g.ps)};
    const cuuint32_t box[4] = {64, (cuuint32_t)(g.S < 128 ? g.S : 128), 1, 1};
    if (!encode(&maps[1 + i], 4, (i ? g.v : g.k) + a.layer * g.ls, dim, str, box)) return cudaErrorInvalidValue;
  }
  if (one && p.T * p.G <= PAGES_FEW_ROWS) return launch_pages_few(p, maps, fp16, device, st);
  if (g.D == 128) {
    if (one) return fp16 ? launch_t<128, 1, true>(p, maps, device, st) : launch_t<128, 1, false>(p, maps, device, st);
    return fp16 ? launch_t<128, 2, true>(p, maps, device, st) : launch_t<128, 2, false>(p, maps, device, st);
  }
  if (one) return fp16 ? launch_t<64, 1, true>(p, maps, device, st) : launch_t<64, 1, false>(p, maps, device, st);
  return fp16 ? launch_t<64, 2, true>(p, maps, device, st) : launch_t<64, 2, false>(p, maps, device, st);
}

}  // namespace qe
