// qe_pages_few.cu -- attention over the cached pages for tiles of at most 16 query rows (decode steps, a few drafts).
//
// Bound by reading the cache, so everything else has to fit under it: the products are taken the other way round, keys (then
// channels) as the 128 rows of the tensor cores and the few query rows as N = 16 columns:
//   S^T = K Q^T (128 keys x N),   O^T += V^T P^T (head_dim channels x 2 N, keys inner),
// with the formulas and the split of the line of qe_pages_attn.cu.  A block costs the tensor cores about 600 cycles instead of 1536,
// and a thread 16 exponentials instead of 64 whatever the rows (decode step of 16 sequences of up to 32K tokens: 302 -> 287 us with
// 128 channels, 236 -> 171 us with 64).
//  * P^T is written to shared memory in two parts per probability, rounded and remainder, as 2 N columns (about 17 significant bits
//    for bf16); the output adds the two columns of a row.  A key's 2 N columns are 64 bytes; the P of odd blocks is the other half
//    of the same 128-byte rows.
//  * A softmax thread has one key and all rows: references and running sums are per column, in registers; a column's maximum
//    is taken across the 128 threads only for a tile's first block and when a logit passes its reference by 2^8 (a vote over the four
//    warps otherwise).
// CTA: warps 0-3 softmax, 4 TMA of keys and values, 5 tensor-core issue, 6 TMA of the queries, 7 tensor memory.
// mbarriers: kfull / kempty per slot, qfull / qempty per query buffer, s[i] (S i complete), p[i] (P i written; one arrival per
// softmax warp), o[i] (the P V of an even or odd block complete, as with NH = 1 there).  Waits are bounded as in qe_pages_attn.cu.
#include <atomic>

#include "qe_pages_attn.cuh"

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
  static constexpr int SLOTS = (ALL - 2 * Q_BUF - P_BUF) / TILE;
  static constexpr int SMEM = ALL + 1024;
  static constexpr int TM_O = 2 * N, TM_COLS = 4 * N;             // tensor memory: S 0, S 1 (N columns each), O (2 N)
};

// Reduces v[0 .. 16) over the warp's lanes; returns the column whose result v[0] then is (lanes 2 i and 2 i + 1 both have column i).
// Each step halves the columns a lane keeps: 16 exchanges instead of 80.
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

template <int D, bool FP16>
__global__ void __launch_bounds__(PF_THREADS, 1)
    pages_few_kernel(const __grid_constant__ PaParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv) {
  using Sh = PfShape<D>;
  constexpr int NS = Sh::SLOTS, N = Sh::N;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) unsigned long long b_kfull[NS], b_kempty[NS], b_qfull[2], b_qempty[2], b_s[2], b_p[2], b_o[2], b_end;
  __shared__ unsigned s_tmem;
  __shared__ int s_abort;
  __shared__ PaPlace s_place[2];
  __shared__ long long s_w[PF_THREADS / 32];
  __shared__ __align__(16) float s_red[N][4];      // a column's value of each softmax warp
  __shared__ float s_inv[N];

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
  pa_find<1, PF_THREADS>(p, s_place, s_w);   // ends with a barrier
  pa_fence_after();
  const unsigned tm = s_tmem;
  const bool work = s_place[0].i < p.c.n && (s_place[0].i != s_place[1].i || s_place[0].h != s_place[1].h || s_place[0].j != s_place[1].j ||
                                             s_place[0].b != s_place[1].b);

  if (work && aux == 0) {
    // ============================== keys and values
    PaCursor<1> cur;
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
  } else if (work && aux == 1) {
    // ============================== tensor cores (the whole warp walks the loop, one lane issues)
    constexpr unsigned FMT = FP16 ? 0u : (1u << 7) | (1u << 10);
    constexpr unsigned ID_S = (1u << 4) | FMT | (((unsigned)N >> 3) << 17) | ((128u >> 4) << 24);
    constexpr unsigned ID_O = (1u << 4) | FMT | (1u << 15) | (1u << 16) | ((2u * N >> 3) << 17) | (((unsigned)D >> 4) << 24);
    PaCursor<1> cur;
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
          const unsigned long long a = PA_DESC_K | ((sm_kv + kslot * Sh::TILE) >> 4), b = PA_DESC_K | ((sm_q + qb * Sh::Q_BUF) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            pa_mma_ss(tm + (n & 1) * N, a + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), b + (((k >> 2) * Sh::Q_CB + (k & 3) * 32) >> 4), ID_S,
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
          const unsigned long long a = PA_DESC_V | ((sm_kv + slot * Sh::TILE) >> 4), b = PA_DESC_V | ((sm_p + pb * 64) >> 4);
#pragma unroll
          for (int k = 0; k < PA_BN / 16; ++k) pa_mma_ss(tm + Sh::TM_O, a + k * 128, b + k * 128, ID_O, !was_first || k > 0);
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
    // ============================== queries
    if (lane == 0) {
      PaCursor<1> cur;
      cur.set(p, s_place);
      PaFill fill[2];
      int tile = 0, blocks = 0, till = PaWait::counted(p, PaWait::QUERIES);   // (blocks: of the tiles before)
#pragma unroll 1
      for (; cur.count() > 0; cur.next_tile(p)) {
        const int qb = tile & 1;
        if (!wait.count(till, smem_u32(&b_qempty[qb]), fill[qb].empty(), blocks)) break;
        const unsigned full = smem_u32(&b_qfull[qb]);
        mbar_expect_tx(full, p.T * p.G * 128 * Sh::CB);
        for (int cb = 0; cb < Sh::CB; ++cb)
          pa_tma3(sm_q + qb * Sh::Q_BUF + cb * Sh::Q_CB, &mq, cb * 64, cur.h * p.G, cur.q.s.q0 + cur.j * p.T, full);
        ++fill[qb].sent;
        ++tile;
        blocks += cur.count();
      }
      for (int qb = 0; qb < 2; ++qb)
        if (fill[qb].sent > 0) wait.drain(smem_u32(&b_qfull[qb]), fill[qb].landed());
    }
  } else if (work && aux < 0) {
    // ============================== softmax: a key of every block, all rows
    const int kl = tid;
    const unsigned lane_off = (unsigned)(warp * 32) << 16;
    const unsigned prow = sm_p + kl * 128, x7 = kl & 7;   // this key's probabilities, in chunks of 16 bytes swizzled by the key
    PaCursor<1> cur;
    cur.set(p, s_place);
    int sp = 0, n = 0;   // (bit i of sp: the parity of s[i])
    auto larger = [](float a, float b) { return fmaxf(a, b); };
    auto plus = [](float a, float b) { return a + b; };
    // A wait that fails (the CTA is leaving) lets the loops run out without waiting, so that the warps' barriers stay in step.
#pragma unroll 1
    for (int cnt; (cnt = cur.count()) > 0; cur.next_tile(p)) {
      const int off = cur.q.s.len - cur.q.s.m + cur.j * p.T;        // the tile's first token sees the keys [0, off]
      const int every = p.causal ? off + 1 : cur.q.s.len;           // keys that all rows see
      constexpr float UP = PA_UP<FP16>;
      float base[N], sum[N];                                        // UP - reference (log2 units), and this key's part of the sum
#pragma unroll
      for (int c = 0; c < N; ++c) sum[c] = 0.f;
#pragma unroll 1
      for (int k = 0; k < cnt; ++k, ++n) {
        const int key = (cur.b + k) * PA_BN + kl;
        wait(smem_u32(&b_s[n & 1]), sp >> (n & 1) & 1);
        sp ^= 1 << (n & 1);
        __syncwarp();
        pa_fence_after();
        unsigned s[N];
        pa_ld16(tm + (n & 1) * N + lane_off, s);
        pa_wait_ld<N>(s);
        if (__builtin_expect((cur.b + k + 1) * PA_BN > every, 0)) {
          // rows from `from` on see this key
          const int from = key >= cur.q.s.len ? N : (p.causal ? min(max(key - off, 0), N) * p.G : 0);
#pragma unroll
          for (int c = 0; c < N; ++c)
            if (c < from) s[c] = 0xFF800000u;   // -inf, whatever lies there
          if ((cur.b + k + 1) * PA_BN > cur.q.s.len) {
            // the values behind the sequence's end may be anything: zeros, so that 0 x NaN does not reach the sum
            const int place = 2 * n + 1, slot = place % NS;
            wait(smem_u32(&b_kfull[slot]), (place / NS) & 1);
            if (key >= cur.q.s.len) {
              const unsigned row = sm_kv + slot * Sh::TILE + kl * 128;
#pragma unroll 1
              for (int cb = 0; cb < Sh::CB; ++cb)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + cb * 16384 + e * 16), "r"(0) : "memory");
            }
            __syncwarp();
          }
        }
        bool over = false;
        if (k > 0) {
#pragma unroll
          for (int c = 0; c < N; ++c) over |= fmaf(__uint_as_float(s[c]), p.scale2, base[c]) > PA_LAZY + UP;
        }
        if (__builtin_expect(k == 0 || pf_or(over), 0)) {
          float m[N], f[N];
#pragma unroll
          for (int c = 0; c < N; ++c) m[c] = __uint_as_float(s[c]);
          const int col = pf_reduce<N>(m, larger);
          s_red[col][warp] = m[0];
          pf_sync();
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float4 w = *reinterpret_cast<const float4*>(s_red[c]);
            const float top = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) * p.scale2;
            // (a row that sees none of these keys keeps its reference; of a first block, any)
            const float nb = top == -INFINITY ? (k == 0 ? UP : base[c]) : UP - top;
            const float use = k == 0 ? nb : fminf(base[c], nb);
            f[c] = k == 0 ? 1.f : ex2(use - base[c]);
            base[c] = use;
            sum[c] *= f[c];
          }
          if (k > 0) {
            wait(smem_u32(&b_o[(n - 1) & 1]), (n - 1) >> 1 & 1);   // the P V before this block's
            __syncwarp();
            pa_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              unsigned o[N];
              const unsigned at = tm + Sh::TM_O + part * N + lane_off;
              pa_ld16(at, o);
              pa_wait_ld<N>(o);
#pragma unroll
              for (int c = 0; c < N; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              pa_st16(at, o);
            }
            pa_wait_st();
          }
          pf_sync();   // s_red may be written again
        }
        // (this S says that the P V two blocks ago is complete: its P may be overwritten)
        const int pb = n & 1;
        const unsigned long long sc2 = f2_pack(p.scale2, p.scale2);
#pragma unroll
        for (int c = 0; c < N; c += 8) {
          unsigned hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
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
      const int col = pf_reduce<N>(sum, plus);
      s_red[col][warp] = sum[0];
      pf_sync();
      const bool whole = cnt == cur.nb;
      const int ntok = min(p.T, cur.q.s.m - cur.j * p.T), rows = ntok * p.G;
      const long long part = (long long)blockIdx.x * 2 + (cur.b == 0 ? 1 : 0);
      if (kl < rows) {   // a thread per row
        const int row = kl;
        float ref = 0.f;   // (of the sums: UP below the reference)
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (c == kl) ref = -base[c];
        const float4 w = *reinterpret_cast<const float4*>(s_red[row]);
        const float all = w.x + w.y + w.z + w.w;
        s_inv[row] = all == 0.f ? 0.f : 1.f / all;
        if (!whole) {
          p.part_ml[part * 128 + row] = make_float2(all == 0.f ? -INFINITY : ref, all);
        } else if (p.lse) {
          const int t = row / p.G;
          p.lse[(long long)(cur.q.s.q0 + cur.j * p.T + t) * p.Hq + cur.h * p.G + (row - t * p.G)] =
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
      unsigned o[N], l[N];
      pa_ld16(tm + Sh::TM_O + lane_off, o);
      pa_ld16(tm + Sh::TM_O + N + lane_off, l);
      pa_wait_ld<N>(o);
      pa_wait_ld<N>(l);
      uint16_t* dst = p.out + (long long)(cur.q.s.q0 + cur.j * p.T) * p.ots + (long long)cur.h * p.G * p.ohs + chan;
      float* po = p.part_o + (part * (D / 4) + chan / 4) * 512 + chan % 4;
      int g = 0;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) {
          const float x = __uint_as_float(o[c]) + __uint_as_float(l[c]);
          if (have && whole) *dst = (uint16_t)pa_pack<FP16>(x * s_inv[c], 0.f);
          if (have && !whole) po[c * 4] = x;
          dst += p.ohs;
          if (++g == p.G) {
            g = 0;
            dst += p.ots - p.G * p.ohs;
          }
        }
      pa_fence_before();
      pf_sync();   // O and the sums are read whole before the next tile's
    }
  }
  __syncthreads();
  if (aux == 3) {
    pa_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(Sh::TM_COLS) : "memory");
  }
}

template <int D, bool FP16>
static cudaError_t few_t(const PaParams& p, const CUtensorMap* maps, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};   // devices whose copy of the kernel has its attribute
  if (device >= 64 || !(ready.load() >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(pages_few_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, PfShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (device < 64) ready.fetch_or(1ull << device);
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(PF_THREADS);
  cfg.dynamicSmemBytes = PfShape<D>::SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_few_kernel<D, FP16>, p, maps[0], maps[1], maps[2]);
  return e != cudaSuccess || !p.rec ? e : launch_pages_join(p, 1, FP16, st);   // (no rec: no tile is cut)
}

cudaError_t launch_pages_few(const PaParams& p, const CUtensorMap* maps, int fp16, int device, cudaStream_t st) {
  if (p.pg.D == 128) return fp16 ? few_t<128, true>(p, maps, device, st) : few_t<128, false>(p, maps, device, st);
  return fp16 ? few_t<64, true>(p, maps, device, st) : few_t<64, false>(p, maps, device, st);
}

}  // namespace qe
