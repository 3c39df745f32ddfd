// qe_pages_ranges.cu -- attention over two ranges of cached keys: a sliding window with the first tokens, or a prefix that
// other sequences share with the sequence's own tokens behind it.
//
// For the row of token t (of a chunk of m, at position p = kv_len - m + t) and query head h:
//   window:  keys [0, min(sinks, p - window + 1)) and [max(0, p - window + 1), p];
//   shared:  keys [0, prefix) of the group's first sequence and [prefix, p] of its own,
//   out = sum_i e^(x_i - M) v_i / sum_i e^(x_i - M),   x_i = scale q . k_i,
// in one pass with a running maximum M, sum and accumulator in float32.  A warp per row: right for every case, and bound by its
// own instructions (some 30 for a key).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qe_common.cuh"
#include "qe_pages.cuh"

namespace qe {

template <int D, bool FP16>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&x)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const unsigned u = *reinterpret_cast<const unsigned*>(p + i * 64 + lane * 2);
    if constexpr (FP16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = bf16lo_to_f32(u);
      x[2 * i + 1] = bf16hi_to_f32(u);
    }
  }
}

template <int D, bool FP16, bool SHARED>
__global__ void __launch_bounds__(128) pages_ranges_kernel(const PagesAttendParams p, const PagesWindow w, const PagesGroups gr) {
  griddep_wait();
  const int lane = threadIdx.x & 31, tok = blockIdx.x, h = blockIdx.y, G = p.Hq / p.pg.H;
  const int seq = pages_count_below(p.c.q_start + 1, p.c.n, tok);
  if (seq >= p.c.n) return;
  const bool report = lane == 0 && threadIdx.x == 0;
  const SeqInfo s = seq_info(p.pg, p.t, p.c, seq, report);
  if (tok < s.q0 || tok >= s.q0 + s.m) return;
  const int pos = s.len - s.m + (tok - s.q0);
  int row0 = s.row, end0, from1, end1 = p.causal ? pos + 1 : s.len;
  if (SHARED) {
    const int g = pages_count_below(gr.start + 1, gr.n, seq);
    if (g >= gr.n) {
      if (report) pages_report(p.pg, QE_PAGES_ERR_ROW);
      return;
    }
    const int first = gr.start[g], end = gr.start[g + 1];
    if (first < 0 || first > seq || end > p.c.n) {
      if (report) pages_report(p.pg, QE_PAGES_ERR_ROW);
      if (first < 0 || first > seq) return;
    }
    const SeqInfo f = seq_info(p.pg, p.t, p.c, first, false);
    const int want = gr.prefix[g];
    const int whole = max(want, 0) & ~(p.pg.S - 1);
    if ((want < 0 || want > f.len || (whole > 0 && whole > (p.causal ? s.len - s.m : s.len))) && report) pages_report(p.pg, QE_PAGES_ERR_ROW);
    end0 = from1 = min(max(want, 0), f.len) & ~(p.pg.S - 1);
    row0 = f.row;
  } else {
    from1 = max(0, pos - w.window + 1);
    end0 = min(w.sinks, from1);
  }
  for (int q = threadIdx.x >> 5; q < G; q += 4) {
    const int head = h * G + q;
    float x[D / 32], o[D / 32] = {}, m = -INFINITY, sum = 0.f;
    load_row<D, FP16>(p.q + tok * p.qts + head * p.qhs, x);
    auto walk = [&](int row, int a, int b) {
      for (int key = a; key < b; ++key) {
        const int page = p.t.table[(long long)row * p.t.stride + (key >> p.pg.lgS)];
        float k[D / 32] = {}, v[D / 32] = {};
        if (page >= 0 && page < p.pg.P) {
          const long long at = p.layer * p.pg.ls + page * p.pg.ps + h * p.pg.hs + (key & (p.pg.S - 1)) * p.pg.ts;
          load_row<D, FP16>(p.pg.k + at, k);
          load_row<D, FP16>(p.pg.v + at, v);
        } else if (lane == 0) {
          pages_report(p.pg, QE_PAGES_ERR_PAGE);
        }
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) d = fmaf(x[i], k[i], d);
#pragma unroll
        for (int i = 16; i; i >>= 1) d += __shfl_xor_sync(~0u, d, i);
        d *= p.scale;
        const float top = fmaxf(m, d), f = __expf(m - top), e = __expf(d - top);
        m = top;
        sum = sum * f + e;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = o[i] * f + e * v[i];
      }
    };
    walk(row0, 0, end0);
    walk(s.row, from1, end1);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint16_t* to = p.out + tok * p.ots + head * p.ohs + i * 64 + lane * 2;
      if constexpr (FP16) *reinterpret_cast<__half2*>(to) = __floats2half2_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
      else *reinterpret_cast<unsigned*>(to) = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    }
    if (p.lse && lane == 0) p.lse[(long long)tok * p.Hq + head] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
}

template <bool SHARED>
static cudaError_t launch_ranges(const PagesAttendParams& p, const PagesWindow& w, const PagesGroups& g, int fp16, cudaStream_t st) {
  const dim3 grid(p.c.total, p.pg.H);
  if (p.pg.D == 128) fp16 ? pages_ranges_kernel<128, true, SHARED><<<grid, 128, 0, st>>>(p, w, g) : pages_ranges_kernel<128, false, SHARED><<<grid, 128, 0, st>>>(p, w, g);
  else fp16 ? pages_ranges_kernel<64, true, SHARED><<<grid, 128, 0, st>>>(p, w, g) : pages_ranges_kernel<64, false, SHARED><<<grid, 128, 0, st>>>(p, w, g);
  return cudaGetLastError();
}

cudaError_t launch_pages_attend_window(const PagesAttendParams& p, const PagesWindow& w, int fp16, int, int, void*, cudaStream_t st) {
  return launch_ranges<false>(p, w, PagesGroups{}, fp16, st);
}
cudaError_t launch_pages_attend_shared(const PagesAttendParams& p, const PagesGroups& g, int fp16, int, int, void*, cudaStream_t st) {
  return launch_ranges<true>(p, PagesWindow{}, g, fp16, st);
}

}  // namespace qe
