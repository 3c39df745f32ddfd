// qe_pages_attn.cu -- attention of a chunk of new tokens over the cached pages.
//
// For query row (token t of a chunk of m, head h) with V visible keys (causal: kv_len - m + j + 1):
//   out = sum_i exp(s_i - M) v_i / sum_i exp(s_i - M),  s_i = scale q . k_i,  M = max s_i,
// in one pass over the keys with a running maximum, sum and accumulator in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qe_common.cuh"
#include "qe_pages.cuh"

namespace qe {

template <bool FP16>
__device__ __forceinline__ float pages_to_f(uint16_t x) {
  if constexpr (FP16) return __half2float(__ushort_as_half(x));
  return __uint_as_float((unsigned)x << 16);
}
template <bool FP16>
__device__ __forceinline__ uint16_t pages_from_f(float x) {
  if constexpr (FP16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One warp per (packed token, query head); lane l holds channels l, l + 32, ...
template <int D, bool FP16>
__global__ void __launch_bounds__(256) pages_attend_kernel(const PagesAttendParams p) {
  constexpr int E = D / 32;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int tok = (int)(w / p.Hq), h = (int)(w - (long long)tok * p.Hq);
  if (blockIdx.x == 0) check_starts(p.pg, p.c);
  if (tok >= p.c.total) return;
  int lo = 0, hi = p.c.n;   // the sequence whose packed tokens hold tok
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.c.q_start[mid + 1] <= tok) lo = mid + 1; else hi = mid;
  }
  if (lo >= p.c.n) return;
  const SeqInfo s = seq_info(p.pg, p.t, p.c, lo, lane == 0);
  if (tok < s.q0 || tok >= s.q0 + s.m) return;
  const int vis = p.causal ? max(0, s.len - s.m + (tok - s.q0) + 1) : s.len;
  const int kvh = h / (p.Hq / p.pg.H);
  float q[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = pages_to_f<FP16>(p.q[tok * p.qts + h * p.qhs + e * 32 + lane]) * p.scale;
  float m = -INFINITY, l = 0.f;
  int page = -1;
  for (int i = 0; i < vis; ++i) {
    if ((i & (p.pg.S - 1)) == 0) page = page_at(p.pg, p.t, s.row, i);
    const long long at = p.layer * p.pg.ls + max(page, 0) * p.pg.ps + kvh * p.pg.hs + (i & (p.pg.S - 1)) * p.pg.ts;
    float dot = 0.f;
    if (page >= 0)
#pragma unroll
      for (int e = 0; e < E; ++e) dot += q[e] * pages_to_f<FP16>(p.pg.k[at + e * 32 + lane]);
#pragma unroll
    for (int k = 16; k; k >>= 1) dot += __shfl_xor_sync(~0u, dot, k);
    const float mn = fmaxf(m, dot), f = __expf(m - mn), pr = __expf(dot - mn);
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + (page >= 0 ? pr * pages_to_f<FP16>(p.pg.v[at + e * 32 + lane]) : 0.f);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[tok * p.ots + h * p.ohs + e * 32 + lane] = pages_from_f<FP16>(o[e] * inv);
  if (p.lse && lane == 0) p.lse[(long long)tok * p.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

cudaError_t launch_pages_attend(const PagesAttendParams& p, int fp16, cudaStream_t st) {
  const long long blocks = ((long long)p.c.total * p.Hq + 7) / 8;
  if (p.pg.D == 128) {
    if (fp16) pages_attend_kernel<128, true><<<(unsigned)blocks, 256, 0, st>>>(p);
    else pages_attend_kernel<128, false><<<(unsigned)blocks, 256, 0, st>>>(p);
  } else {
    if (fp16) pages_attend_kernel<64, true><<<(unsigned)blocks, 256, 0, st>>>(p);
    else pages_attend_kernel<64, false><<<(unsigned)blocks, 256, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace qe
