// qe_pages_launch.cuh -- the launch of an attention over the cached pages, of one mode (PaMode).
#pragma once
#include <atomic>
#include <numeric>
#include <type_traits>

#include "qe_pages_few.cuh"
#include "qe_pages_halves.cuh"

namespace qe {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn pages_encode_fn();

template <int D, int NH, bool FP16, int MODE, bool REST = NH == 1>
static cudaError_t halves_t(const PaParams& p, const CUtensorMap* maps, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};   // devices whose copy of the kernel has its attribute
  if (device >= 64 || !(ready.load() >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(pages_attend_kernel<D, NH, FP16, MODE, REST>, cudaFuncAttributeMaxDynamicSharedMemorySize, PaShape<D>::SMEM);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, pages_attend_kernel<D, NH, FP16, MODE, REST>, p, maps[0], maps[1], maps[2]);
  return e != cudaSuccess || !p.rec ? e : launch_pages_join(p, NH, FP16, st);   // (no rec: no tile is cut)
}

template <int D, int R, bool FP16, int MODE>
static cudaError_t few_t(const PaParams& p, const CUtensorMap* maps, int device, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};   // devices whose copy of the kernel has its attribute
  if (device >= 64 || !(ready.load() >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(pages_few_kernel<D, R, FP16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, PfShape<D>::SMEM);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_few_kernel<D, R, FP16, MODE>, p, maps[0], maps[1], maps[2]);
  return e != cudaSuccess || !p.rec ? e : launch_pages_join(p, 1, FP16, st);   // (no rec: no tile is cut)
}

// w: of PA_WINDOW, gr: of PA_SHARED
template <int MODE>
static cudaError_t launch_pages_mode(const PagesAttendParams& a, const PagesWindow& w, const PagesGroups& gr, int fp16, int device, int n_sm,
                                     void* ws, cudaStream_t st) {
  const EncodeFn enc = pages_encode_fn();
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
  p.items = MODE == PA_SHARED ? gr.n : a.c.n;
  p.win = w;
  p.sa = MODE == PA_WINDOW ? (w.sinks + (g.S < PA_BN ? g.S : PA_BN) - 1) & -(g.S < PA_BN ? g.S : PA_BN) : 0;
  p.gr = gr;
  // One half where the rows of the longest chunk (the largest group) fit it (bound by reading the cache), else two.  The tile takes
  // no more tokens than that, so that its query copy does not read the next ones' rows.
  const int fit = 128 / p.G;
  int most = MODE == PA_SHARED ? gr.max_len : a.max_q_len;
  if (MODE == PA_SHARED && (most == 0 || most > a.c.total)) most = a.c.total;
  const bool one = most > 0 && most <= fit;
  p.T = one ? most : fit;
  p.q_rows = one && p.T * p.G <= 64 ? 64 : 128;
  const int nh = one ? 1 : 2;
  // whether any tile may be cut (a window's only has what it sees)
  const bool cuts = MODE == PA_SHARED || (pages_attend_cuts(g, a.t) &&
                                          (MODE != PA_WINDOW || (long long)w.window + p.sa + nh * p.T + 2 * PA_BN > PA_WHOLE * PA_BN));
  if (cuts) {
    char* at = static_cast<char*>(ws);
    p.part_o = reinterpret_cast<float*>(at);
    at += (size_t)n_sm * 2 * nh * 128 * g.D * sizeof(float);
    p.part_ml = reinterpret_cast<float2*>(at);
    at += (size_t)n_sm * 2 * nh * 128 * sizeof(float2);
    p.rec = reinterpret_cast<PaRec*>(at);
  }

  CUtensorMap maps[3];
  const CUtensorMapDataType ty = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
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
  // keys and values (PaParams); `unit`: the heads' places are so many elements apart
  const long long unit = g.hs && g.ps ? std::gcd(g.hs, g.ps) : (g.hs ? g.hs : (g.ps ? g.ps : g.D));
  const long long places = (g.P - 1) * (g.ps / unit) + (g.H - 1) * (g.hs / unit) + 1;
  p.wide = places <= INT_MAX;
  p.of_page = (int)(g.ps / unit);
  p.of_head = (int)(g.hs / unit);
  p.all = (int)places;
  for (int i = 0; i < 2; ++i) {
    uint16_t* base = (i ? g.v : g.k) + a.layer * g.ls;
    const cuuint32_t cb = (cuuint32_t)(g.D / 64), rows = (cuuint32_t)(g.S < PA_BN ? g.S : PA_BN);
    const cuuint64_t wide_dim[5] = {64, 8, cb, (cuuint64_t)(g.S / 8), (cuuint64_t)places}, wide_str[4] = {bytes(g.ts), 128, bytes(8 * g.ts), bytes(unit)};
    const cuuint32_t wide_box[5] = {64, 8, cb, rows / 8, 1};
    const cuuint64_t dim[5] = {64, cb, (cuuint64_t)g.S, (cuuint64_t)g.H, (cuuint64_t)g.P}, str[4] = {128, bytes(g.ts), bytes(g.hs), bytes(g.ps)};
    const cuuint32_t box[5] = {64, 1, 8, 1, 1};
    if (!(p.wide ? encode(&maps[1 + i], 5, base, wide_dim, wide_str, wide_box) : encode(&maps[1 + i], 5, base, dim, str, box))) return cudaErrorInvalidValue;
  }
  if (one && p.T * p.G <= PAGES_FEW_ROWS) {
    // (columns that the softmax takes: those of a decode step with 4 heads to a group need not pay for 16)
    auto few = [&](auto r) {
      constexpr int R = decltype(r)::value;
      if (g.D == 128) return fp16 ? few_t<128, R, true, MODE>(p, maps, device, st) : few_t<128, R, false, MODE>(p, maps, device, st);
      return fp16 ? few_t<64, R, true, MODE>(p, maps, device, st) : few_t<64, R, false, MODE>(p, maps, device, st);
    };
    const int rows = p.T * p.G;
    if (rows <= 4) return few(std::integral_constant<int, 4>{});
    return rows <= 8 ? few(std::integral_constant<int, 8>{}) : few(std::integral_constant<int, 16>{});
  }
  if constexpr (MODE == PA_SHARED)   // (chunks that an attention without groups takes with one half keep their bits in groups of any size)
    if (!one && a.max_q_len > 0 && a.max_q_len <= fit) {
      if (g.D == 128) return fp16 ? halves_t<128, 2, true, MODE, true>(p, maps, device, st) : halves_t<128, 2, false, MODE, true>(p, maps, device, st);
      return fp16 ? halves_t<64, 2, true, MODE, true>(p, maps, device, st) : halves_t<64, 2, false, MODE, true>(p, maps, device, st);
    }
  if (g.D == 128) {
    if (one) return fp16 ? halves_t<128, 1, true, MODE>(p, maps, device, st) : halves_t<128, 1, false, MODE>(p, maps, device, st);
    return fp16 ? halves_t<128, 2, true, MODE>(p, maps, device, st) : halves_t<128, 2, false, MODE>(p, maps, device, st);
  }
  if (one) return fp16 ? halves_t<64, 1, true, MODE>(p, maps, device, st) : halves_t<64, 1, false, MODE>(p, maps, device, st);
  return fp16 ? halves_t<64, 2, true, MODE>(p, maps, device, st) : halves_t<64, 2, false, MODE>(p, maps, device, st);
}

}  // namespace qe
