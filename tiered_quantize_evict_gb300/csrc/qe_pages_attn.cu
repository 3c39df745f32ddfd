// qe_pages_attn.cu -- what the attentions over the cached pages share on the host, the join of cut tiles, and the attention over all keys
// (qe_pages_halves.cuh and qe_pages_few.cuh have the kernels, and the mathematics).
#include <atomic>

#include "qe_pages_launch.cuh"

namespace qe {

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
  if (p.gr.n > 0 && pa_strange<FP16, CH / 2>(x)) pages_report(p.pg, QE_PAGES_ERR_VALUE);
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

EncodeFn pages_encode_fn() {
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
static cudaError_t join_t(const PaParams& p, cudaStream_t st) {
  // at most so many tiles; few: the blocks for them all run at once, two to an SM
  const long long tt = (long long)NH * p.T, tiles = (p.items + (p.c.total > p.items ? (p.c.total - p.items) / tt : 0)) * p.pg.H;
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
  return launch_pages_mode<PA_PLAIN>(a, PagesWindow{}, PagesGroups{}, fp16, device, n_sm, ws, st);
}

}  // namespace qe
