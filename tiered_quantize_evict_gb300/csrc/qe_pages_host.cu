// qe_pages_host.cu -- C ABI of the paged cache (include/qe.h): checks of the arguments, launches.
//
// No handle and no state: a call checks what the host can see, builds the kernels' parameters and
// launches on the caller's stream, with the buffers' device current for the duration of the call.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "qe.h"
#include "qe_handle.hpp"
#include "qe_pages.cuh"

namespace {

qe_status fail(qe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  qe::set_global_error(buf);
  return s;
}
qe_status cuda_fail(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  return fail(QE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool misaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// The buffers' device, current for one call.
struct DeviceGuard {
  int before = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceGuard(int dev) {
    err = cudaGetDevice(&before);
    if (err == cudaSuccess && before != dev) err = cudaSetDevice(dev);
    else if (err == cudaSuccess) before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
};

qe_status sm_count(int dev, int* n) {
  static std::atomic<int> known[64];   // a property of the device, read once
  if (dev < 64 && (*n = known[dev].load()) > 0) return QE_OK;
  const cudaError_t e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "no CUDA device");
  if (dev < 64) known[dev].store(*n);
  return QE_OK;
}

#define QE_TRY(call)                    \
  do {                                  \
    const qe_status s_ = (call);        \
    if (s_ != QE_OK) return s_;         \
  } while (0)

qe_status check_pages(const qe_pages* g, qe::PagesView* o) {
  if (!g) return fail(QE_ERR_INVALID_ARG, "pages is null");
  if (!g->k || !g->v) return fail(QE_ERR_INVALID_ARG, "pages: k or v is null");
  if (g->dtype != QE_DTYPE_BF16 && g->dtype != QE_DTYPE_FP16) return fail(QE_ERR_INVALID_ARG, "pages: dtype must be bf16 or fp16");
  if (g->device < 0) return fail(QE_ERR_INVALID_ARG, "pages: bad device");
  if (g->n_layers < 1 || g->n_pages < 1 || g->n_kv_heads < 1)
    return fail(QE_ERR_INVALID_ARG, "pages: n_layers, n_pages and n_kv_heads must be >= 1");
  if (g->head_dim != 64 && g->head_dim != 128) return fail(QE_ERR_INVALID_ARG, "pages: head_dim must be 64 or 128");
  int lg = 4;
  while (lg < 8 && (1 << lg) != g->page_size) ++lg;
  if ((1 << lg) != g->page_size) return fail(QE_ERR_INVALID_ARG, "pages: page_size must be 16, 32, 64, 128 or 256");
  if (misaligned(g->k, 16) || misaligned(g->v, 16)) return fail(QE_ERR_INVALID_ARG, "pages: k and v must be 16-byte aligned");
  const long long st[4] = {g->layer_stride, g->page_stride, g->head_stride, g->token_stride};
  const int n[4] = {g->n_layers, g->n_pages, g->n_kv_heads, g->page_size};
  for (int i = 0; i < 4; ++i)
    if (n[i] > 1 && (st[i] < g->head_dim || st[i] % 8 || st[i] >= (1ll << 39)))
      return fail(QE_ERR_INVALID_ARG, "pages: strides must be positive multiples of 8 elements, at least head_dim");
  if (misaligned(g->err, 4)) return fail(QE_ERR_INVALID_ARG, "pages: err must be 4-byte aligned");
  o->k = static_cast<uint16_t*>(g->k);
  o->v = static_cast<uint16_t*>(g->v);
  o->ls = n[0] > 1 ? st[0] : 0;
  o->ps = n[1] > 1 ? st[1] : 0;
  o->hs = n[2] > 1 ? st[2] : 0;
  o->ts = st[3];
  o->L = n[0];
  o->P = n[1];
  o->H = n[2];
  o->S = n[3];
  o->lgS = lg;
  o->D = g->head_dim;
  o->err = g->err;
  return QE_OK;
}

qe_status check_table(const qe_page_table* t, bool refs, qe::TableView* o) {
  if (!t || !t->table || !t->kv_len) return fail(QE_ERR_INVALID_ARG, "page table: null pointer");
  if (refs && !t->refs) return fail(QE_ERR_INVALID_ARG, "page table: refs is null");
  if (t->n_rows < 1 || t->max_pages < 1) return fail(QE_ERR_INVALID_ARG, "page table: n_rows and max_pages must be >= 1");
  if (refs && ((long long)t->max_pages + 1) * t->n_rows > 0x7FFFFFFF)   // (pages are counted in 32 bits)
    return fail(QE_ERR_INVALID_ARG, "page table: too large to be managed: n_rows * (max_pages + 1) must be below 2^31");
  if (t->n_rows > 1 && t->row_stride < t->max_pages) return fail(QE_ERR_INVALID_ARG, "page table: row_stride is below max_pages");
  if (misaligned(t->table, 4) || misaligned(t->kv_len, 4) || misaligned(t->refs, 4))
    return fail(QE_ERR_INVALID_ARG, "page table: pointers must be 4-byte aligned");
  *o = qe::TableView{t->table, t->kv_len, t->refs, t->n_rows > 1 ? t->row_stride : 0, t->n_rows, t->max_pages};
  return QE_OK;
}

qe_status check_chunks(const qe_chunks* c, qe::ChunksView* o) {
  if (!c) return fail(QE_ERR_INVALID_ARG, "chunks is null");
  if (c->n_seqs < 0 || c->n_seqs > 65536 || c->total_q < 0 || c->total_q > (1 << 30))
    return fail(QE_ERR_INVALID_ARG, "chunks: n_seqs must be 0 .. 65536 and total_q 0 .. 2^30");
  if (c->n_seqs > 0 && c->total_q > 0 && !c->q_start) return fail(QE_ERR_INVALID_ARG, "chunks: q_start is null");
  if (misaligned(c->q_start, 4) || misaligned(c->rows, 4)) return fail(QE_ERR_INVALID_ARG, "chunks: pointers must be 4-byte aligned");
  *o = qe::ChunksView{c->q_start, c->rows, c->n_seqs, c->total_q};
  return QE_OK;
}

qe_status check_layer(const qe_pages* g, int layer) {
  if (layer < 0 || layer >= g->n_layers) return fail(QE_ERR_INVALID_ARG, "layer %d out of range", layer);
  return QE_OK;
}

// a [tokens][heads][head_dim] operand
qe_status check_rows(const char* what, const void* p, long long ts, long long hs, int tokens, int heads, int d) {
  if (!p) return fail(QE_ERR_INVALID_ARG, "%s is null", what);
  if (misaligned(p, 16)) return fail(QE_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
  if ((tokens > 1 && (ts < d || ts % 8 || ts >= (1ll << 39))) || (heads > 1 && (hs < d || hs % 8 || hs >= (1ll << 39))))
    return fail(QE_ERR_INVALID_ARG, "%s: strides must be positive multiples of 8 elements, at least head_dim", what);
  return QE_OK;
}

qe_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) return fail(QE_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
  if (misaligned(ws, 16)) return fail(QE_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return QE_OK;
}

qe_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? QE_OK : cuda_fail(e, what); }

// the arguments that every attention has; *some is false where there is nothing to do
qe_status attend_params(const qe_pages* pages, int layer, const qe_page_table* seqs, const qe_chunks* chunks, const qe_pages_attend_args* a,
                        qe::PagesAttendParams* o, bool* some) {
  qe::PagesAttendParams& p = *o;
  *some = false;
  QE_TRY(check_pages(pages, &p.pg));
  QE_TRY(check_layer(pages, layer));
  QE_TRY(check_table(seqs, false, &p.t));
  QE_TRY(check_chunks(chunks, &p.c));
  if (!a) return fail(QE_ERR_INVALID_ARG, "args is null");
  if (a->n_q_heads < 1 || a->n_q_heads % p.pg.H || a->n_q_heads / p.pg.H > 128)
    return fail(QE_ERR_INVALID_ARG, "n_q_heads must be a multiple of n_kv_heads, at most 128 per KV head");
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return fail(QE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (a->max_q_len < 0) return fail(QE_ERR_INVALID_ARG, "max_q_len must be >= 0");
  if (p.c.n == 0 || p.c.total == 0) return QE_OK;
  QE_TRY(check_rows("q", a->q, a->q_token_stride, a->q_head_stride, p.c.total, a->n_q_heads, p.pg.D));
  QE_TRY(check_rows("out", a->out, a->out_token_stride, a->out_head_stride, p.c.total, a->n_q_heads, p.pg.D));
  if (misaligned(a->lse, 4)) return fail(QE_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  p.q = static_cast<const uint16_t*>(a->q);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.qts = a->q_token_stride;
  p.qhs = a->q_head_stride;
  p.ots = a->out_token_stride;
  p.ohs = a->out_head_stride;
  p.layer = layer;
  p.Hq = a->n_q_heads;
  p.causal = a->causal != 0;
  p.max_q_len = a->max_q_len;
  p.scale = a->scale;
  *some = true;
  return QE_OK;
}

// need: bytes of workspace for so many SMs; launch: with their number
template <class Need, class Launch>
qe_status attend_launch(const char* name, const qe_pages* pages, qe::PagesAttendParams& p, void* workspace, size_t bytes, Need need, Launch launch) {
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  if (const size_t n = need(n_sm)) QE_TRY(check_workspace(workspace, bytes, n));
  p.expire = qe::take_pages_expire();
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  return launched(launch(n_sm), name);
}

size_t attend_need(const qe::PagesAttendParams& p, int n_sm) { return qe::pages_attend_cuts(p.pg, p.t) ? qe::pages_attend_bytes(n_sm, p.pg.D) : 0; }

qe_status check_window(int window, int sinks, qe::PagesWindow* o) {
  if (window < 1 || sinks < 0) return fail(QE_ERR_INVALID_ARG, "window must be >= 1 and sinks >= 0");
  constexpr int MOST = 1 << 30;   // (a row holds no more tokens)
  *o = qe::PagesWindow{window < MOST ? window : MOST, sinks < MOST ? sinks : MOST};
  return QE_OK;
}

}  // namespace

extern "C" {

qe_status qe_pages_append(const qe_pages* pages, int layer, const qe_page_table* seqs, const qe_chunks* chunks,
                          const qe_pages_append_args* a, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_append");
  qe::PagesAppendParams p{};
  QE_TRY(check_pages(pages, &p.pg));
  QE_TRY(check_layer(pages, layer));
  QE_TRY(check_table(seqs, false, &p.t));
  QE_TRY(check_chunks(chunks, &p.c));
  if (!a) return fail(QE_ERR_INVALID_ARG, "args is null");
  if (p.c.n == 0 || p.c.total == 0) return QE_OK;
  const int D = p.pg.D, total = p.c.total;
  QE_TRY(check_rows("k", a->k, a->k_token_stride, a->k_head_stride, total, p.pg.H, D));
  QE_TRY(check_rows("v", a->v, a->v_token_stride, a->v_head_stride, total, p.pg.H, D));
  if (a->q) {
    if (a->n_q_heads < 1 || a->n_q_heads > 65536) return fail(QE_ERR_INVALID_ARG, "n_q_heads must be 1 .. 65536");
    QE_TRY(check_rows("q", a->q, a->q_token_stride, a->q_head_stride, total, a->n_q_heads, D));
    QE_TRY(check_rows("q_out", a->q_out, a->q_out_token_stride, a->q_out_head_stride, total, a->n_q_heads, D));
  } else if (a->q_out) {
    return fail(QE_ERR_INVALID_ARG, "q_out without q");
  }
  if (const qe_rope* r = a->rope) {
    if (r->rot_dim < 0 || r->rot_dim > D || r->rot_dim % 2) return fail(QE_ERR_INVALID_ARG, "rope: rot_dim must be even, 0 .. head_dim");
    if (r->halves && r->rot_dim % 16) return fail(QE_ERR_INVALID_ARG, "rope: rot_dim must be a multiple of 16 with halves");
    if (r->n_axes < 1 || r->n_axes > 8) return fail(QE_ERR_INVALID_ARG, "rope: n_axes must be 1 .. 8");
    if (misaligned(a->positions, 4)) return fail(QE_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    if (a->positions && r->n_axes > 1 && a->pos_stride < total) return fail(QE_ERR_INVALID_ARG, "pos_stride is below total_q");
    p.R = r->rot_dim;
    p.halves = r->halves != 0 && r->rot_dim > 0;
    p.positions = a->positions;
    p.pos_stride = a->pos_stride;
    for (int i = 0; i < r->rot_dim / 2; ++i) {
      if (r->axis[i] < 0 || r->axis[i] >= r->n_axes) return fail(QE_ERR_INVALID_ARG, "rope: axis of pair %d out of range", i);
      const double f = r->inv_freq[i];
      if (!std::isfinite(f)) return fail(QE_ERR_INVALID_ARG, "rope: inv_freq of pair %d is not finite", i);
      p.axis[i] = r->axis[i];
      double turn = f * 0.15915494309189533577;   // 1 / (2 pi)
      turn -= std::floor(turn);
      p.turn[i] = turn >= 1.0 ? 0ull : static_cast<unsigned long long>(std::ldexp(turn, 64) < 0x1p64 ? std::ldexp(turn, 64) : 0.0);
    }
  } else if (a->positions) {
    return fail(QE_ERR_INVALID_ARG, "positions without rope");
  }
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.kts = a->k_token_stride;
  p.khs = a->k_head_stride;
  p.vts = a->v_token_stride;
  p.vhs = a->v_head_stride;
  p.qts = a->q_token_stride;
  p.qhs = a->q_head_stride;
  p.ots = a->q_out_token_stride;
  p.ohs = a->q_out_head_stride;
  p.layer = layer;
  p.Hq = a->n_q_heads;
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  return launched(qe::launch_pages_append(p, pages->dtype == QE_DTYPE_FP16, n_sm, static_cast<cudaStream_t>(stream)), "qe_pages_append");
}

qe_status qe_pages_attend_workspace(const qe_pages* pages, const qe_page_table* seqs, size_t* bytes) {
  qe::PagesView pg{};
  qe::TableView t{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_table(seqs, false, &t));
  if (!bytes) return fail(QE_ERR_INVALID_ARG, "bytes is null");
  *bytes = 0;
  if (!qe::pages_attend_cuts(pg, t)) return QE_OK;
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  *bytes = qe::pages_attend_bytes(n_sm, pg.D);
  return QE_OK;
}

qe_status qe_pages_attend(const qe_pages* pages, int layer, const qe_page_table* seqs, const qe_chunks* chunks,
                          const qe_pages_attend_args* a, void* workspace, size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_attend");
  qe::PagesAttendParams p{};
  bool some;
  QE_TRY(attend_params(pages, layer, seqs, chunks, a, &p, &some));
  if (!some) return QE_OK;
  return attend_launch("qe_pages_attend", pages, p, workspace, bytes, [&](int n_sm) { return attend_need(p, n_sm); }, [&](int n_sm) {
    return qe::launch_pages_attend(p, pages->dtype == QE_DTYPE_FP16, pages->device, n_sm, workspace, static_cast<cudaStream_t>(stream));
  });
}

qe_status qe_pages_attend_window(const qe_pages* pages, int layer, const qe_page_table* seqs, const qe_chunks* chunks,
                                 const qe_pages_attend_args* a, int window, int sinks, void* workspace, size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_attend_window");
  qe::PagesAttendParams p{};
  qe::PagesWindow w{};
  bool some;
  QE_TRY(attend_params(pages, layer, seqs, chunks, a, &p, &some));
  QE_TRY(check_window(window, sinks, &w));
  if (!a->causal) return fail(QE_ERR_INVALID_ARG, "a window needs causal attention");
  if (!some) return QE_OK;
  return attend_launch("qe_pages_attend_window", pages, p, workspace, bytes, [&](int n_sm) { return attend_need(p, n_sm); }, [&](int n_sm) {
    return qe::launch_pages_attend_window(p, w, pages->dtype == QE_DTYPE_FP16, pages->device, n_sm, workspace, static_cast<cudaStream_t>(stream));
  });
}

qe_status qe_pages_attend_shared_workspace(const qe_pages* pages, size_t* bytes) {
  qe::PagesView pg{};
  QE_TRY(check_pages(pages, &pg));
  if (!bytes) return fail(QE_ERR_INVALID_ARG, "bytes is null");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  *bytes = qe::pages_attend_bytes(n_sm, pg.D);
  return QE_OK;
}

qe_status qe_pages_attend_shared(const qe_pages* pages, int layer, const qe_page_table* seqs, const qe_chunks* chunks,
                                 const qe_pages_attend_args* a, const qe_groups* groups, void* workspace, size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_attend_shared");
  qe::PagesAttendParams p{};
  bool some;
  QE_TRY(attend_params(pages, layer, seqs, chunks, a, &p, &some));
  if (!groups) return fail(QE_ERR_INVALID_ARG, "groups is null");
  if (groups->n_groups < 0 || groups->n_groups > 65536 || groups->max_group_len < 0)
    return fail(QE_ERR_INVALID_ARG, "groups: n_groups must be 0 .. 65536 and max_group_len >= 0");
  if (misaligned(groups->group_start, 4) || misaligned(groups->prefix_len, 4))
    return fail(QE_ERR_INVALID_ARG, "groups: pointers must be 4-byte aligned");
  if (!some) return QE_OK;
  if (groups->n_groups == 0) return fail(QE_ERR_INVALID_ARG, "groups: the call's sequences are in no group");
  if (!groups->group_start || !groups->prefix_len) return fail(QE_ERR_INVALID_ARG, "groups: null pointer");
  // (the keys of a tile, a prefix and the own tokens of its sequences, are counted in 32 bits)
  const int per = 256 * p.pg.H / p.Hq;
  if (((long long)(p.c.n < per ? p.c.n : per) + 1) * p.t.cols * p.pg.S > 0x7FFFFFFF)
    return fail(QE_ERR_INVALID_ARG,
                "page table: too large for shared prefixes: (min(n_seqs, 256 n_kv_heads / n_q_heads) + 1) * max_pages * page_size must be below 2^31");
  const qe::PagesGroups g{groups->group_start, groups->prefix_len, groups->n_groups, groups->max_group_len};
  return attend_launch("qe_pages_attend_shared", pages, p, workspace, bytes, [&](int n_sm) { return qe::pages_attend_bytes(n_sm, p.pg.D); }, [&](int n_sm) {
    return qe::launch_pages_attend_shared(p, g, pages->dtype == QE_DTYPE_FP16, pages->device, n_sm, workspace, static_cast<cudaStream_t>(stream));
  });
}

qe_status qe_pages_drop(const qe_pages* pages, const qe_page_table* seqs, const int* rows, int n, int window, int sinks, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_drop");
  qe::PagesView pg{};
  qe::TableView t{};
  qe::PagesWindow w{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_table(seqs, true, &t));
  QE_TRY(check_window(window, sinks, &w));
  if (n < 0 || n > (1 << 24)) return fail(QE_ERR_INVALID_ARG, "n must be 0 .. 2^24");
  if (n == 0) return QE_OK;
  if (!rows || misaligned(rows, 4)) return fail(QE_ERR_INVALID_ARG, "rows must be non-null and 4-byte aligned");
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  return launched(qe::launch_pages_drop(pg, t, rows, n, w, n_sm, static_cast<cudaStream_t>(stream)), "qe_pages_drop");
}

qe_status qe_pages_manage_workspace(const qe_pages* pages, const qe_page_table* seqs, int n, size_t* bytes) {
  qe::PagesView pg{};
  qe::TableView t{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_table(seqs, false, &t));
  if (n < 0 || !bytes) return fail(QE_ERR_INVALID_ARG, "n must be >= 0 and bytes not null");
  *bytes = qe::pages_manage_bytes(pg.P, t.rows, n);
  return QE_OK;
}

static qe_status manage(const char* name, const qe_pages* pages, const qe_page_table* seqs, const int* a, const int* b, int n,
                        bool fork, void* workspace, size_t bytes, void* stream) {
  qe::PagesView pg{};
  qe::TableView t{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_table(seqs, true, &t));
  if (n < 0 || n > (1 << 24)) return fail(QE_ERR_INVALID_ARG, "n must be 0 .. 2^24");
  if (n == 0) return QE_OK;
  if (!a || (fork && !b) || misaligned(a, 4) || misaligned(b, 4)) return fail(QE_ERR_INVALID_ARG, "index arrays must be non-null and 4-byte aligned");
  QE_TRY(check_workspace(workspace, bytes, qe::pages_manage_bytes(pg.P, t.rows, n)));
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launched(fork ? qe::launch_pages_fork(pg, t, a, b, n, workspace, n_sm, st)
                       : qe::launch_pages_resize(pg, t, a, b, n, workspace, n_sm, st), name);
}

qe_status qe_pages_resize(const qe_pages* pages, const qe_page_table* seqs, const int* rows, const int* new_len, int n,
                          void* workspace, size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_resize");
  return manage("qe_pages_resize", pages, seqs, rows, new_len, n, false, workspace, bytes, stream);
}

qe_status qe_pages_fork(const qe_pages* pages, const qe_page_table* seqs, const int* src, const int* dst, int n, void* workspace,
                        size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_fork");
  return manage("qe_pages_fork", pages, seqs, src, dst, n, true, workspace, bytes, stream);
}

qe_status qe_pages_compact(const qe_pages* pages, const qe_page_table* seqs, int* table_out, int* refs_out, int* n_live,
                           void* workspace, size_t bytes, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_compact");
  qe::PagesView pg{};
  qe::TableView t{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_table(seqs, true, &t));
  if (!table_out != !refs_out) return fail(QE_ERR_INVALID_ARG, "table_out and refs_out go together");
  if (misaligned(table_out, 4) || misaligned(refs_out, 4) || misaligned(n_live, 4))
    return fail(QE_ERR_INVALID_ARG, "outputs must be 4-byte aligned");
  QE_TRY(check_workspace(workspace, bytes, qe::pages_manage_bytes(pg.P, t.rows, 0)));
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  return launched(qe::launch_pages_compact(pg, t, table_out ? table_out : t.table, refs_out ? refs_out : t.refs, n_live, workspace,
                                           n_sm, static_cast<cudaStream_t>(stream)), "qe_pages_compact");
}

qe_status qe_pages_copy(const qe_pages* pages, const int* src, const int* dst, int n, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_copy");
  qe::PagesView pg{};
  QE_TRY(check_pages(pages, &pg));
  if (n < 0) return fail(QE_ERR_INVALID_ARG, "n must be >= 0");
  if (n == 0) return QE_OK;
  if (!src || !dst || misaligned(src, 4) || misaligned(dst, 4))
    return fail(QE_ERR_INVALID_ARG, "src and dst must be non-null and 4-byte aligned");
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  return launched(qe::launch_pages_copy(pg, src, dst, n, n_sm, static_cast<cudaStream_t>(stream)), "qe_pages_copy");
}

qe_status qe_pages_gather(const qe_pages* pages, int layer, const qe_page_table* seqs, const int* rows, int n_seqs, int start,
                          int n_tokens, void* k_out, void* v_out, void* stream) {
  qe::NvtxRange nvtx_("qe_pages_gather");
  qe::PagesView pg{};
  qe::TableView t{};
  QE_TRY(check_pages(pages, &pg));
  QE_TRY(check_layer(pages, layer));
  QE_TRY(check_table(seqs, false, &t));
  if (n_seqs < 0 || start < 0 || n_tokens < 0 || start > 0x7FFFFFFF - 256 - n_tokens)
    return fail(QE_ERR_INVALID_ARG, "n_seqs, start and n_tokens must be >= 0, start + n_tokens below 2^31 - 256");
  if (n_seqs == 0 || n_tokens == 0) return QE_OK;
  if (!rows && n_seqs > t.rows) return fail(QE_ERR_INVALID_ARG, "n_seqs is above n_rows");
  if (!k_out || !v_out || misaligned(k_out, 16) || misaligned(v_out, 16) || misaligned(rows, 4))
    return fail(QE_ERR_INVALID_ARG, "k_out and v_out must be non-null and 16-byte aligned, rows 4-byte aligned");
  DeviceGuard guard(pages->device);
  if (guard.err != cudaSuccess) return cuda_fail(guard.err, "cudaSetDevice");
  int n_sm = 0;
  QE_TRY(sm_count(pages->device, &n_sm));
  return launched(qe::launch_pages_gather(pg, t, layer, rows, n_seqs, start, n_tokens, static_cast<uint16_t*>(k_out),
                                          static_cast<uint16_t*>(v_out), n_sm, static_cast<cudaStream_t>(stream)), "qe_pages_gather");
}

}  // extern "C"
