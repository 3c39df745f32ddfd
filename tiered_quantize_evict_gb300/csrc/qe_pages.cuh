// qe_pages.cuh -- parameters and launchers of the paged cache's kernels (include/qe.h, "paged cache").
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "qe.h"

namespace qe {

// The pool as the kernels see it: strides in elements (0 for an axis of one entry).
struct PagesView {
  uint16_t* k;
  uint16_t* v;
  long long ls, ps, hs, ts;   // layer, page, head, token
  int L, P, H, S, lgS, D;     // layers, pages, KV heads, page size and its log2, head_dim
  unsigned* err;
};

struct TableView {
  int* table;
  int* kv_len;
  int* refs;
  long long stride;
  int rows, cols;
};

struct ChunksView {
  const int* q_start;
  const int* rows;
  int n, total;
};

struct PagesAppendParams {
  PagesView pg;
  TableView t;
  ChunksView c;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  long long kts, khs, vts, vhs, qts, qhs, ots, ohs;
  int layer, Hq;
  int R, halves;              // rotated channels (0: none)
  const int* positions;
  long long pos_stride;
  signed char axis[64];
  unsigned long long turn[64];   // inv_freq / (2 pi) mod 1, in units of 2^-64 turns
};

struct PagesAttendParams {
  PagesView pg;
  TableView t;
  ChunksView c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  long long qts, qhs, ots, ohs;
  int layer, Hq, causal, max_q_len;
  int expire;                 // qe_debug_inject (qe_pages_attn.cuh); 0: none
  float scale;
};

// what a planned resize or fork does to one row (written by the planning kernel)
struct PagesRowMove {
  int row, src;          // row changed; fork: source row, else -1.  row < 0: nothing
  int old_len, new_len;
  int first_new;         // index of the row's first page in the list of pages taken
  int copy_page;         // page that takes the partly filled page's copy, or -1
};
struct PagesPair {
  int src, dst, rows, refs;   // copy `rows` tokens of page src to dst
};

cudaError_t launch_pages_append(const PagesAppendParams& p, int fp16, int n_sm, cudaStream_t st);
cudaError_t launch_pages_attend(const PagesAttendParams& p, int fp16, int device, int n_sm, void* ws, cudaStream_t st);
size_t pages_attend_bytes(int n_sm, int D);
bool pages_attend_cuts(const PagesView& pg, const TableView& t);   // whether any row of the table may be cut (and needs workspace)
cudaError_t launch_pages_resize(const PagesView& pg, const TableView& t, const int* rows, const int* new_len, int n, void* ws,
                                int n_sm, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesView& pg, const TableView& t, const int* src, const int* dst, int n, void* ws,
                              int n_sm, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesView& pg, const TableView& t, int* table_out, int* refs_out, int* n_live, void* ws,
                                 int n_sm, cudaStream_t st);
cudaError_t launch_pages_copy(const PagesView& pg, const int* src, const int* dst, int n, int n_sm, cudaStream_t st);
cudaError_t launch_pages_gather(const PagesView& pg, const TableView& t, int layer, const int* rows, int n, int start, int n_tok,
                                uint16_t* k, uint16_t* v, int n_sm, cudaStream_t st);
size_t pages_manage_bytes(int n_pages, int n_rows, int n);

// qe_host.cu: the message behind qe_last_error(NULL)
void set_global_error(const char* msg);
// qe_host.cu: the injected expiry of the next attention, once
int take_pages_expire();

#if defined(__CUDACC__)
__device__ __forceinline__ void pages_report(const PagesView& pg, unsigned bit) {
  if (pg.err) atomicOr(pg.err, bit);
}

// the most tokens a row can have
__device__ __forceinline__ long long pages_most(const PagesView& pg, const TableView& t) {
  const long long m = (long long)t.cols << pg.lgS;
  return m < (1ll << 30) ? m : 1ll << 30;
}

// Length of a row, within what its table can hold; 0 (reported) for a row that does not exist.
__device__ __forceinline__ int row_len(const PagesView& pg, const TableView& t, int row, bool report) {
  bool bad = row < 0 || row >= t.rows;
  int len = 0;
  if (!bad) {
    const int x = t.kv_len[row];
    const long long most = pages_most(pg, t);
    len = x < 0 ? 0 : (x > most ? (int)most : x);
    bad = x != len;
  }
  if (bad && report) pages_report(pg, QE_PAGES_ERR_ROW);
  return len;
}

// One sequence of a call: its packed tokens [q0, q0 + m), its row and its length, all within bounds
// (a row that does not exist has length 0).
struct SeqInfo {
  int q0, m, row, len;
};
__device__ __forceinline__ SeqInfo seq_info(const PagesView& pg, const TableView& t, const ChunksView& c, int s, bool report) {
  SeqInfo r;
  const int a = c.q_start[s], b = c.q_start[s + 1];
  r.q0 = min(max(a, 0), c.total);
  const int q1 = min(max(b, r.q0), c.total);
  r.m = q1 - r.q0;
  r.row = c.rows ? c.rows[s] : s;
  r.len = row_len(pg, t, r.row, report);   // (before q_start is looked at: their loads go together)
  if ((a != r.q0 || b != q1) && report) pages_report(pg, QE_PAGES_ERR_ROW);
  return r;
}

// reports a q_start that decreases or leaves [0, total] (called by one block's threads)
__device__ __forceinline__ void check_starts(const PagesView& pg, const ChunksView& c) {
  bool bad = false;
  for (int i = threadIdx.x; i < c.n; i += blockDim.x) {
    const int a = c.q_start[i], b = c.q_start[i + 1];
    bad |= a < 0 || b < a || b > c.total;
  }
  if (bad) pages_report(pg, QE_PAGES_ERR_ROW);
}

// page of position pos of a row, or -1 (reported) when the table names none
__device__ __forceinline__ int page_at(const PagesView& pg, const TableView& t, int row, int pos) {
  const int p = t.table[(long long)row * t.stride + (pos >> pg.lgS)];
  if (p >= 0 && p < pg.P) return p;
  pages_report(pg, QE_PAGES_ERR_PAGE);
  return -1;
}
#endif

}  // namespace qe
