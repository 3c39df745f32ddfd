// qe_pages_window.cu -- attention over the cached pages with a sliding window and sinks: the kernels of qe_pages_halves.cuh and
// qe_pages_few.cuh, over the blocks that a tile's rows see (qe_pages_attn.cuh: pa_shift).
#include "qe_pages_launch.cuh"

namespace qe {

cudaError_t launch_pages_attend_window(const PagesAttendParams& a, const PagesWindow& w, int fp16, int device, int n_sm, void* ws, cudaStream_t st) {
  return launch_pages_mode<PA_WINDOW>(a, w, PagesGroups{}, fp16, device, n_sm, ws, st);
}

}  // namespace qe
