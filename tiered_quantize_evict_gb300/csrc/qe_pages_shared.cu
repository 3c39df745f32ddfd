// qe_pages_shared.cu -- attention over the cached pages for sequences that share prefixes: the kernels of qe_pages_halves.cuh and
// qe_pages_few.cuh, over the line of groups (qe_pages_shared.cuh).
#include "qe_pages_launch.cuh"

namespace qe {

cudaError_t launch_pages_attend_shared(const PagesAttendParams& a, const PagesGroups& g, int fp16, int device, int n_sm, void* ws, cudaStream_t st) {
  return launch_pages_mode<PA_SHARED>(a, PagesWindow{}, g, fp16, device, n_sm, ws, st);
}

}  // namespace qe
