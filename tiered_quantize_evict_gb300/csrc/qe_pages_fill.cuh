// qe_pages_fill.cuh -- the parities of a buffer that copies fill and products empty in turn.  Host and device: the host test builds
// it and follows it with simulated barriers.
#pragma once
#include "qe_common.cuh"

namespace qe {

// Two mbarriers, `full` completed by each copy, `empty` by the products that read it.  To be counted (++sent) once a copy is sent,
// not before: what a failed wait leaves must still name the last copy, which has to land before its shared memory is given up.
struct PaFill {
  int sent = 0;
  QE_HD unsigned empty() const { return (unsigned)(sent & 1) ^ 1u; }   // of `empty`: the last copy's products are done (at first: nothing to wait for)
  QE_HD unsigned landed() const { return (unsigned)(sent - 1) & 1u; }   // of `full`: the last copy is there (sent > 0)
};

}  // namespace qe
