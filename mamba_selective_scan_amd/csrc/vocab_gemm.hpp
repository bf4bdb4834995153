// vocab_gemm.hpp -- the three products of the losses over a vocabulary.
#pragma once

#include <algorithm>

#include "mss_train.hpp"

namespace mss {

// logits of the piece's rows: stats, and with `keep` the codes or logits
hipError_t launch_logits(const LossArgs& a, int first, bool io_bf16, bool keep, hipStream_t stream);
// part = dz weight, by splits of the vocabulary
hipError_t launch_dx(const LossArgs& a, int first, hipStream_t stream);
// dweight = dz^T x, or its sum over the pieces so far
hipError_t launch_dw(const LossArgs& a, int first, bool io_bf16, hipStream_t stream);

}  // namespace mss
