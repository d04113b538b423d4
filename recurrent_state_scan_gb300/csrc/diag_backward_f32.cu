// diag_backward_f32.cu -- the kernels of diag_backward.cuh for fp32 rows.
#include "diag_backward.cuh"

namespace gdn {
template cudaError_t diag_backward_by_kind<float>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
