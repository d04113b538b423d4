// diag_backward_bf16.cu -- the kernels of diag_backward.cuh for bfloat16 rows.
#include "diag_backward.cuh"

namespace gdn {
template cudaError_t diag_backward_by_kind<__nv_bfloat16>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
