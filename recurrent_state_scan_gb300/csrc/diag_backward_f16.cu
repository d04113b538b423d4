// diag_backward_f16.cu -- the kernels of diag_backward.cuh for float16 rows.
#include "diag_backward.cuh"

namespace gdn {
template cudaError_t diag_backward_by_kind<__half>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
