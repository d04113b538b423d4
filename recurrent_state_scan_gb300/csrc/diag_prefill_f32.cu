// diag_prefill_f32.cu -- the kernels of diag_prefill.cuh for fp32 rows.
#include "diag_prefill.cuh"

namespace gdn {
template cudaError_t diag_prefill_by_kind<float>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
