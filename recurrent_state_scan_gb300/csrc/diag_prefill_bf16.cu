// diag_prefill_bf16.cu -- the kernels of diag_prefill.cuh for bfloat16 rows.
#include "diag_prefill.cuh"

namespace gdn {
template cudaError_t diag_prefill_by_kind<__nv_bfloat16>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
