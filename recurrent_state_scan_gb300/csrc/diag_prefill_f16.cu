// diag_prefill_f16.cu -- the kernels of diag_prefill.cuh for float16 rows.
#include "diag_prefill.cuh"

namespace gdn {
template cudaError_t diag_prefill_by_kind<__half>(const DiagParams &p, int gate, int weighting, cudaStream_t s);
}  // namespace gdn
