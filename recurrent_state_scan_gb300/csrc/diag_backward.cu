// diag_backward.cu -- the dispatch of the diagonal recurrence's backward pass (the kernel: diag_backward.cuh), and its sums over
// several parts.
#include "diag_internal.cuh"

namespace gdn {
namespace {

// The parts' sums in their order.
__global__ void diag_sum_parts(const __grid_constant__ DiagParams p) {
    if (!offsets_ok(p)) return;
    const int64_t C = p.channels, ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int k = blockIdx.y;
    float *out = k == 0 ? p.dA_log : k == 1 ? p.da_bias : p.db_bias;
    if (ch >= C || out == nullptr) return;
    float t = 0.f;
    for (int q = 0; q < p.parts; ++q) t += p.partial[((int64_t)q * 3 + k) * C + ch];
    out[ch] = t;
}

}  // namespace

cudaError_t launch_diag_backward(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream) {
    cudaError_t e;
    switch (io) {
        case GDN_F32: e = diag_backward_by_kind<float>(p, gate, weighting, stream); break;
        case GDN_BF16: e = diag_backward_by_kind<__nv_bfloat16>(p, gate, weighting, stream); break;
        default: e = diag_backward_by_kind<__half>(p, gate, weighting, stream);
    }
    if (e != cudaSuccess || p.parts == 1 || !(p.dA_log || p.da_bias || p.db_bias)) return e;
    diag_sum_parts<<<dim3((p.channels + 255) / 256, 3), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
