// diag_backward.cu -- the dispatch of the diagonal recurrence's backward pass (the kernel: diag_backward.cuh), and its sums over
// the tiles.
#include "diag_internal.cuh"

namespace gdn {
namespace {

// The tiles' sums: 8 threads to a channel, each over every 8th tile, then the 8 in their order.
__global__ void __launch_bounds__(256) diag_sum_tiles(const __grid_constant__ DiagParams p) {
    if (!offsets_ok(p)) return;
    __shared__ float part[8][32];
    const int tiles = (int)((p.rows + kDiagTile - 1) / kDiagTile), k = blockIdx.y, lane = threadIdx.x % 32, r = threadIdx.x / 32;
    const int64_t C = p.channels, ch = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (ch < C) {
#pragma unroll 4
        for (int j = r; j < tiles; j += 8) t += p.partial[((int64_t)j * 3 + k) * C + ch];
    }
    part[r][lane] = t;
    __syncthreads();
    float *out = k == 0 ? p.dA_log : k == 1 ? p.da_bias : p.db_bias;
    if (r > 0 || ch >= C || out == nullptr) return;
    for (int q = 1; q < 8; ++q) t += part[q][lane];
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
    if (e != cudaSuccess || diag_tiles(p.rows) == 1 || !(p.dA_log || p.da_bias || p.db_bias)) return e;
    diag_sum_tiles<<<dim3((p.channels + 31) / 32, 3), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
