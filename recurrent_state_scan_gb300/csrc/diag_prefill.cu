// diag_prefill.cu -- how a call of the diagonal recurrence is laid out, and its dispatch (the kernel: diag_prefill.cuh).
#include "diag_internal.cuh"

namespace gdn {

int diag_slices(int channels) { return (int)(((int64_t)channels + kDiagSlice - 1) / kDiagSlice); }
int64_t diag_tiles(int64_t rows) { return (rows + kDiagTile - 1) / kDiagTile; }

size_t diag_walk_bytes(int64_t rows, int channels, size_t *zeroed) {
    const size_t items = (size_t)diag_tiles(rows) * diag_slices(channels);
    if (diag_tiles(rows) < 2) return *zeroed = 0;
    *zeroed = 256 + (items * 4 + 255) / 256 * 256;
    return *zeroed + items * (sizeof(float4) + 2 * sizeof(float2)) * 32;
}
void diag_walk_layout(DiagParams &p, void *workspace) {
    size_t zeroed;
    if (diag_walk_bytes(p.rows, p.channels, &zeroed) == 0) return;
    uint8_t *at = static_cast<uint8_t *>(workspace);
    const size_t items = (size_t)diag_tiles(p.rows) * diag_slices(p.channels);
    p.ticket = reinterpret_cast<uint32_t *>(at);
    p.flags = reinterpret_cast<uint32_t *>(at + 256);
    p.product = reinterpret_cast<float4 *>(at + zeroed);
    p.shift = reinterpret_cast<float2 *>(p.product + items * 32);
    p.after = p.shift + items * 32;
}
cudaError_t diag_clear(const DiagParams &p, cudaStream_t stream) {
    size_t zeroed;
    return diag_walk_bytes(p.rows, p.channels, &zeroed) == 0 ? cudaSuccess : cudaMemsetAsync(p.ticket, 0, zeroed, stream);
}
unsigned diag_grid(const DiagParams &p, int per_sm) {
    const int64_t items = diag_tiles(p.rows) * diag_slices(p.channels), most = 152 * per_sm;
    return (unsigned)(items < 1 ? 1 : diag_tiles(p.rows) < 2 || items < most ? items : most);
}

cudaError_t launch_diag_prefill(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream) {
    switch (io) {
        case GDN_F32: return diag_prefill_by_kind<float>(p, gate, weighting, stream);
        case GDN_BF16: return diag_prefill_by_kind<__nv_bfloat16>(p, gate, weighting, stream);
        default: return diag_prefill_by_kind<__half>(p, gate, weighting, stream);
    }
}

}  // namespace gdn
