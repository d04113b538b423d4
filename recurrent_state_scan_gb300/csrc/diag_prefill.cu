// diag_prefill.cu -- how a call of the diagonal recurrence is laid out, and its dispatch (the kernel: diag_prefill.cuh).
#include "diag_internal.cuh"

namespace gdn {

int diag_slices(int channels) { return (int)(((int64_t)channels + kDiagSlice - 1) / kDiagSlice); }
// CTAs of a cluster: as many as there are tiles, up to the 8 that every GPU can hold together.
int diag_cluster(int64_t rows) {
    const int64_t tiles = (rows + kDiagTile - 1) / kDiagTile;
    return tiles >= 8 ? 8 : tiles > 4 ? 8 : tiles > 2 ? 4 : tiles > 1 ? 2 : 1;
}
// Stretches of whole sequences side by side, where one cluster to a slice leaves SMs idle: up to
// three CTAs for each of 152 SMs, at least 8 tiles to a part.
int diag_parts(int64_t rows, int64_t num_seqs, int channels) {
    const int64_t ctas = (int64_t)diag_slices(channels) * diag_cluster(rows), tiles = (rows + kDiagTile - 1) / kDiagTile;
    int64_t parts = 456 / ctas;
    if (parts > tiles / 8) parts = tiles / 8;
    if (parts > num_seqs) parts = num_seqs;
    return parts < 1 ? 1 : (int)parts;
}

cudaError_t launch_diag_prefill(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream) {
    switch (io) {
        case GDN_F32: return diag_prefill_by_kind<float>(p, gate, weighting, stream);
        case GDN_BF16: return diag_prefill_by_kind<__nv_bfloat16>(p, gate, weighting, stream);
        default: return diag_prefill_by_kind<__half>(p, gate, weighting, stream);
    }
}

}  // namespace gdn
