// diag_prefill.cu -- how a call of the diagonal recurrence is laid out, and its dispatch (the kernel: diag_prefill.cuh).
#include "diag_internal.cuh"

namespace gdn {

int diag_slices(int channels) { return (int)(((int64_t)channels + kDiagSlice - 1) / kDiagSlice); }
int64_t diag_tiles(int64_t rows) { return (rows + kDiagTile - 1) / kDiagTile; }

namespace {
struct WalkLayout {
    size_t table, words, total;      // behind the counter, which comes first
};
WalkLayout walk_layout(int64_t rows, int channels) {
    const size_t slices = diag_slices(channels), items = (size_t)diag_tiles(rows) * slices;
    WalkLayout l;
    l.table = 256;
    l.words = l.table + 5 * slices * kDiagSlice * sizeof(float);
    l.total = l.words + items * 128 * sizeof(unsigned long long);
    return l;
}

__global__ void __launch_bounds__(256) diag_begin_kernel(const __grid_constant__ DiagParams p, uint32_t items) {
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, all = gridDim.x * 256;
    if (i == 0) *p.ticket = 0u;
    static_assert(kNone == ~0ull, "all bits set");
    for (uint64_t k = i; k < (uint64_t)items * 64; k += all) reinterpret_cast<uint4 *>(p.words)[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
    const int slices = (p.channels + kDiagSlice - 1) / kDiagSlice, row = slices * kDiagSlice;
    for (int c = 2 * (int)i; c < row; c += 2 * (int)all) {
        const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, p.channels);
        const F2 v[5] = {l.rate, l.ninverse, l.abias, l.nabias, l.nbbias};
        for (int k = 0; k < 5; ++k) *reinterpret_cast<float2 *>(p.table + (int64_t)k * row + c) = make_float2(v[k].x, v[k].y);
    }
}
}  // namespace

size_t diag_walk_bytes(int64_t rows, int channels) { return diag_tiles(rows) < 2 ? 0 : walk_layout(rows, channels).total; }
void diag_walk_layout(DiagParams &p, void *workspace) {
    const uint32_t slices = diag_slices(p.channels);
    int bits = 0;
    while ((1ull << bits) < slices) ++bits;
    p.magic = (uint32_t)(((1ull << (31 + bits)) + slices - 1) / slices);
    p.magic_shift = 31 + bits;
    if (diag_tiles(p.rows) < 2) return;
    const WalkLayout l = walk_layout(p.rows, p.channels);
    uint8_t *at = static_cast<uint8_t *>(workspace);
    p.ticket = reinterpret_cast<uint32_t *>(at);
    p.table = reinterpret_cast<float *>(at + l.table);
    p.words = reinterpret_cast<unsigned long long *>(at + l.words);
}
cudaError_t diag_begin(const DiagParams &p, cudaStream_t stream) {
    if (diag_tiles(p.rows) < 2) return cudaSuccess;
    const uint32_t items = (uint32_t)(diag_tiles(p.rows) * diag_slices(p.channels)), blocks = (items * 64ull + 1023) / 1024;
    diag_begin_kernel<<<blocks < 16 ? 16 : blocks > 1216 ? 1216 : blocks, 256, 0, stream>>>(p, items);
    return cudaGetLastError();
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
