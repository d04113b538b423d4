// diag_prefill.cu -- the diagonal recurrence h_t = alpha_t h_{t-1} + w_t i_t x_t over whole sequences.
//
// A cluster of CTAs walks down the rows of one slice of 64 channels, a tile of 64 rows to a CTA and step.
// A warp holds LT rows of the slice (two channels to a lane) as (alpha, w i x) in registers: it folds them to
// a map h -> P h + H, the CTA folds its warps' maps, the cluster its CTAs' (through shared memory, in
// the order of the rows, so results do not depend on timing), and then the warp knows the h before its first row
// and runs its rows once more from the registers.  Every input is read once and every output written once; all
// sequences are one run of rows with edges where h starts anew, so short and long ones cost the same.
#include "diag_internal.cuh"

namespace gdn {
namespace {

template <typename IO, int GATE, int WEIGHT, int LT>
__global__ void __launch_bounds__(kDiagTile / LT * 32) diag_prefill_kernel(const __grid_constant__ DiagParams p) {
    constexpr int W = kDiagTile / LT;
    __shared__ DiagMaps maps[2][W], cta_maps[2][8];
    __shared__ int edge_first[W][LT + 1], edge_last[W][LT + 1];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, cl = gridDim.x, rank = blockIdx.x, slice = blockIdx.y;
    const int64_t C = p.channels, c = (int64_t)slice * kDiagSlice + 2 * lane;
    if (!offsets_ok(p)) return;
    const DiagPart part = diag_part(p, blockIdx.z, lane);
    for (int n = part.n0 + rank * W + w; n < part.n1; n += cl * W) {     // sequences without tokens keep their state
        if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
        store_state(p.state_out + n * C, p.state_in ? load_state(p.state_in + n * C, c, C) : both(0.f), c, C);
    }
    if (part.r0 >= part.r1) return;
    if (cl > 1) cluster_arrive();
    const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, C);
    const bool fast = p.pairs && (slice + 1) * kDiagSlice <= C, has_b = p.has_b;
    const int64_t tile0 = part.r0 / kDiagTile, tiles = (part.r1 + kDiagTile - 1) / kDiagTile - tile0, lo = part.r0, hi = part.r1;
    const int slices = gridDim.y;
    F2 carry = both(0.f);
    int from = part.n0;
    for (int64_t j0 = 0, step = 0; j0 < tiles; j0 += cl, ++step) {
        const int64_t tile = tile0 + j0 + rank, w0 = tile * kDiagTile + w * LT;
        const int buf = step & 1;
        const bool some = w0 < hi && w0 + LT > lo;
        F2 alpha[LT], u[LT], sum_g = both(0.f), H = both(0.f);
        uint32_t edges = 0;
        bool anew = false;
        if (some) {
            typename Pair<IO>::Raw x[LT], a[LT], b[LT];
            load_rows<IO, LT>(x, (const IO *)p.x, p.ld_x, w0, lo, hi, c, C, fast);
            load_rows<IO, LT>(a, (const IO *)p.a, p.ld_a, w0, lo, hi, c, C, fast);
            if (has_b) load_rows<IO, LT>(b, (const IO *)p.b, p.ld_b, w0, lo, hi, c, C, fast);
            edges = find_edges<LT>(p, (uint32_t)w0, from, edge_first[w], edge_last[w], lane);
#pragma unroll
            for (int t = 0; t < LT; ++t) {
                const DiagGates o = diag_gates<GATE, WEIGHT, false>(Pair<IO>::wide(a[t]), has_b ? Pair<IO>::wide(b[t]) : both(0.f), has_b, l);
                F2 v = mul2(o.i, Pair<IO>::wide(x[t]));
                v = WEIGHT == GDN_DIAG_PLAIN ? v : mul2(o.w, v);
                const bool in = w0 + t >= lo && w0 + t < hi;
                alpha[t] = in ? o.alpha : both(1.f);
                u[t] = in ? v : both(0.f);
                if (in && (edges >> t & 1)) {       // a sequence's first row
                    if (p.state_in) u[t] = fma2(alpha[t], load_state(p.state_in + edge_last[w][t] * C, c, C), u[t]);
                    anew = true;
                    H = u[t];
                } else {
                    H = fma2(alpha[t], H, u[t]);
                }
                if (in) sum_g = add2(sum_g, o.g);
            }
            if (p.codes) {
                const uint64_t at = (uint64_t)slice * p.rows + w0, all = (uint64_t)slices * p.rows;
                uint32_t mine[3] = {0, 0, 0};
#pragma unroll
                for (int t = 0; t < LT; ++t) {
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        if (k == 2 && !has_b) break;
                        const F2 v = Pair<IO>::wide(k == 0 ? x[t] : k == 1 ? a[t] : b[t]);
                        const uint32_t e = code_step(__reduce_max_sync(~0u, magnitude(v)));
                        const float inv = code_inverse(e);
                        if (lane == t) mine[k] = e;
                        if (w0 + t >= lo && w0 + t < hi)
                            *reinterpret_cast<char2 *>(p.codes + (k * all + at + t) * kDiagSlice + 2 * lane) =
                                make_char2((signed char)code_of(v.x, inv), (signed char)code_of(v.y, inv));
                    }
                }
                if (lane < LT && w0 + lane >= lo && w0 + lane < hi) {
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        if (k < 2 || has_b) p.steps[k * all + at + lane] = (uint8_t)mine[k];
                }
            }
        }
        put_map(maps[buf][w], lane, diag_product(sum_g, anew), H);
        __syncthreads();
        F2 h = carry;
        if (cl > 1) {
            DiagProduct all = get_product(maps[buf][0], lane);
            F2 shift = get_pair(maps[buf][0].shift, lane);
#pragma unroll
            for (int k = 1; k < W; ++k) {
                const DiagProduct m = get_product(maps[buf][k], lane);
                shift = diag_apply(m, get_pair(maps[buf][k].shift, lane), shift);
                all = diag_join(all, m);
            }
            if (step == 0) cluster_wait();      // (every CTA of the cluster has started)
            for (int r = w; r < cl; r += W) put_map_at(cta_maps[buf][rank], r, lane, all, shift);
            cluster_arrive();
            cluster_wait();
            for (int r = 0; r < cl; ++r) {
                if (r == rank) h = carry;
                carry = diag_apply(get_product(cta_maps[buf][r], lane), get_pair(cta_maps[buf][r].shift, lane), carry);
            }
        }
        if (p.kept && w == 0 && tile * kDiagTile > lo && tile * kDiagTile < hi)
            *reinterpret_cast<float2 *>(p.kept + (tile * slices + slice) * kDiagSlice + 2 * lane) = make_float2(h.x, h.y);
        F2 hw = h;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (k == w) hw = h;
            h = diag_apply(get_product(maps[buf][k], lane), get_pair(maps[buf][k].shift, lane), h);
        }
        if (cl == 1) carry = h;
        if (some) {
            IO *y = (IO *)p.y + w0 * p.ld_y + c;
#pragma unroll
            for (int t = 0; t < LT; ++t) {
                if (w0 + t < lo || w0 + t >= hi) continue;
                hw = edges >> t & 1 ? u[t] : fma2(alpha[t], hw, u[t]);
                store_pair<IO>(y + t * p.ld_y, hw, c, C, fast);
                if (edges >> (t + 1) & 1) store_state(p.state_out + (edge_first[w][t + 1] - 1) * C, hw, c, C);
            }
        }
        __syncwarp();       // (the next step's edges overwrite these)
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    constexpr int LT = 8;
    cudaLaunchConfig_t cfg{};
    const int cl = diag_cluster(p.rows);
    cfg.gridDim = dim3(cl, diag_slices(p.channels), p.parts);
    cfg.blockDim = dim3(kDiagTile / LT * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, diag_prefill_kernel<IO, GATE, WEIGHT, LT>, p);
}

template <typename IO> cudaError_t by_kind(const DiagParams &p, int gate, int weighting, cudaStream_t s) {
    if (gate == GDN_DIAG_SOFTPLUS)
        return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_NORM>(p, s)
               : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_COMPLEMENT>(p, s)
                                                  : launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_PLAIN>(p, s);
    return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_NORM>(p, s)
           : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_COMPLEMENT>(p, s)
                                              : launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_PLAIN>(p, s);
}

}  // namespace

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
        case GDN_F32: return by_kind<float>(p, gate, weighting, stream);
        case GDN_BF16: return by_kind<__nv_bfloat16>(p, gate, weighting, stream);
        default: return by_kind<__half>(p, gate, weighting, stream);
    }
}

}  // namespace gdn
