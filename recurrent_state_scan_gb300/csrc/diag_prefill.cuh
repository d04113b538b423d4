// diag_prefill.cuh -- the diagonal recurrence h_t = alpha_t h_{t-1} + w_t i_t x_t over whole sequences.
//
// A cluster of CTAs walks down the rows of one slice of 64 channels, a tile of 64 rows to a CTA and step.
// A warp stages its 8 rows in shared memory, takes them into registers as (alpha, w i x), two channels to a lane,
// has the next step's rows fetched in their place, and folds its own to a map h -> P h + H.  The CTA folds its warps' maps,
// the cluster its CTAs' (through shared memory, in the order of the rows, so results do not depend on timing); then
// the warp knows the h before its first row and runs its rows once more from the registers.  Every input is read once
// and every output written once; all sequences are one run of rows with edges where h starts anew, so short and
// long ones cost the same.
#pragma once

#include <type_traits>

#include "diag_internal.cuh"

namespace gdn {
namespace {

constexpr int LT = 8, W = kDiagTile / LT;      // a warp's rows; warps

template <typename IO> struct Shared {
    IO rows[W][3][LT][kDiagSlice];              // x, a, b
    DiagMaps maps[W], before[W], cta_maps[2][8];    // a warp's rows; the tile's rows before them; the cluster's tiles
    float2 start[32];                               // h before the tile
    int edge_first[W][LT + 1], edge_last[W][LT + 1];
};

template <typename IO, int GATE, int WEIGHT, bool CODES>
__global__ void __launch_bounds__(W * 32, 3) diag_prefill_kernel(const __grid_constant__ DiagParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Shared<IO> &sh = *reinterpret_cast<Shared<IO> *>(raw_shared);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, cl = gridDim.x, rank = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
    const int C = p.channels, c0 = slice * kDiagSlice, c = c0 + 2 * lane;
    if (!offsets_ok(p)) return;
    const DiagPart part = diag_part(p, blockIdx.z, lane);
    for (int n = part.n0 + rank * W + w; n < part.n1; n += cl * W) {     // sequences without tokens keep their state
        if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
        store_state(p.state_out + (int64_t)n * C, p.state_in ? load_state(p.state_in + (int64_t)n * C, c, C) : both(0.f), c, C);
    }
    if (part.r0 >= part.r1) return;
    if (cl > 1) cluster_arrive();
    const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, C);
    const bool fast = p.pairs && c0 + kDiagSlice <= C, has_b = p.has_b, near = diag_near<GATE>(l);
    const int tile0 = part.r0 / kDiagTile, tiles = (part.r1 + kDiagTile - 1) / kDiagTile - tile0, lo = part.r0, hi = part.r1;
    IO *sx = &sh.rows[w][0][0][0], *sa = &sh.rows[w][1][0][0], *sb = &sh.rows[w][2][0][0];
    const uint32_t shut = infinity_bits<IO>(true);
    if (!has_b) fill_rows<IO, LT>(sb, infinity_bits<IO>(false), lane);
    auto stage = [&](int w0) {
        stage_rows<IO, LT>(sx, (const IO *)p.x, p.ld_x, w0, lo, hi, c0, C, p.wide, 0u, lane);
        stage_rows<IO, LT>(sa, (const IO *)p.a, p.ld_a, w0, lo, hi, c0, C, p.wide, shut, lane);
        if (has_b) stage_rows<IO, LT>(sb, (const IO *)p.b, p.ld_b, w0, lo, hi, c0, C, p.wide, 0u, lane);
        stage_commit();
    };
    stage((tile0 + rank) * kDiagTile + w * LT);
    EdgeWindow window = edge_window(p, part.n0, lane);
    F2 carry = both(0.f);
    for (int j0 = 0, step = 0; j0 < tiles; j0 += cl, ++step) {
        const int tile = tile0 + j0 + rank, w0 = tile * kDiagTile + w * LT;
        const int buf = step & 1;
        const bool some = w0 < hi && w0 + LT > lo, full = w0 >= lo && w0 + LT <= hi;
        F2 alpha[LT], u[LT], sum_G = both(0.f), H = both(0.f);
        uint32_t begins = 0, ends = 0;
        if (some) {
            const uint32_t edges = find_edges<LT>(p, window, (uint32_t)w0, part.n0, 0, sh.edge_first[w], sh.edge_last[w], lane);
            uint32_t live = (1u << LT) - 1;
            if (!full) {
                if (w0 < lo) live &= ~0u << (lo - w0);
                if (w0 + LT > hi) live &= (1u << (hi - w0)) - 1;
            }
            begins = edges & live;
            ends = edges >> 1 & live;
        }
        stage_wait();
        if (some) {
            auto take = [&](auto only_near) {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    const F2 G = diag_exponent<GATE>(staged(sa, t, lane), l), i = diag_sigmoid(staged(sb, t, lane), l.nbbias);
                    const DiagDecay d = diag_decay<decltype(only_near)::value>(G);
                    const F2 v = mul2(i, staged(sx, t, lane));
                    alpha[t] = d.alpha;
                    u[t] = WEIGHT == GDN_DIAG_PLAIN ? v : mul2(diag_weigh<WEIGHT>(d.n).w, v);
                    sum_G = add2(sum_G, G);
                }
            };
            if (near) take(std::true_type{});
            else take(std::false_type{});
            if (CODES) {
                const int64_t all = (p.rows + kDiagTile - 1) / kDiagTile * kDiagTile;
#pragma unroll 1
                for (int k = 0; k < (has_b ? 3 : 2); ++k) {
                    const IO *from = sx + k * LT * kDiagSlice;
                    const int64_t at = (k * slices + slice) * all + w0;
                    uint32_t mine = 0;
#pragma unroll
                    for (int t = 0; t < LT; ++t) {
                        const F2 v = staged(from, t, lane);
                        const uint32_t e = code_step(__reduce_max_sync(~0u, magnitude(v)));
                        if (lane == t) mine = e;
                        if (full || (w0 + t >= lo && w0 + t < hi))
                            *reinterpret_cast<uint16_t *>(p.codes + (at + t) * kDiagSlice + 2 * lane) = (uint16_t)codes_of(v, e);
                    }
                    if (lane < LT && w0 + lane >= lo && w0 + lane < hi) p.steps[at + lane] = (uint8_t)mine;
                }
            }
        }
        __syncwarp();
        if (j0 + cl < tiles) stage(w0 + cl * kDiagTile);
        if (some) {
            if (begins == 0) {
#pragma unroll
                for (int t = 0; t < LT; ++t) H = fma2(alpha[t], H, u[t]);
            } else {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    if (begins >> t & 1) {          // a sequence's first row
                        if (p.state_in) u[t] = fma2(alpha[t], load_state(p.state_in + (int64_t)sh.edge_last[w][t] * C, c, C), u[t]);
                        H = u[t];
                    } else {
                        H = fma2(alpha[t], H, u[t]);
                    }
                }
            }
        }
        put_map(sh.maps[w], lane, diag_product(sum_G, begins != 0), H);
        __syncthreads();
        DiagProduct all;
        F2 shift;
        if (w == 0) {
            all = get_product(sh.maps[0], lane);
            shift = get_pair(sh.maps[0].shift, lane);
#pragma unroll
            for (int k = 1; k < W; ++k) {
                put_map(sh.before[k], lane, all, shift);
                const DiagProduct m = get_product(sh.maps[k], lane);
                shift = diag_apply(m, get_pair(sh.maps[k].shift, lane), shift);
                all = diag_join(all, m);
            }
        }
        if (cl > 1) {
            if (step == 0) cluster_wait();      // (every CTA of the cluster has started)
            if (w == 0) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (r >= cl) break;
                    put_map_at(sh.cta_maps[buf][rank], r, lane, all, shift);
                }
            }
            cluster_arrive();
            cluster_wait();
        }
        if (w == 0) {
            F2 h = carry;
            if (cl > 1) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (r >= cl) break;
                    if (r == rank) h = carry;
                    carry = diag_apply(get_product(sh.cta_maps[buf][r], lane), get_pair(sh.cta_maps[buf][r].shift, lane), carry);
                }
            } else {
                carry = diag_apply(all, shift, carry);
            }
            sh.start[lane] = make_float2(h.x, h.y);
            if (p.kept && tile * kDiagTile > lo && tile * kDiagTile < hi)
                *reinterpret_cast<float2 *>(p.kept + ((int64_t)tile * slices + slice) * kDiagSlice + 2 * lane) = make_float2(h.x, h.y);
        }
        __syncthreads();
        F2 hw = get_pair(sh.start, lane);
        if (w > 0) hw = diag_apply(get_product(sh.before[w], lane), get_pair(sh.before[w].shift, lane), hw);
        if (some) {
            IO *y = (IO *)p.y + (int64_t)w0 * p.ld_y + c;
            if (full && fast && (begins | ends) == 0) {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    hw = fma2(alpha[t], hw, u[t]);
                    *reinterpret_cast<typename Pair<IO>::Raw *>(y) = Pair<IO>::narrow(hw);
                    y += p.ld_y;
                }
            } else {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    if (w0 + t < lo || w0 + t >= hi) continue;
                    hw = begins >> t & 1 ? u[t] : fma2(alpha[t], hw, u[t]);
                    store_pair<IO>(y + t * p.ld_y, hw, c, C, fast);
                    if (ends >> t & 1) store_state(p.state_out + (int64_t)(sh.edge_first[w][t + 1] - 1) * C, hw, c, C);
                }
            }
        }
        __syncwarp();       // (the next step's edges overwrite these)
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    const auto kernel = p.codes ? diag_prefill_kernel<IO, GATE, WEIGHT, true> : diag_prefill_kernel<IO, GATE, WEIGHT, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared<IO>));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    const int cl = diag_cluster(p.rows);
    cfg.gridDim = dim3(cl, diag_slices(p.channels), p.parts);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = sizeof(Shared<IO>);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

template <typename IO> cudaError_t diag_prefill_by_kind(const DiagParams &p, int gate, int weighting, cudaStream_t s) {
    if (gate == GDN_DIAG_SOFTPLUS)
        return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_NORM>(p, s)
               : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_COMPLEMENT>(p, s)
                                                  : launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_PLAIN>(p, s);
    return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_NORM>(p, s)
           : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_COMPLEMENT>(p, s)
                                              : launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_PLAIN>(p, s);
}

}  // namespace gdn
