// diag_prefill.cuh -- the diagonal recurrence h_t = alpha_t h_{t-1} + w_t i_t x_t over whole sequences.
//
// A CTA takes a tile of 64 rows and 64 channels at a time (DiagWalk).  A warp stages its 8 rows in shared memory, takes them into
// registers as (alpha, w i x), two channels to a lane, has the next item's rows fetched in their place, and folds its own to a
// map h -> P h + H; one warp folds the CTA's maps, hands the tile's on and finds the h before the tile; then each warp
// knows the h before its first row and runs its rows once more from the registers.  Every input is read once and every output
// written once; all sequences are one run of rows with edges where h starts anew, so short and long ones cost the same.
#pragma once

#include <type_traits>

#include "diag_internal.cuh"

namespace gdn {
namespace {

constexpr int LT = 8, W = kDiagTile / LT;      // a warp's rows; warps

template <typename IO> struct Shared {
    IO rows[W][3][LT][kDiagSlice];              // x, a, b
    DiagMaps maps[W], before[W];                    // a warp's rows; the tile's rows before them
    float2 start[32];                               // h before the tile
    uint32_t next;
    int edge_first[W][LT + 1], edge_last[W][LT + 1];
};

template <typename IO, int GATE, int WEIGHT, bool CODES>
__global__ void __launch_bounds__(W * 32, 3) diag_prefill_kernel(const __grid_constant__ DiagParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Shared<IO> &sh = *reinterpret_cast<Shared<IO> *>(raw_shared);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, C = p.channels, slices = (C + kDiagSlice - 1) / kDiagSlice;
    if (!offsets_ok(p)) return;
    for (int n = blockIdx.x; n < p.num_seqs; n += gridDim.x) {          // sequences without tokens keep their state
        if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
        for (int c = threadIdx.x; c < C; c += W * 32) p.state_out[(int64_t)n * C + c] = p.state_in ? p.state_in[(int64_t)n * C + c] : 0.f;
    }
    const int rows = (int)p.rows, tiles = (rows + kDiagTile - 1) / kDiagTile;
    const DiagWalk walk{p, tiles, slices, lane};
    const uint32_t items = walk.items();
    const bool has_b = p.has_b;
    IO *sx = &sh.rows[w][0][0][0], *sa = &sh.rows[w][1][0][0], *sb = &sh.rows[w][2][0][0];
    const uint32_t shut = infinity_bits<IO>(true);
    if (!has_b) fill_rows<IO, LT>(sb, infinity_bits<IO>(false), lane);
    auto stage = [&](uint32_t item) {
        const int w0 = item / slices * kDiagTile + w * LT, c0 = item % slices * kDiagSlice;
        stage_rows<IO, LT>(sx, (const IO *)p.x, p.ld_x, w0, 0, rows, c0, C, p.wide, 0u, lane);
        stage_rows<IO, LT>(sa, (const IO *)p.a, p.ld_a, w0, 0, rows, c0, C, p.wide, shut, lane);
        if (has_b) stage_rows<IO, LT>(sb, (const IO *)p.b, p.ld_b, w0, 0, rows, c0, C, p.wide, 0u, lane);
        stage_commit();
    };
    EdgeWindow window = edge_window(p, 0, lane);
    uint32_t item = walk.first(sh.next);
    if (item < items) stage(item);
    while (item < items) {
        if (threadIdx.x == 0) sh.next = walk.ticket();
        const int tile = item / slices, slice = item % slices, w0 = tile * kDiagTile + w * LT, c0 = slice * kDiagSlice, c = c0 + 2 * lane;
        const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, C);
        const bool fast = p.pairs && c0 + kDiagSlice <= C, near = diag_near<GATE>(l);
        const bool some = w0 < rows, full = w0 + LT <= rows;
        F2 alpha[LT], u[LT], sum_G = both(0.f), H = both(0.f);
        uint32_t begins = 0, ends = 0;
        if (some) {
            const uint32_t edges = find_edges<LT>(p, window, (uint32_t)w0, 0, 0, sh.edge_first[w], sh.edge_last[w], lane);
            const uint32_t live = (1u << (full ? LT : rows - w0)) - 1;
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
                    const int64_t at = ((int64_t)k * slices + slice) * all + w0;
                    uint32_t mine = 0;
#pragma unroll
                    for (int t = 0; t < LT; ++t) {
                        const F2 v = staged(from, t, lane);
                        const uint32_t e = code_step(__reduce_max_sync(~0u, magnitude(v)));
                        if (lane == t) mine = e;
                        if (full || w0 + t < rows)
                            *reinterpret_cast<uint16_t *>(p.codes + (at + t) * kDiagSlice + 2 * lane) = (uint16_t)codes_of(v, e);
                    }
                    if (lane < LT && w0 + lane < rows) p.steps[at + lane] = (uint8_t)mine;
                }
            }
        }
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
        const uint32_t next = sh.next;
        if (next < items) stage(next);
        if (w == 0) {
            DiagProduct all = get_product(sh.maps[0], lane);
            F2 shift = get_pair(sh.maps[0].shift, lane);
#pragma unroll
            for (int k = 1; k < W; ++k) {
                put_map(sh.before[k], lane, all, shift);
                const DiagProduct m = get_product(sh.maps[k], lane);
                shift = diag_apply(m, get_pair(sh.maps[k].shift, lane), shift);
                all = diag_join(all, m);
            }
            if (tile + 1 < tiles) walk.hand_on_map(tile, slice, all, shift);
            const F2 h = walk.come_in(tile, slice);
            sh.start[lane] = make_float2(h.x, h.y);
            if (p.kept && tile > 0)
                *reinterpret_cast<float2 *>(p.kept + ((int64_t)tile * slices + slice) * kDiagSlice + 2 * lane) = make_float2(h.x, h.y);
            if (tile + 1 < tiles) walk.hand_on(tile, slice, diag_apply(all, shift, h));
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
                    if (w0 + t >= rows) continue;
                    hw = begins >> t & 1 ? u[t] : fma2(alpha[t], hw, u[t]);
                    store_pair<IO>(y + t * p.ld_y, hw, c, C, fast);
                    if (ends >> t & 1) store_state(p.state_out + (int64_t)(sh.edge_first[w][t + 1] - 1) * C, hw, c, C);
                }
            }
        }
        item = next;
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    const auto kernel = p.codes ? diag_prefill_kernel<IO, GATE, WEIGHT, true> : diag_prefill_kernel<IO, GATE, WEIGHT, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared<IO>));
    if (e == cudaSuccess) e = diag_clear(p, stream);
    if (e != cudaSuccess) return e;
    kernel<<<diag_grid(p, sizeof(IO) == 4 ? 2 : 3), W * 32, sizeof(Shared<IO>), stream>>>(p);
    return cudaGetLastError();
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
