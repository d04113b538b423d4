// diag_prefill.cuh -- the diagonal recurrence h_t = alpha_t h_{t-1} + w_t i_t x_t over whole sequences.
//
// A CTA takes tiles of 64 rows and 64 channels (DiagWalk), four warps of 16 rows each, two channels to a lane.  A warp stages its
// rows in shared memory, takes them into registers as (alpha, w i x), has the next tile's rows fetched in their place, and
// folds its own to a map h -> P h + H.  A fifth warp folds the four maps, hands the tile's on and finds the h before the tile,
// while the four are already at the next tile; only then do they run the rows of the earlier one once more, from shared
// memory, and store h.  Every input is read once and every output written once; all sequences are one run of rows with
// edges where h starts anew, so short and long ones cost the same.
//
// Bound by instructions: 36 a value (58 with codes), at half the issue slots of the 12 row warps that registers and shared memory
// leave an SM.  8,192 bf16 rows of 4,096 channels take 65 us (4.1 TB/s; with codes 93), of which the bytes alone would take 40
// (54).  Clusters of CTAs that walk down a slice in step took 82.
#pragma once

#include <type_traits>

#include "diag_internal.cuh"

namespace gdn {
namespace {

constexpr int LT = kDiagRows, W = kDiagTile / LT;      // a warp's rows; the warps that take rows
constexpr int kThreads = (W + 1) * 32;

template <typename IO> struct Shared {
    alignas(16) IO rows[W][3][LT][kDiagSlice];      // x, a, b
    float4 held[W][LT][32];                         // alpha, w i x of the tile before
    DiagMaps maps[2][W], before[2][W];              // a warp's rows; the tile's rows before them
    float2 start[2][32];                            // h before the tile
    uint32_t items[2];                              // the item after the next one, of two in turn
    int edge_first[2][W][LT + 1], edge_last[2][W][LT + 1];
};

template <typename IO, int GATE, int WEIGHT, bool CODES>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 4 ? 2 : 3) diag_prefill_kernel(const __grid_constant__ DiagParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Shared<IO> &sh = *reinterpret_cast<Shared<IO> *>(raw_shared);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, C = p.channels, slices = (C + kDiagSlice - 1) / kDiagSlice;
    if (!offsets_ok(p)) return DiagWalk::wait_for_first();
    for (int n = blockIdx.x; n < p.num_seqs; n += gridDim.x) {          // sequences without tokens keep their state
        if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
        for (int c = threadIdx.x; c < C; c += kThreads) p.state_out[(int64_t)n * C + c] = p.state_in ? p.state_in[(int64_t)n * C + c] : 0.f;
    }
    const int rows = (int)p.rows, tiles = (rows + kDiagTile - 1) / kDiagTile;
    const DiagWalk walk{p, tiles, slices, lane};
    const uint32_t items = walk.items();
    uint32_t item = walk.first(sh.items[0]);
    const uint32_t second = tiles > 1 ? walk.first(sh.items[1]) : items;
    if (w == W) {
        uint32_t next = second;
        for (int k = 0; item < items; ++k) {
            const int buf = k & 1, tile = walk.tile_of(item), slice = (int)item - tile * slices;
            side_sync<kThreads>(1 + buf);      // (two barriers of each kind in turn: the one side cannot be two steps ahead)
            // The item behind the next one, as late as can be: one that its CTA has not begun holds up all that come after it.
            const uint32_t later = lane == 0 && next < items ? walk.ticket() : items;
            DiagProduct all = get_product(sh.maps[buf][0], lane);
            F2 shift = get_pair(sh.maps[buf][0].shift, lane);
#pragma unroll
            for (int r = 1; r < W; ++r) {
                put_map(sh.before[buf][r], lane, all, shift);
                const DiagProduct m = get_product(sh.maps[buf][r], lane);
                shift = diag_apply(m, get_pair(sh.maps[buf][r].shift, lane), shift);
                all = diag_join(all, m);
            }
            if (tile + 1 < tiles) walk.hand_on_map(tile, slice, all, shift);
            const F2 h = walk.come_in(tile, slice);
            if (tile + 1 < tiles) walk.hand_on(tile, slice, diag_apply(all, shift, h));
            sh.start[buf][lane] = make_float2(h.x, h.y);
            if (lane == 0) sh.items[buf] = later;
            __syncwarp();
            side_arrive<kThreads>(3 + buf);
            item = next;
            next = __shfl_sync(~0u, later, 0);
        }
        return;
    }
    const bool has_b = p.has_b;
    IO *sx = &sh.rows[w][0][0][0], *sa = &sh.rows[w][1][0][0], *sb = &sh.rows[w][2][0][0];
    float4 *held = &sh.held[w][0][lane];
    const uint32_t shut = infinity_bits<IO>(true);
    if (!has_b) fill_rows<IO, LT>(sb, infinity_bits<IO>(false), lane);
    const Stager<IO, LT> from_x(p.x, p.ld_x, lane), from_a(p.a, p.ld_a, lane), from_b(p.b, p.ld_b, lane);
    auto stage = [&](uint32_t item) {
        const int tile = walk.tile_of(item), w0 = tile * kDiagTile + w * LT, c0 = ((int)item - tile * slices) * kDiagSlice;
        from_x.rows(sx, w0, rows, c0, C, p.wide, 0u, lane);
        from_a.rows(sa, w0, rows, c0, C, p.wide, shut, lane);
        if (has_b) from_b.rows(sb, w0, rows, c0, C, p.wide, 0u, lane);
        stage_commit();
    };
    EdgeWindow window = edge_window(p, 0, lane);
    uint32_t begins = 0, ends = 0;
    int old_w0 = 0, old_c = 0;
    uint32_t old_begins = 0, old_ends = 0;
    DiagLane l{};
    auto parameters = [&](uint32_t of) { l = diag_lane(p, ((int)of - walk.tile_of(of) * slices) * kDiagSlice + 2 * lane, slices); };
    if (item < items) {
        stage(item);
        parameters(item);
    }
    for (int k = 0;; ++k) {
        const bool more = item < items;
        const int buf = k & 1, tile = walk.tile_of(item), slice = (int)item - tile * slices, w0 = tile * kDiagTile + w * LT;
        const int c0 = slice * kDiagSlice, c = c0 + 2 * lane;
        F2 alpha[LT], u[LT];
        if (more) {
            const bool near = diag_near<GATE>(l), full = w0 + LT <= rows;
            F2 sum_G = both(0.f), H = both(0.f);
            begins = ends = 0;
            if (w0 < rows) {
                const uint32_t edges = find_edges<LT>(p, window, (uint32_t)w0, 0, 0, sh.edge_first[buf][w], sh.edge_last[buf][w], lane);
                const uint32_t live = (1u << (full ? LT : rows - w0)) - 1;
                begins = edges & live;
                ends = edges >> 1 & live;
            }
            stage_wait();
            if (CODES && w0 < rows) {
                const int64_t all = (p.rows + kDiagTile - 1) / kDiagTile * kDiagTile;
#pragma unroll 1
                for (int q = 0; q < (has_b ? 3 : 2); ++q) {
                    const IO *from = sx + q * LT * kDiagSlice;
                    const int64_t at = ((int64_t)q * slices + slice) * all + w0;
                    bool infinite = false;
                    if constexpr (sizeof(IO) == 2) {
                        infinite = code_rows<IO>(from, p.codes + at * kDiagSlice, p.steps + at, rows - w0, lane);
                    } else {
#pragma unroll 4
                        for (int t = 0; t < LT; ++t) {
                            const F2 v = staged(from, t, lane);
                            const uint32_t most = __reduce_max_sync(~0u, magnitude(v)), e = code_step(most);
                            if (w0 + t >= rows) break;
                            infinite |= most == 0x7f800000u;
                            *reinterpret_cast<uint16_t *>(p.codes + (at + t) * kDiagSlice + 2 * lane) = (uint16_t)codes_of(v, e);
                            if (lane == 0) p.steps[at + t] = (uint8_t)e;
                        }
                    }
                    if (infinite && q > 0) code_gate_rows<IO>(from, p.codes + at * kDiagSlice, p.steps + at, rows - w0, lane);
                }
            }
            auto take = [&](auto only_near) {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    const F2 G = diag_exponent<GATE>(staged(sa, t, lane), l), i = diag_sigmoid(staged(sb, t, lane), l.nbbias);
                    const DiagDecay d = diag_decay<decltype(only_near)::value>(G);
                    const F2 v = mul2(i, staged(sx, t, lane));
                    alpha[t] = d.alpha;
                    u[t] = WEIGHT == GDN_DIAG_PLAIN ? v : mul2(diag_weigh<WEIGHT>(d.n), v);
                    sum_G = add2(sum_G, G);
                    H = fma2(d.alpha, H, u[t]);
                }
            };
            if (near) take(std::true_type{});
            else take(std::false_type{});
            if (begins) {
                H = both(0.f);
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    if (begins >> t & 1) {          // a sequence's first row
                        if (p.state_in) u[t] = fma2(alpha[t], load_state(p.state_in + (int64_t)sh.edge_last[buf][w][t] * C, c, C), u[t]);
                        H = u[t];
                    } else {
                        H = fma2(alpha[t], H, u[t]);
                    }
                }
            }
            DiagProduct product = diag_product(sum_G, begins != 0);
            if (product.hi.x == 0.f || product.hi.y == 0.f) {
                F2 least = both(1.f);
#pragma unroll
                for (int t = 0; t < LT; ++t) least = {fminf(least.x, alpha[t].x), fminf(least.y, alpha[t].y)};
                if (product.hi.x == 0.f && least.x > 0.f) product.hi.x = kLeast;
                if (product.hi.y == 0.f && least.y > 0.f) product.hi.y = kLeast;
            }
            put_map(sh.maps[buf][w], lane, product, H);
            __syncwarp();
            side_arrive<kThreads>(1 + buf);
        }
        if (k > 0) side_sync<kThreads>(3 + (buf ^ 1));
        const uint32_t next = !more ? items : k == 0 ? second : sh.items[buf ^ 1];
        if (next < items) {
            stage(next);
            parameters(next);
        }
        if (k > 0) {
            F2 h = get_pair(sh.start[buf ^ 1], lane);
            if (w > 0) h = diag_apply(get_product(sh.before[buf ^ 1][w], lane), get_pair(sh.before[buf ^ 1][w].shift, lane), h);
            if (p.kept && old_w0 < rows && (!CODES || w == 0)) {
                const int64_t row = CODES ? old_w0 / kDiagTile : old_w0 / LT;
                *reinterpret_cast<float2 *>(p.kept + row * slices * kDiagSlice + old_c) = make_float2(h.x, h.y);
            }
            const bool fast = p.pairs && (old_c | (kDiagSlice - 1)) < C;
            IO *y = (IO *)p.y + (int64_t)old_w0 * p.ld_y + old_c;
            if (old_w0 + LT <= rows && fast && (old_begins | old_ends) == 0) {
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    const float4 v = held[t * 32];
                    h = fma2({v.x, v.y}, h, {v.z, v.w});
                    *reinterpret_cast<typename Pair<IO>::Raw *>(y) = Pair<IO>::narrow(h);
                    y += p.ld_y;
                }
            } else {
#pragma unroll 1
                for (int t = 0; t < LT && old_w0 + t < rows; ++t) {
                    const float4 v = held[t * 32];
                    h = old_begins >> t & 1 ? F2{v.z, v.w} : fma2({v.x, v.y}, h, {v.z, v.w});
                    store_pair<IO>(y + t * p.ld_y, h, old_c, C, fast);
                    if (old_ends >> t & 1) store_state(p.state_out + (int64_t)(sh.edge_first[buf ^ 1][w][t + 1] - 1) * C, h, old_c, C);
                }
            }
        }
        if (!more) return;
#pragma unroll
        for (int t = 0; t < LT; ++t) held[t * 32] = make_float4(alpha[t].x, alpha[t].y, u[t].x, u[t].y);
        old_w0 = w0;
        old_c = c;
        old_begins = begins;
        old_ends = ends;
        item = next;
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    const auto kernel = p.codes ? diag_prefill_kernel<IO, GATE, WEIGHT, true> : diag_prefill_kernel<IO, GATE, WEIGHT, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared<IO>));
    if (e == cudaSuccess) e = diag_begin(p, stream);
    if (e != cudaSuccess) return e;
    return diag_launch(kernel, diag_grid(p, sizeof(IO) == 4 ? 2 : 3), kThreads, sizeof(Shared<IO>), p, stream);
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
