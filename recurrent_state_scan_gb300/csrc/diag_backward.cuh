// diag_backward.cuh -- gradients of the diagonal recurrence.
//
// With G_t = dy_t + alpha_{t+1} G_{t+1} the gradient at h_t (dstate_out joins at a sequence's last row), and with
// i, s the gates' sigmoids and w(g) the input's weight,
//     dx = G w i,   db = dx x (1 - i),   dg = G (alpha h_{t-1} + i x w'(g)),   w' = -alpha^2 / w | -alpha | 0,
//     da = dg g (1 - s) (sigmoid gate) | -dg e^A_log s (softplus gate),
//     dA_log = sum dg g,  da_bias = sum da,  db_bias = sum db,  dstate_in = alpha G at a sequence's first row.
// The walk is the forward pass's, from the last tile to the first: warps fold their rows to G's map, a fifth warp hands it on, and
// while that one waits they run h forward again from the kept states.  Of what the gates give, the decays' exponents G (of a sigmoid
// gate its e^-z, from which s, G and 1 - s follow; with G alone 1 - s = 1 - G / e^A_log loses the digits of a gate that is nearly open:
// 16,384 rows of 4,096 in 255 us, so in 268) and h stay in shared memory for the last pass over the rows; the rest is made again, in
// loops of four rows (all 16 in a row, their code did not fit the instruction cache: 440 us where these took 245).  The rows that come
// an iteration later are fetched into L2 meanwhile (247 us then; without 255).
//
// Bound by instructions: 86 a value (99 from codes), at 60% of the issue slots; with the gates' arithmetic taken out and no wait
// for other tiles the same loads, stores and barriers took 190 us of then 255.  8,192 bf16 rows of 4,096 channels take 128 us
// (3.7 TB/s; from codes 145), of which the bytes alone would take 69 (54).
#pragma once

#include <type_traits>

#include "diag_internal.cuh"

namespace gdn {
namespace {

constexpr int LT = kDiagRows, W = kDiagTile / LT;      // a warp's rows; the warps that take rows
constexpr int kThreads = (W + 1) * 32;
constexpr int kGroup = 4;                       // rows whose loads go out together

// A warp's rows as they are staged, and of what the gates give the decays' exponents (or what they follow from) in G and the inputs
// w i x, which become h.  The staged a lies at the end of G's place: G's rows are written when a's that lie there have been read.
// (Each array is copied to 16 bytes at a time, the steps too.)
template <typename IO, bool CODES> struct Staged {
    alignas(16) IO x[LT][kDiagSlice], b[LT][kDiagSlice], dy[LT][kDiagSlice];
    alignas(16) float2 G[LT][32], h[LT][32];
    alignas(16) float table[5][kDiagSlice], kept[kDiagSlice];       // the channels' parameters, h before the rows
    __device__ __forceinline__ IO *a() { return reinterpret_cast<IO *>(G + LT) - LT * kDiagSlice; }
};
template <typename IO> struct Staged<IO, true> {
    alignas(16) int8_t x[LT][kDiagSlice], b[LT][kDiagSlice], codes_a[LT][kDiagSlice];
    alignas(16) IO dy[LT][kDiagSlice];
    alignas(16) uint8_t xs[LT], bs[LT], as[LT];
    alignas(16) float step_x[LT], gate_a[LT], gate_b[LT];       // steps; those of the sigmoids' arguments times -log2 e
    alignas(16) float2 G[LT][32], h[LT][32];
    alignas(16) float table[5][kDiagSlice], kept[kDiagSlice];
};
static_assert(LT * kDiagSlice % 16 == 0 && LT == 16, "what follows an array is aligned as it is");
template <typename IO, bool CODES> struct Shared {
    Staged<IO, CODES> rows[W];
    DiagMaps maps[W];                   // a warp's rows, G's
    float2 shift[CODES ? W : 1][32];    // with codes: h's, whose product is the same
    DiagMaps behind[W - 1];             // G's: the tile's rows behind a warp's
    float2 start[32];                   // what comes back to the tile
    float2 sums[2][W][3][32];           // the parameters' gradients, of two items in turn
    uint32_t next;
    int edge_first[W][LT + 1], edge_last[W][LT + 1];
};

// Rows [r0, r0 + LT) of codes; those outside [lo, hi) as `outside`, with a step of 0 (-1.1e37: a code of 1 shuts a gate).
__device__ __forceinline__ void stage_codes(int8_t *to, uint8_t *to_steps, const DiagParams &p, int k, int slice, int slices, int r0,
                                            int lo, int hi, uint32_t outside, int lane) {
    const int64_t all = (p.rows + kDiagTile - 1) / kDiagTile * kDiagTile, at = ((int64_t)k * slices + slice) * all + r0;
    const int8_t *from = p.codes + at * kDiagSlice;
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to)), ds = static_cast<uint32_t>(__cvta_generic_to_shared(to_steps));
    const bool full = r0 >= lo && r0 + LT <= hi;
#pragma unroll
    for (int i = 0; i < LT / 8; ++i) {
        const int piece = i * 32 + lane;
        const int row = r0 + piece / 4;
        if (full || (row >= lo && row < hi))
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst + piece * 16), "l"(from + piece * 16) : "memory");
        else
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + piece * 16), "r"(outside) : "memory");
    }
    if (full) {
        if (lane == 0) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ds), "l"(p.steps + at), "n"(LT) : "memory");
    } else if (lane < LT) {
        to_steps[lane] = r0 + lane >= lo && r0 + lane < hi ? p.steps[at + lane] : (uint8_t)0;
    }
}
// The pair of row t, in units of its step.
__device__ __forceinline__ F2 code_pair(const int8_t *rows, int t, int lane) { return code_values(reinterpret_cast<const uint16_t *>(rows)[t * 32 + lane]); }
// A gate's argument: with codes in units of their step, `by` being that times what the gate multiplies it by.
struct Argument {
    F2 v;
    float by;
};
// Codes of gates that are held shut, as what they stand for.
template <int N> __device__ __forceinline__ void shut_gates(Argument (&to)[N]) {
    const float minus = __uint_as_float(0xff800000u);
#pragma unroll
    for (int k = 0; k < N; ++k) to[k].v = {to[k].v.x == kShutCode ? minus : to[k].v.x, to[k].v.y == kShutCode ? minus : to[k].v.y};
}
// What belongs to N rows, alike for all lanes.
template <int N> struct PerRow {
    float v[N];
    __device__ __forceinline__ PerRow(const float *from) {
        if constexpr (N == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(from);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = from[k];
        }
    }
};

template <typename IO, int GATE, int WEIGHT, bool CODES>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 4 ? 2 : 3) diag_backward_kernel(const __grid_constant__ DiagParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Shared<IO, CODES> &sh = *reinterpret_cast<Shared<IO, CODES> *>(raw_shared);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, C = p.channels, slices = (C + kDiagSlice - 1) / kDiagSlice;
    if (!offsets_ok(p)) return DiagWalk::wait_for_first();
    if (p.dstate_in)
        for (int n = blockIdx.x; n < p.num_seqs; n += gridDim.x) {      // sequences without tokens
            if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
            for (int c = threadIdx.x; c < C; c += kThreads) p.dstate_in[(int64_t)n * C + c] = p.dstate_out ? p.dstate_out[(int64_t)n * C + c] : 0.f;
        }
    const int rows = (int)p.rows, tiles = (rows + kDiagTile - 1) / kDiagTile;
    const DiagWalk walk{p, tiles, slices, lane};
    const uint32_t items = walk.items();
    uint32_t item = walk.first(sh.next);
    if (w == W) {
        // The parameters' gradients of an item, over the rows' warps in their order.
        auto put_sums = [&](uint32_t of, const float2 (*sums)[3][32]) {
            const int j = walk.tile_of(of), c = ((int)of - j * slices) * kDiagSlice + 2 * lane;
            float *one[3] = {p.dA_log, p.da_bias, p.db_bias};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                F2 total = get_pair(sums[0][k], lane);
#pragma unroll
                for (int r = 1; r < W; ++r) total = add2(total, get_pair(sums[r][k], lane));
                if (tiles > 1) store_state(p.partial + ((int64_t)j * 3 + k) * C, total, c, C);
                else if (one[k]) store_state(one[k], total, c, C);
            }
        };
        uint32_t last = items;
        int turn = 0;
        for (; item < items; turn ^= 1) {
            const int j = walk.tile_of(item), slice = (int)item - j * slices;
            const uint32_t later = lane == 0 ? walk.ticket() : 0u;
            side_sync<kThreads>(1);
            DiagProduct all = get_product(sh.maps[W - 1], lane);
            F2 shift = get_pair(sh.maps[W - 1].shift, lane);
#pragma unroll
            for (int r = W - 2; r >= 0; --r) {
                put_map(sh.behind[r], lane, all, shift);
                const DiagProduct m = get_product(sh.maps[r], lane);
                shift = diag_apply(m, get_pair(sh.maps[r].shift, lane), shift);
                all = diag_join(all, m);
            }
            if (j + 1 < tiles) walk.hand_on_map(j, slice, all, shift);
            const F2 in = walk.come_in(j, slice);
            if (j + 1 < tiles) walk.hand_on(j, slice, diag_apply(all, shift, in));
            sh.start[lane] = make_float2(in.x, in.y);
            if (lane == 0) sh.next = later;
            __syncwarp();
            side_arrive<kThreads>(2);
            if (last < items) put_sums(last, sh.sums[turn ^ 1]);        // (out of the way of what is handed on)
            last = item;
            item = __shfl_sync(~0u, later, 0);
        }
        side_sync<kThreads>(1);
        if (last < items) put_sums(last, sh.sums[turn ^ 1]);
        return;
    }
    const bool has_b = p.has_b;
    Staged<IO, CODES> &st = sh.rows[w];
    float2 *sG = &st.G[0][0], *sh_ = &st.h[0][0];
    const uint32_t shut = infinity_bits<IO>(true);
    if (!has_b) {                   // codes of 1 with the largest step are as good as infinity
        if constexpr (CODES) {
            fill_rows<int8_t, LT>(&st.b[0][0], 0x01010101u, lane);
            if (lane < LT) st.bs[lane] = 254;
        } else {
            fill_rows<IO, LT>(&st.b[0][0], infinity_bits<IO>(false), lane);
        }
    }
    const Stager<IO, LT> from_x(p.x, p.ld_x, lane), from_a(p.a, p.ld_a, lane), from_b(p.b, p.ld_b, lane), from_dy(p.dy, p.ld_y, lane);
    auto stage = [&](uint32_t item) {
        const int j = walk.tile_of(item), slice = (int)item - j * slices, w0 = (tiles - 1 - j) * kDiagTile + w * LT, c0 = slice * kDiagSlice;
        if constexpr (CODES) {
            stage_codes(&st.x[0][0], st.xs, p, 0, slice, slices, w0, 0, rows, 0u, lane);
            stage_codes(&st.codes_a[0][0], st.as, p, 1, slice, slices, w0, 0, rows, 0x01010101u, lane);
            if (has_b) stage_codes(&st.b[0][0], st.bs, p, 2, slice, slices, w0, 0, rows, 0u, lane);
        } else {
            from_x.rows(&st.x[0][0], w0, rows, c0, C, p.wide, 0u, lane);
            from_a.rows(st.a(), w0, rows, c0, C, p.wide, shut, lane);
            if (has_b) from_b.rows(&st.b[0][0], w0, rows, c0, C, p.wide, 0u, lane);
        }
        from_dy.rows(&st.dy[0][0], w0, rows, c0, C, p.wide, 0u, lane);
        // Without codes h is there before each warp's rows; else before the tile's.
        const int held = CODES ? tiles - 1 - j : w0 / LT;
        if (lane < 16) {
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&st.table[0][4 * lane]));
            const float *from = p.table + c0 + 4 * lane;
            if (p.table) {
#pragma unroll
                for (int k = 0; k < 5; ++k, from += slices * kDiagSlice)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * kDiagSlice * 4), "l"(from) : "memory");
            }
        } else if (held > 0 && w0 < rows) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&st.kept[4 * (lane - 16)]))),
                         "l"(p.kept + (int64_t)held * slices * kDiagSlice + c0 + 4 * (lane - 16))
                         : "memory");
        }
        stage_commit();
        item += gridDim.x;
        if (item < items) {
            const int j = walk.tile_of(item), r0 = (tiles - 1 - j) * kDiagTile + w * LT, f0 = ((int)item - j * slices) * kDiagSlice;
            if constexpr (!CODES) {
                fetch_rows<IO>(p.x, p.ld_x, p.a, p.ld_a, r0, rows, f0, C, lane);
                fetch_rows<IO>(p.dy, p.ld_y, has_b ? p.b : nullptr, p.ld_b, r0, rows, f0, C, lane);
            } else {
                fetch_rows<IO>(p.dy, p.ld_y, nullptr, 0, r0, rows, f0, C, lane);
                const int64_t all = (int64_t)tiles * kDiagTile, k = lane / 8;
                if (k < 2 + has_b) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.codes + ((k * slices + f0 / kDiagSlice) * all + r0) * kDiagSlice + lane % 8 * 128));
            }
        }
    };
    // Rows' pairs: x, and the gates' arguments beside what the gate multiplies them by.
    auto get_x = [&](auto &to, int t0) {
        constexpr int N = sizeof(to) / sizeof(F2);
        if constexpr (CODES) {
            const PerRow<N> step(&st.step_x[t0]);
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = mul2(code_pair(&st.x[0][0], t0 + k, lane), both(step.v[k]));
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = staged(&st.x[0][0], t0 + k, lane);
        }
    };
    auto get_a = [&](auto &to, int t0, bool masked) {
        constexpr int N = sizeof(to) / sizeof(Argument);
        if constexpr (CODES) {
            const PerRow<N> by(&st.gate_a[t0]);
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = {code_pair(&st.codes_a[0][0], t0 + k, lane), by.v[k]};
            if (masked) shut_gates(to);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = {staged(st.a(), t0 + k, lane), kGateUnit<GATE>};
        }
    };
    auto get_b = [&](auto &to, int t0, bool masked) {
        constexpr int N = sizeof(to) / sizeof(Argument);
        if constexpr (CODES) {
            const PerRow<N> by(&st.gate_b[t0]);
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = {code_pair(&st.b[0][0], t0 + k, lane), by.v[k]};
            if (masked) shut_gates(to);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) to[k] = {staged(&st.b[0][0], t0 + k, lane), -kLog2e};
        }
    };
    EdgeWindow window = edge_window(p, 0, lane);
    if (item < items) stage(item);
    for (int turn = 0; item < items; turn ^= 1) {
        const int j = walk.tile_of(item), tile = tiles - 1 - j, slice = (int)item - j * slices, w0 = tile * kDiagTile + w * LT, c0 = slice * kDiagSlice;
        const int c = c0 + 2 * lane;
        const bool fast = p.pairs && c0 + kDiagSlice <= C;
        F2 sum_A = both(0.f), sum_a = both(0.f), sum_b = both(0.f);
        const bool some = w0 < rows, full = w0 + LT <= rows;
        F2 sum_G = both(0.f), D = both(0.f);
        uint32_t begins = 0, ends = 0;
        if (some) {
            const uint32_t edges = find_edges<LT>(p, window, (uint32_t)w0, 0, 28, sh.edge_first[w], sh.edge_last[w], lane);
            const uint32_t live = (1u << (full ? LT : rows - w0)) - 1;
            begins = edges & live;
            ends = edges >> 1 & live;
        }
        const uint32_t special = begins | ends;
        stage_wait();
        const DiagLane l = p.table ? diag_lane(&st.table[0][0], kDiagSlice, lane) : diag_lane(p, c, slices);
        const bool near = diag_near<GATE>(l);
        F2 at = some && (CODES ? tile : w0) > 0 ? get_pair(reinterpret_cast<const float2 *>(st.kept), lane) : both(0.f);
        bool masked = false;            // whether codes of a or b are -128
        if constexpr (CODES) {
            masked = any_shut(&st.codes_a[0][0], &st.b[0][0], lane);
            if (lane < LT) {
                st.step_x[lane] = code_scale(st.xs[lane]);
                st.gate_a[lane] = kGateUnit<GATE> * code_scale(st.as[lane]);
                st.gate_b[lane] = -kLog2e * code_scale(st.bs[lane]);
            }
            __syncwarp();
        }
        // Of what stays in G's place, the exponent.
        auto exponent = [&](F2 held) { return GATE == GDN_DIAG_SIGMOID ? mul2(l.rate, diag_opening(held)) : held; };
        // What G's map needs, for the fifth warp to hand on; with codes h's map as well, from which the other warps find their h.
        F2 through = both(1.f), H = both(0.f);
        auto minus_input = [&](Argument b, F2 x, F2 n) {
            const F2 v = mul2(diag_minus_sigmoid(b.v, l.nbbias, b.by), x);
            return WEIGHT == GDN_DIAG_PLAIN ? v : mul2(diag_weigh<WEIGHT>(n), v);
        };
        auto take = [&](auto only_near, auto masks) {
            constexpr bool kNear = decltype(only_near)::value;
#pragma unroll 1
            for (int t0 = 0; t0 < LT; t0 += kGroup) {       // (the loads of a group go out before its stores)
                Argument a[kGroup], b[kGroup];
                F2 x[kGroup], dy[kGroup], held[kGroup];
                get_a(a, t0, decltype(masks)::value);
                if (CODES) {
                    get_b(b, t0, decltype(masks)::value);
                    get_x(x, t0);
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) dy[k] = staged(&st.dy[0][0], t0 + k, lane);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    if (GATE == GDN_DIAG_SIGMOID) {
                        held[k] = diag_closing(a[k].v, l.nabias, a[k].by);
                    } else {            // finite, for a decay to 0 times it; a NaN stays one
                        held[k] = diag_exponent<GATE>(a[k].v, l, a[k].by);
                        asm("min.NaN.f32 %0, %0, 0f7149F2CA;" : "+f"(held[k].x));
                        asm("min.NaN.f32 %0, %0, 0f7149F2CA;" : "+f"(held[k].y));
                    }
                    const F2 G = exponent(held[k]);
                    sum_G = add2(sum_G, G);
                    const DiagDecay d = diag_decay<kNear>(G);
                    through = mul2(through, d.alpha);
                    D = fma2(through, dy[k], D);
                    if (CODES) {
                        x[k] = minus_input(b[k], x[k], d.n);
                        H = fma2(d.alpha, H, x[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    sG[(t0 + k) * 32 + lane] = make_float2(held[k].x, held[k].y);
                    if (CODES) sh_[(t0 + k) * 32 + lane] = make_float2(x[k].x, x[k].y);
                }
            }
        };
        if (CODES && masked) take(std::false_type{}, std::true_type{});
        else if (near) take(std::true_type{}, std::false_type{});
        else take(std::false_type{}, std::false_type{});
        if (!full) {            // rows outside are the identity, whatever the parameters make of them (an infinite bias: NaN)
            const float none = GATE == GDN_DIAG_SIGMOID ? __uint_as_float(0x7f800000u) : 0.f;
            sum_G = D = both(0.f);
#pragma unroll 1
            for (int t = 0; t < LT; ++t) {
                if (w0 + t < rows) sum_G = add2(sum_G, exponent(get_pair(sG + t * 32, lane)));
                else sG[t * 32 + lane] = make_float2(none, none);
            }
        }
        if (special) {          // nothing behind a sequence's first row comes back to here
            through = both(1.f);
            D = both(0.f);
#pragma unroll 1
            for (int t = 0; t < LT && !(begins >> t & 1); ++t) {
                F2 dy = staged(&st.dy[0][0], t, lane);
                if ((ends >> t & 1) && p.dstate_out)
                    dy = add2(dy, load_state(p.dstate_out + (int64_t)(sh.edge_first[w][t + 1] - 1) * C, c, C));
                through = mul2(through, diag_decay<false>(exponent(get_pair(sG + t * 32, lane))).alpha);
                D = fma2(through, dy, D);
            }
        }
        // -h before each row, or from 0 the map's; with codes the inputs are in h's place.
        auto follow_edges = [&](F2 nat, bool map) {
#pragma unroll 1
            for (int t = 0; t < LT; ++t) {
                const DiagDecay d = diag_decay<false>(exponent(get_pair(sG + t * 32, lane)));
                if (begins >> t & 1) {
                    nat = p.state_in ? load_state(p.state_in + (int64_t)sh.edge_last[w][t] * C, c, C) : both(0.f);
                    nat = mul2(nat, both(-1.f));
                }
                F2 in;
                if (CODES) {
                    in = get_pair(sh_ + t * 32, lane);
                } else {
                    Argument b[1];
                    F2 x[1];
                    get_b(b, t, false);
                    get_x(x, t);
                    in = minus_input(b[0], x[0], d.n);
                }
                if (!map) sh_[t * 32 + lane] = make_float2(nat.x, nat.y);
                nat = fma2(d.alpha, nat, in);
            }
            return nat;
        };
        if (CODES && begins) H = follow_edges(both(0.f), true);
        put_map(sh.maps[w], lane, diag_product(sum_G, begins != 0), D);
        if (CODES) sh.shift[w][lane] = make_float2(-H.x, -H.y);
        __syncwarp();
        side_arrive<kThreads>(1);
        // -h before each row, while the fifth warp hands on and waits.
        auto follow = [&](auto only_near) {
            F2 nat = mul2(at, both(-1.f));
#pragma unroll 1
            for (int t0 = 0; t0 < LT; t0 += kGroup) {
                Argument b[kGroup];
                F2 G[kGroup], x[kGroup], out[kGroup];
                if (!CODES) {
                    get_b(b, t0, false);
                    get_x(x, t0);
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    G[k] = exponent(get_pair(sG + (t0 + k) * 32, lane));
                    if (CODES) x[k] = get_pair(sh_ + (t0 + k) * 32, lane);
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const DiagDecay d = diag_decay<decltype(only_near)::value>(G[k]);
                    out[k] = nat;
                    nat = fma2(d.alpha, nat, CODES ? x[k] : minus_input(b[k], x[k], d.n));
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) sh_[(t0 + k) * 32 + lane] = make_float2(out[k].x, out[k].y);
            }
        };
        if constexpr (CODES) {
            side_sync<W * 32>(3);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                if (k < w) at = diag_apply(get_product(sh.maps[k], lane), get_pair(sh.shift[k], lane), at);
        }
        if (begins) follow_edges(mul2(at, both(-1.f)), false);
        else if (near) follow(std::true_type{});
        else follow(std::false_type{});
        side_sync<kThreads>(2);
        const uint32_t next = sh.next;
        F2 back = get_pair(sh.start, lane);     // what comes back from the rows behind the warp's
        if (w < W - 1) back = diag_apply(get_product(sh.behind[w], lane), get_pair(sh.behind[w].shift, lane), back);
        if (some) {
            IO *dx = (IO *)p.dx + (int64_t)(w0 + LT - 1) * p.ld_dx + c, *da = (IO *)p.da + (int64_t)(w0 + LT - 1) * p.ld_da + c;
            IO *db = (IO *)p.db + (int64_t)(w0 + LT - 1) * p.ld_db + c;
            // PLAIN: all rows are there, stored by pairs, no sequence begins or ends, and no code holds a gate shut.
            auto give = [&](auto only_near, auto plain) {
                constexpr bool kPlain = decltype(plain)::value;
                constexpr int N = kPlain ? kGroup : 1;
#pragma unroll 1
                for (int t0 = LT - N; t0 >= 0; t0 -= N) {
                    Argument b[N];
                    F2 x[N], dy[N], held[N], h[N];
                    get_b(b, t0, !kPlain && masked);
                    get_x(x, t0);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        dy[k] = staged(&st.dy[0][0], t0 + k, lane);
                        held[k] = get_pair(sG + (t0 + k) * 32, lane);
                        h[k] = get_pair(sh_ + (t0 + k) * 32, lane);
                    }
                    F2 out_x[N], out_a[N], out_b[N];
#pragma unroll
                    for (int k = N - 1; k >= 0; --k) {
                        const int t = t0 + k;
                        F2 g = add2(dy[k], back);           // the gradient at h_t
                        if (!kPlain && (ends >> t & 1) && p.dstate_out)
                            g = add2(g, load_state(p.dstate_out + (int64_t)(sh.edge_first[w][t + 1] - 1) * C, c, C));
                        const F2 close_b = diag_closing(b[k].v, l.nbbias, b[k].by), i = diag_opening(close_b), v = mul2(i, x[k]);
                        const F2 s = diag_opening(held[k]), G = GATE == GDN_DIAG_SIGMOID ? mul2(l.rate, s) : held[k];
                        const DiagDecay d = diag_decay<decltype(only_near)::value>(G);
                        F2 slope = h[k], weight = d.n;                              // dG / (g alpha), G = -g (h: negative)
                        if (WEIGHT == GDN_DIAG_NORM) {
                            const F2 unweight = diag_unweigh(d.n);
                            slope = fma2(mul2(v, d.alpha), unweight, slope);
                            weight = mul2(mul2(d.n, fma2(d.n, both(-1.f), both(2.f))), unweight);
                        }
                        if (WEIGHT == GDN_DIAG_COMPLEMENT) slope = add2(v, slope);
                        const F2 ag = mul2(d.alpha, g), dv = WEIGHT == GDN_DIAG_PLAIN ? g : mul2(g, weight);
                        // (The products with G come first: a shut gate's is 0, whatever x is.)
                        const F2 dGG = mul2(mul2(ag, G), slope);
                        const F2 nsp = mul2(G, l.ninverse);                         // a softplus gate's opening, negative
                        const F2 da_ = GATE == GDN_DIAG_SIGMOID ? mul2(dGG, diag_closed(held[k], s))
                                                                : mul2(mul2(ag, mul2(l.rate, diag_decay<false>(F2{-nsp.x, -nsp.y}).n)), slope);
                        out_x[k] = mul2(dv, i);
                        const F2 db_ = mul2(out_x[k], mul2(diag_closed(close_b, i), x[k]));     // dx x (1 - i)
                        out_a[k] = da_;
                        out_b[k] = db_;
                        if (kPlain || w0 + t < rows) {
                            sum_A = add2(sum_A, dGG);
                            sum_a = add2(sum_a, da_);
                            sum_b = add2(sum_b, db_);
                        }
                        back = ag;
                        if (!kPlain && (begins >> t & 1)) {
                            if (p.dstate_in) store_state(p.dstate_in + (int64_t)sh.edge_last[w][t] * C, back, c, C);
                            back = both(0.f);
                        }
                    }
#pragma unroll
                    for (int k = N - 1; k >= 0; --k, dx -= p.ld_dx, da -= p.ld_da, db -= p.ld_db) {
                        if (!kPlain && w0 + t0 + k >= rows) continue;
                        store_pair<IO>(dx, out_x[k], c, C, kPlain || fast);
                        store_pair<IO>(da, out_a[k], c, C, kPlain || fast);
                        if (has_b) store_pair<IO>(db, out_b[k], c, C, kPlain || fast);
                    }
                }
            };
            if (!full || !fast || special || masked) give(std::false_type{}, std::false_type{});
            else if (near) give(std::true_type{}, std::true_type{});
            else give(std::false_type{}, std::true_type{});
        }
        const F2 all_sums[3] = {sum_A, sum_a, sum_b};
#pragma unroll
        for (int k = 0; k < 3; ++k) sh.sums[turn][w][k][lane] = make_float2(all_sums[k].x, all_sums[k].y);
        __syncwarp();
        if (next < items) stage(next);
        item = next;
    }
    side_arrive<kThreads>(1);
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    const auto kernel = p.codes ? diag_backward_kernel<IO, GATE, WEIGHT, true> : diag_backward_kernel<IO, GATE, WEIGHT, false>;
    const size_t shared = p.codes ? sizeof(Shared<IO, true>) : sizeof(Shared<IO, false>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e == cudaSuccess) e = diag_begin(p, stream);
    if (e != cudaSuccess) return e;
    return diag_launch(kernel, diag_grid(p, sizeof(IO) == 4 ? 2 : 3), kThreads, shared, p, stream);
}

}  // namespace

template <typename IO> cudaError_t diag_backward_by_kind(const DiagParams &p, int gate, int weighting, cudaStream_t s) {
    if (gate == GDN_DIAG_SOFTPLUS)
        return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_NORM>(p, s)
               : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_COMPLEMENT>(p, s)
                                                  : launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_PLAIN>(p, s);
    return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_NORM>(p, s)
           : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_COMPLEMENT>(p, s)
                                              : launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_PLAIN>(p, s);
}

}  // namespace gdn
