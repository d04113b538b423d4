// diag_backward.cuh -- gradients of the diagonal recurrence.
//
// With G_t = dy_t + alpha_{t+1} G_{t+1} the gradient at h_t (dstate_out joins at a sequence's last row), and with
// i, s the gates' sigmoids and w(g) the input's weight,
//     dx = G w i,   db = dx x (1 - i),   dg = G (alpha h_{t-1} + i x w'(g)),   w' = -alpha^2 / w | -alpha | 0,
//     da = dg g (1 - s) (sigmoid gate) | -dg e^A_log s (softplus gate),
//     dA_log = sum dg g,  da_bias = sum da,  db_bias = sum db,  dstate_in = alpha G at a sequence's first row.
// The walk is the forward pass's, from the last rows to the first: warps fold their rows to G's map and, from the kept
// h before each tile, to h's, both with the same product of decays.  Of what the gates give only g, h and alpha (in shared
// memory) stay for the second pass over the rows; the rest is made again from the staged rows.
#pragma once

#include "diag_internal.cuh"

namespace gdn {
namespace {

constexpr int LT = 16, W = kDiagTile / LT;      // a warp's rows; warps

template <typename IO, bool CODES> struct Staged {
    IO x[LT][kDiagSlice], a[LT][kDiagSlice], b[LT][kDiagSlice], dy[LT][kDiagSlice];
};
template <typename IO> struct Staged<IO, true> {
    int8_t x[LT][kDiagSlice], a[LT][kDiagSlice], b[LT][kDiagSlice];
    uint8_t xs[LT], as[LT], bs[LT];
    IO dy[LT][kDiagSlice];
};
template <typename IO, bool CODES> struct Shared {
    Staged<IO, CODES> rows[W];
    float2 alpha[W][LT][32];
    DiagMaps maps[2][W], cta_maps[2][8];        // (maps: h's; with `back`, G's)
    float2 back[2][W][32];
    int edge_first[W][LT + 1], edge_last[W][LT + 1];
};

// Rows [r0, r0 + LT) of codes; those outside [lo, hi) as `outside`, with a step of 0 (-1.1e37: a code of 1 shuts a gate).
__device__ __forceinline__ void stage_codes(int8_t *to, uint8_t *to_steps, const DiagParams &p, int k, int slice, int slices, int64_t r0,
                                            int64_t lo, int64_t hi, uint32_t outside, int lane) {
    const int64_t all = (p.rows + kDiagTile - 1) / kDiagTile * kDiagTile, at = ((int64_t)k * slices + slice) * all + r0;
    const int8_t *from = p.codes + at * kDiagSlice;
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to)), ds = static_cast<uint32_t>(__cvta_generic_to_shared(to_steps));
    const bool full = r0 >= lo && r0 + LT <= hi;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int piece = i * 32 + lane;
        const int64_t row = r0 + piece / 4;
        if (full || (row >= lo && row < hi))
            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst + piece * 16), "l"(from + piece * 16) : "memory");
        else
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + piece * 16), "r"(outside) : "memory");
    }
    if (full) {
        if (lane == 0) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ds), "l"(p.steps + at) : "memory");
    } else if (lane < LT) {
        to_steps[lane] = r0 + lane >= lo && r0 + lane < hi ? p.steps[at + lane] : (uint8_t)0;
    }
}
__device__ __forceinline__ F2 code_pair(const int8_t *rows, const uint8_t *steps, int t, int lane) {
    const char2 q = reinterpret_cast<const char2 *>(rows)[t * 32 + lane];
    return mul2({(float)q.x, (float)q.y}, both(code_scale(steps[t])));
}

template <typename IO, int GATE, int WEIGHT, bool CODES>
__global__ void __launch_bounds__(W * 32, sizeof(IO) == 4 ? 2 : 3) diag_backward_kernel(const __grid_constant__ DiagParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Shared<IO, CODES> &sh = *reinterpret_cast<Shared<IO, CODES> *>(raw_shared);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, cl = gridDim.x, rank = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
    const int64_t C = p.channels, c0 = (int64_t)slice * kDiagSlice, c = c0 + 2 * lane;
    if (!offsets_ok(p)) return;
    const DiagPart part = diag_part(p, blockIdx.z, lane);
    if (p.dstate_in)
        for (int n = part.n0 + rank * W + w; n < part.n1; n += cl * W) {     // sequences without tokens
            if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
            store_state(p.dstate_in + n * C, p.dstate_out ? load_state(p.dstate_out + n * C, c, C) : both(0.f), c, C);
        }
    const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, C);
    const F2 unrate = {1.f / l.rate.x, 1.f / l.rate.y};     // (a rate is a normal number or 0, whose channel's opening then counts as 0)
    const F2 inverse = {l.rate.x != 0.f ? unrate.x : 0.f, l.rate.y != 0.f ? unrate.y : 0.f};
    const bool fast = p.pairs && c0 + kDiagSlice <= C, has_b = p.has_b;
    const int64_t tile0 = part.r0 / kDiagTile, lo = part.r0, hi = part.r1;
    const int64_t tiles = hi > lo ? (hi + kDiagTile - 1) / kDiagTile - tile0 : 0;
    Staged<IO, CODES> &st = sh.rows[w];
    float2 *salpha = &sh.alpha[w][0][0];
    const uint32_t shut = shut_bits<IO>();
    auto stage = [&](int64_t w0) {
        if constexpr (CODES) {
            stage_codes(&st.x[0][0], st.xs, p, 0, slice, slices, w0, lo, hi, 0u, lane);
            stage_codes(&st.a[0][0], st.as, p, 1, slice, slices, w0, lo, hi, 0x01010101u, lane);
            if (has_b) stage_codes(&st.b[0][0], st.bs, p, 2, slice, slices, w0, lo, hi, 0u, lane);
        } else {
            stage_rows<IO, LT>(&st.x[0][0], (const IO *)p.x, p.ld_x, w0, lo, hi, c0, C, p.wide, 0u, lane);
            stage_rows<IO, LT>(&st.a[0][0], (const IO *)p.a, p.ld_a, w0, lo, hi, c0, C, p.wide, shut, lane);
            if (has_b) stage_rows<IO, LT>(&st.b[0][0], (const IO *)p.b, p.ld_b, w0, lo, hi, c0, C, p.wide, 0u, lane);
        }
        stage_rows<IO, LT>(&st.dy[0][0], (const IO *)p.dy, p.ld_y, w0, lo, hi, c0, C, p.wide, 0u, lane);
        stage_commit();
    };
    auto get_x = [&](int t) -> F2 {
        if constexpr (CODES) return code_pair(&st.x[0][0], st.xs, t, lane);
        else return staged(&st.x[0][0], t, lane);
    };
    auto get_a = [&](int t) -> F2 {
        if constexpr (CODES) return code_pair(&st.a[0][0], st.as, t, lane);
        else return staged(&st.a[0][0], t, lane);
    };
    auto get_b = [&](int t) -> F2 {
        if (!has_b) return both(0.f);
        if constexpr (CODES) return code_pair(&st.b[0][0], st.bs, t, lane);
        else return staged(&st.b[0][0], t, lane);
    };
    if (tiles > 0 && cl > 1) cluster_arrive();
    if (tiles > rank) stage((tile0 + tiles - 1 - rank) * kDiagTile + w * LT);
    EdgeWindow window = edge_window(p, part.n0, lane);
    F2 carry = both(0.f), sum_A = both(0.f), sum_a = both(0.f), sum_b = both(0.f);
    for (int64_t j0 = 0, step = 0; j0 < tiles; j0 += cl, ++step) {
        const int64_t tile = tile0 + tiles - 1 - j0 - rank, w0 = tile * kDiagTile + w * LT;     // (below tile0: nothing to do)
        const int buf = step & 1;
        const bool some = tile >= tile0 && w0 < hi && w0 + LT > lo, full = some && w0 >= lo && w0 + LT <= hi;
        F2 g[LT], u[LT], sum_g = both(0.f), H = both(0.f), D = both(0.f);
        uint32_t begins = 0, ends = 0;
        if (some) {
            const uint32_t edges = find_edges<LT>(p, window, (uint32_t)w0, part.n0, 28, sh.edge_first[w], sh.edge_last[w], lane);
            uint32_t live = (1u << LT) - 1;
            if (!full) {
                if (w0 < lo) live &= ~0u << (lo - w0);
                if (w0 + LT > hi) live &= (1u << (hi - w0)) - 1;
            }
            begins = edges & live;
            ends = edges >> 1 & live;
        }
        // dy, with a final state's gradient at a sequence's last row
        auto get_dy = [&](int t) -> F2 {
            F2 v = staged(&st.dy[0][0], t, lane);
            if ((ends >> t & 1) && p.dstate_out) v = add2(v, load_state(p.dstate_out + (sh.edge_first[w][t + 1] - 1) * C, c, C));
            return v;
        };
        stage_wait();
        if (some) {
            F2 through = both(1.f);
#pragma unroll
            for (int t = 0; t < LT; ++t) {
                const DiagGates o = diag_gates<GATE, WEIGHT>(get_a(t), get_b(t), has_b, l);
                const F2 v = mul2(o.i, get_x(t));
                g[t] = o.g;
                u[t] = WEIGHT == GDN_DIAG_PLAIN ? v : mul2(o.w, v);
                salpha[t * 32 + lane] = make_float2(o.alpha.x, o.alpha.y);
                sum_g = add2(sum_g, o.g);
                if ((begins | ends) == 0) {
                    H = fma2(o.alpha, H, u[t]);
                    through = mul2(through, o.alpha);
                    D = fma2(through, staged(&st.dy[0][0], t, lane), D);
                }
            }
            if (begins | ends) {
#pragma unroll 1
                for (int t = 0; t < LT; ++t) {
                    if (begins & ((2u << t) - 1)) break;        // (nothing behind a sequence's first row comes back to here)
                    through = mul2(through, get_pair(salpha + t * 32, lane));
                    D = fma2(through, get_dy(t), D);
                }
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    if (begins >> t & 1) H = p.state_in ? load_state(p.state_in + sh.edge_last[w][t] * C, c, C) : both(0.f);
                    H = fma2(get_pair(salpha + t * 32, lane), H, u[t]);
                }
            }
        }
        put_map(sh.maps[buf][w], lane, diag_product(sum_g, begins != 0), H);
        sh.back[buf][w][lane] = make_float2(D.x, D.y);
        __syncthreads();
        F2 G = carry;   // what comes back from the rows behind the CTA's, then behind the warp's
        if (cl > 1) {
            DiagProduct all = get_product(sh.maps[buf][W - 1], lane);
            F2 shift = get_pair(sh.back[buf][W - 1], lane);
#pragma unroll
            for (int k = W - 2; k >= 0; --k) {
                const DiagProduct m = get_product(sh.maps[buf][k], lane);
                shift = diag_apply(m, get_pair(sh.back[buf][k], lane), shift);
                all = diag_join(all, m);
            }
            if (step == 0) cluster_wait();      // (every CTA of the cluster has started)
            for (int r = w; r < cl; r += W) put_map_at(sh.cta_maps[buf][rank], r, lane, all, shift);
            cluster_arrive();
            cluster_wait();
            for (int r = 0; r < cl; ++r) {
                if (r == rank) G = carry;
                carry = diag_apply(get_product(sh.cta_maps[buf][r], lane), get_pair(sh.cta_maps[buf][r].shift, lane), carry);
            }
        }
        F2 back = G;
#pragma unroll
        for (int k = W - 1; k >= 0; --k) {
            if (k == w) back = G;
            G = diag_apply(get_product(sh.maps[buf][k], lane), get_pair(sh.back[buf][k], lane), G);
        }
        if (cl == 1) carry = G;
        if (some) {
            F2 h = both(0.f);
            if (tile * kDiagTile > lo) h = get_pair(reinterpret_cast<const float2 *>(p.kept + (tile * slices + slice) * kDiagSlice), lane);
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (k < w) h = diag_apply(get_product(sh.maps[buf][k], lane), get_pair(sh.maps[buf][k].shift, lane), h);
#pragma unroll
            for (int t = 0; t < LT; ++t) {          // u[t] becomes the h before row t
                if (begins >> t & 1) h = p.state_in ? load_state(p.state_in + sh.edge_last[w][t] * C, c, C) : both(0.f);
                const F2 next = fma2(get_pair(salpha + t * 32, lane), h, u[t]);
                u[t] = h;
                h = next;
            }
            IO *dx = (IO *)p.dx + w0 * p.ld_dx + c, *da = (IO *)p.da + w0 * p.ld_da + c, *db = (IO *)p.db + w0 * p.ld_db + c;
#pragma unroll
            for (int t = LT - 1; t >= 0; --t) {
                if (!full && (w0 + t < lo || w0 + t >= hi)) continue;
                const F2 Gt = add2(get_dy(t), back), alpha = get_pair(salpha + t * 32, lane), x = get_x(t);
                F2 in = both(1.f), nin = both(0.f);         // i and 1 - i = e^-z i
                if (has_b) {
                    const F2 z = fma2(get_b(t), both(-kLog2e), l.nbbias);
                    F2 e = {ex2(z.x), ex2(z.y)};
                    const F2 d = add2(e, both(1.f));
                    in = {rcp(d.x), rcp(d.y)};
                    nin = {in.x > 0.f ? e.x * in.x : 1.f, in.y > 0.f ? e.y * in.y : 1.f};
                }
                const F2 v = mul2(in, x);
                DiagGates o;
                F2 unused;
                o.m = diag_expm1(g[t], unused);
                diag_weigh<WEIGHT>(o);
                F2 dg = mul2(alpha, u[t]);
                if (WEIGHT == GDN_DIAG_NORM) dg = fma2(mul2(v, mul2(alpha, alpha)), F2{-o.winv.x, -o.winv.y}, dg);
                if (WEIGHT == GDN_DIAG_COMPLEMENT) dg = fma2(v, F2{-alpha.x, -alpha.y}, dg);
                dg = mul2(dg, Gt);
                F2 dv = Gt;
                if (WEIGHT != GDN_DIAG_PLAIN) dv = mul2(dv, o.w);
                const F2 dx_ = mul2(dv, in), dgg = mul2(dg, g[t]);
                F2 da_;
                if (GATE == GDN_DIAG_SIGMOID) {             // dg g (1 - s), 1 - s = e^-z s, s = g / rate
                    const F2 z = fma2(get_a(t), both(-kLog2e), l.nabias), s = mul2(g[t], inverse);
                    const F2 e = {fminf(ex2(z.x), 0x1p126f), fminf(ex2(z.y), 0x1p126f)};
                    da_ = mul2(dgg, mul2(e, s));
                } else {                                    // dg rate s, s = 1 - e^-softplus, softplus = g / rate
                    const F2 sp = mul2(g[t], inverse);
                    const F2 s = diag_expm1({-sp.x, -sp.y}, unused);
                    da_ = mul2(dg, mul2(l.rate, F2{-s.x, -s.y}));
                }
                sum_A = add2(sum_A, dgg);
                sum_a = add2(sum_a, da_);
                store_pair<IO>(dx + t * p.ld_dx, dx_, c, C, fast);
                store_pair<IO>(da + t * p.ld_da, da_, c, C, fast);
                if (has_b) {
                    const F2 db_ = mul2(mul2(dv, v), nin);
                    sum_b = add2(sum_b, db_);
                    store_pair<IO>(db + t * p.ld_db, db_, c, C, fast);
                }
                back = mul2(alpha, Gt);
                if (begins >> t & 1) {
                    if (p.dstate_in) store_state(p.dstate_in + sh.edge_last[w][t] * C, back, c, C);
                    back = both(0.f);
                }
            }
        }
        __syncwarp();
        if (tile - cl >= tile0) stage(w0 - cl * kDiagTile);
    }
    // The parameters' gradients: over the CTA's warps, the cluster's CTAs, the parts, in their order.
    __syncthreads();
    float (*sums)[3][kDiagSlice] = reinterpret_cast<float (*)[3][kDiagSlice]>(&sh.alpha[0][0][0]);     // the warps' [W], then rank 0's [8]
    const F2 all[3] = {sum_A, sum_a, sum_b};
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<float2 *>(&sums[8 + w][k][2 * lane]) = make_float2(all[k].x, all[k].y);
    __syncthreads();
    float total[3] = {0.f, 0.f, 0.f};
    if (threadIdx.x < kDiagSlice)
        for (int k = 0; k < 3; ++k)
            for (int r = 0; r < W; ++r) total[k] += sums[8 + r][k][threadIdx.x];
    if (cl > 1) {
        cluster_arrive();               // (every CTA is done with its alphas)
        cluster_wait();
        if (threadIdx.x < kDiagSlice)
            for (int k = 0; k < 3; ++k) {
                const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(&sums[rank][k][threadIdx.x]));
                uint32_t there;
                asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(here));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(total[k]) : "memory");
            }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        if (threadIdx.x < kDiagSlice)
            for (int k = 0; k < 3; ++k) {
                total[k] = 0.f;
                for (int r = 0; r < cl; ++r) total[k] += sums[r][k][threadIdx.x];
            }
    }
    const int64_t ch = c0 + threadIdx.x;
    if (threadIdx.x < kDiagSlice && ch < C) {
        float *out[3] = {p.dA_log, p.da_bias, p.db_bias};
        for (int k = 0; k < 3; ++k) {
            if (p.parts > 1) p.partial[((int64_t)blockIdx.z * 3 + k) * C + ch] = total[k];
            else if (out[k]) out[k][ch] = total[k];
        }
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagParams &p, cudaStream_t stream) {
    const auto kernel = p.codes ? diag_backward_kernel<IO, GATE, WEIGHT, true> : diag_backward_kernel<IO, GATE, WEIGHT, false>;
    const size_t shared = p.codes ? sizeof(Shared<IO, true>) : sizeof(Shared<IO, false>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    const int cl = diag_cluster(p.rows);
    cfg.gridDim = dim3(cl, diag_slices(p.channels), p.parts);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = shared;
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
