// diag_backward.cu -- gradients of the diagonal recurrence.
//
// With G_t = dy_t + alpha_{t+1} G_{t+1} the gradient at h_t (dstate_out joins at a sequence's last row), and with
// i, s the gates' sigmoids and w(g) the input's weight,
//     dx = G w i,   db = dx x (1 - i),   dg = G (alpha h_{t-1} + i x w'(g)),   w' = -alpha^2 / w | -alpha | 0,
//     da = dg g (1 - s) (sigmoid gate) | -dg e^A_log s (softplus gate),
//     dA_log = sum dg g,  da_bias = sum da,  db_bias = sum db,  dstate_in = alpha G at a sequence's first row.
// The walk is the forward pass's, from the last rows to the first: warps fold their rows to G's map and, from the kept
// h before each tile, to h's, both with the same product of decays.
#include "diag_internal.cuh"

namespace gdn {
namespace {

// What 8-bit codes hold, as the pairs of one row.
template <int N>
__device__ __forceinline__ void load_codes(F2 (&v)[N], const DiagParams &p, int k, int slice, int slices, int64_t r0, int64_t lo,
                                           int64_t hi, int lane) {
    const uint64_t at = ((uint64_t)k * slices + slice) * p.rows + r0;
    char2 q[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const bool in = r0 + t >= lo && r0 + t < hi;
        q[t] = in ? *reinterpret_cast<const char2 *>(p.codes + (at + t) * kDiagSlice + 2 * lane) : make_char2(0, 0);
    }
    const uint32_t e = lane < N && r0 + lane >= lo && r0 + lane < hi ? p.steps[at + lane] : 16u;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const float s = code_scale(__shfl_sync(~0u, e, t));
        v[t] = mul2({(float)q[t].x, (float)q[t].y}, both(s));
    }
}

template <typename IO, int GATE, int WEIGHT, int LT, bool CODES>
__global__ void __launch_bounds__(kDiagTile / LT * 32) diag_backward_kernel(const __grid_constant__ DiagParams p) {
    constexpr int W = kDiagTile / LT;
    __shared__ DiagMaps maps[2][W], cta_maps[2][8];     // (maps: h's; the same products with `back` G's)
    __shared__ float2 back_shift[2][W][32];
    __shared__ int edge_first[W][LT + 1], edge_last[W][LT + 1];
    __shared__ float sums[8][3][kDiagSlice];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, cl = gridDim.x, rank = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
    const int64_t C = p.channels, c = (int64_t)slice * kDiagSlice + 2 * lane;
    if (!offsets_ok(p)) return;
    const DiagPart part = diag_part(p, blockIdx.z, lane);
    if (p.dstate_in)
        for (int n = part.n0 + rank * W + w; n < part.n1; n += cl * W) {     // sequences without tokens
            if (seq_begin(p, n) != seq_begin(p, n + 1)) continue;
            store_state(p.dstate_in + n * C, p.dstate_out ? load_state(p.dstate_out + n * C, c, C) : both(0.f), c, C);
        }
    const DiagLane l = diag_lane(p.A_log, p.a_bias, p.b_bias, c, C);
    const bool fast = p.pairs && (slice + 1) * kDiagSlice <= C, has_b = p.has_b;
    const int64_t tile0 = part.r0 / kDiagTile, lo = part.r0, hi = part.r1;
    const int64_t tiles = hi > lo ? (hi + kDiagTile - 1) / kDiagTile - tile0 : 0;
    if (cl > 1 && tiles > 0) cluster_arrive();
    F2 carry = both(0.f), sum_A = both(0.f), sum_a = both(0.f), sum_b = both(0.f);
    for (int64_t j0 = 0, step = 0; j0 < tiles; j0 += cl, ++step) {
        const int64_t tile = tile0 + tiles - 1 - j0 - rank, w0 = tile * kDiagTile + w * LT;     // (below tile0: nothing to do)
        const int buf = step & 1;
        const bool some = tile >= tile0 && w0 < hi && w0 + LT > lo;
        typename Pair<IO>::Raw dy[LT];
        F2 x[LT], g[LT], m[LT], alpha[LT], s[LT], in[LT], u[LT], sum_g = both(0.f), H = both(0.f), D = both(0.f);
        uint32_t edges = 0;
        bool anew = false;
        if (some) {
            int from = part.n0;
            edges = find_edges<LT>(p, (uint32_t)w0, from, edge_first[w], edge_last[w], lane);
            F2 a[LT], b[LT];
            load_rows<IO, LT>(dy, (const IO *)p.dy, p.ld_y, w0, lo, hi, c, C, fast);
            if (CODES) {
                load_codes<LT>(x, p, 0, slice, slices, w0, lo, hi, lane);
                load_codes<LT>(a, p, 1, slice, slices, w0, lo, hi, lane);
                if (has_b) load_codes<LT>(b, p, 2, slice, slices, w0, lo, hi, lane);
            } else {
                typename Pair<IO>::Raw rx[LT], ra[LT], rb[LT];
                load_rows<IO, LT>(rx, (const IO *)p.x, p.ld_x, w0, lo, hi, c, C, fast);
                load_rows<IO, LT>(ra, (const IO *)p.a, p.ld_a, w0, lo, hi, c, C, fast);
                if (has_b) load_rows<IO, LT>(rb, (const IO *)p.b, p.ld_b, w0, lo, hi, c, C, fast);
#pragma unroll
                for (int t = 0; t < LT; ++t) {
                    x[t] = Pair<IO>::wide(rx[t]);
                    a[t] = Pair<IO>::wide(ra[t]);
                    b[t] = has_b ? Pair<IO>::wide(rb[t]) : both(0.f);
                }
            }
#pragma unroll
            for (int t = 0; t < LT; ++t) {
                const DiagGates o = diag_gates<GATE, WEIGHT, true>(a[t], b[t], has_b, l);
                const bool here = w0 + t >= lo && w0 + t < hi;
                g[t] = o.g;
                m[t] = o.m;
                s[t] = o.s;
                in[t] = o.i;
                const F2 v = mul2(o.i, x[t]);
                u[t] = here ? (WEIGHT == GDN_DIAG_PLAIN ? v : mul2(o.w, v)) : both(0.f);
                alpha[t] = here ? o.alpha : both(1.f);
                if (here && (edges >> t & 1)) {
                    anew = true;
                    H = p.state_in ? fma2(alpha[t], load_state(p.state_in + edge_last[w][t] * C, c, C), u[t]) : u[t];
                } else {
                    H = fma2(alpha[t], H, u[t]);
                }
                if (here) sum_g = add2(sum_g, o.g);
            }
#pragma unroll
            for (int t = LT - 1; t >= 0; --t) {
                if (w0 + t < lo || w0 + t >= hi) continue;
                F2 G = add2(Pair<IO>::wide(dy[t]), D);
                if ((edges >> (t + 1) & 1) && p.dstate_out)
                    G = add2(G, load_state(p.dstate_out + (edge_first[w][t + 1] - 1) * C, c, C));
                D = edges >> t & 1 ? both(0.f) : mul2(alpha[t], G);
            }
        }
        put_map(maps[buf][w], lane, diag_product(sum_g, anew), H);
        back_shift[buf][w][lane] = make_float2(D.x, D.y);
        __syncthreads();
        F2 G = carry;   // what comes back from the rows behind the CTA's, then behind the warp's
        if (cl > 1) {
            DiagProduct all = get_product(maps[buf][W - 1], lane);
            F2 shift = get_pair(back_shift[buf][W - 1], lane);
#pragma unroll
            for (int k = W - 2; k >= 0; --k) {
                const DiagProduct m = get_product(maps[buf][k], lane);
                shift = diag_apply(m, get_pair(back_shift[buf][k], lane), shift);
                all = diag_join(all, m);
            }
            if (step == 0) cluster_wait();      // (every CTA of the cluster has started)
            for (int r = w; r < cl; r += W) put_map_at(cta_maps[buf][rank], r, lane, all, shift);
            cluster_arrive();
            cluster_wait();
            for (int r = 0; r < cl; ++r) {
                if (r == rank) G = carry;
                carry = diag_apply(get_product(cta_maps[buf][r], lane), get_pair(cta_maps[buf][r].shift, lane), carry);
            }
        }
        F2 back = G;
#pragma unroll
        for (int k = W - 1; k >= 0; --k) {
            if (k == w) back = G;
            G = diag_apply(get_product(maps[buf][k], lane), get_pair(back_shift[buf][k], lane), G);
        }
        if (cl == 1) carry = G;
        if (some) {
            F2 h = both(0.f);
            if (tile * kDiagTile > lo) {
                const float2 k = *reinterpret_cast<const float2 *>(p.kept + (tile * slices + slice) * kDiagSlice + 2 * lane);
                h = {k.x, k.y};
            }
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (k < w) h = diag_apply(get_product(maps[buf][k], lane), get_pair(maps[buf][k].shift, lane), h);
#pragma unroll
            for (int t = 0; t < LT; ++t) {          // u[t] becomes the h before row t
                if ((edges >> t & 1) && w0 + t >= lo && w0 + t < hi) h = p.state_in ? load_state(p.state_in + edge_last[w][t] * C, c, C) : both(0.f);
                const F2 next = fma2(alpha[t], h, u[t]);
                u[t] = h;
                h = next;
            }
#pragma unroll
            for (int t = LT - 1; t >= 0; --t) {
                const int64_t row = w0 + t;
                if (row < lo || row >= hi) continue;
                F2 Gt = add2(Pair<IO>::wide(dy[t]), back);
                if ((edges >> (t + 1) & 1) && p.dstate_out)
                    Gt = add2(Gt, load_state(p.dstate_out + (edge_first[w][t + 1] - 1) * C, c, C));
                const F2 v = mul2(in[t], x[t]);
                DiagGates o;
                o.m = m[t];
                diag_weigh<WEIGHT>(o);
                F2 dg = mul2(alpha[t], u[t]);
                if (WEIGHT == GDN_DIAG_NORM) dg = fma2(mul2(v, mul2(alpha[t], alpha[t])), F2{-o.winv.x, -o.winv.y}, dg);
                if (WEIGHT == GDN_DIAG_COMPLEMENT) dg = fma2(v, F2{-alpha[t].x, -alpha[t].y}, dg);
                dg = mul2(dg, Gt);
                F2 dx = mul2(Gt, in[t]);
                if (WEIGHT != GDN_DIAG_PLAIN) dx = mul2(dx, o.w);
                const F2 dgg = mul2(dg, g[t]);
                const F2 da = GATE == GDN_DIAG_SIGMOID ? fma2(dgg, F2{-s[t].x, -s[t].y}, dgg) : mul2(dg, mul2(l.rate, s[t]));
                sum_A = add2(sum_A, dgg);
                sum_a = add2(sum_a, da);
                store_pair<IO>((IO *)p.dx + row * p.ld_dx + c, dx, c, C, fast);
                store_pair<IO>((IO *)p.da + row * p.ld_da + c, da, c, C, fast);
                if (has_b) {
                    const F2 dxx = mul2(dx, x[t]), db = fma2(dxx, F2{-in[t].x, -in[t].y}, dxx);
                    sum_b = add2(sum_b, db);
                    store_pair<IO>((IO *)p.db + row * p.ld_db + c, db, c, C, fast);
                }
                back = mul2(alpha[t], Gt);
                if (edges >> t & 1) {
                    if (p.dstate_in) store_state(p.dstate_in + edge_last[w][t] * C, back, c, C);
                    back = both(0.f);
                }
            }
        }
        __syncwarp();
    }
    // The parameters' gradients: over the CTA's warps, the cluster's CTAs, the parts, in their order.
    __syncthreads();
    float *mine = &sums[0][0][0];       // [W][3][64], then rank 0's [cl][3][64]
    static_assert(W <= 8, "the warps' sums share the CTAs'");
    const F2 all[3] = {sum_A, sum_a, sum_b};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        mine[(w * 3 + k) * kDiagSlice + 2 * lane] = all[k].x;
        mine[(w * 3 + k) * kDiagSlice + 2 * lane + 1] = all[k].y;
    }
    __syncthreads();
    float total[3] = {0.f, 0.f, 0.f};
    if (threadIdx.x < kDiagSlice)
        for (int k = 0; k < 3; ++k)
            for (int r = 0; r < W; ++r) total[k] += mine[(r * 3 + k) * kDiagSlice + threadIdx.x];
    if (cl > 1) {
        __syncthreads();                // (every CTA has read its warps' sums before another writes over them)
        cluster_arrive();
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
    const int64_t ch = (int64_t)slice * kDiagSlice + threadIdx.x;
    if (threadIdx.x < kDiagSlice && ch < C) {
        float *out[3] = {p.dA_log, p.da_bias, p.db_bias};
        for (int k = 0; k < 3; ++k) {
            if (p.parts > 1) p.partial[((int64_t)blockIdx.z * 3 + k) * C + ch] = total[k];
            else if (out[k]) out[k][ch] = total[k];
        }
    }
}

// The parts' sums in their order.
__global__ void diag_sum_parts(const __grid_constant__ DiagParams p) {
    if (!offsets_ok(p)) return;
    const int64_t C = p.channels, ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int k = blockIdx.y;
    float *out = k == 0 ? p.dA_log : k == 1 ? p.da_bias : p.db_bias;
    if (ch >= C || out == nullptr) return;
    float t = 0.f;
    for (int q = 0; q < p.parts; ++q) t += p.partial[((int64_t)q * 3 + k) * C + ch];
    out[ch] = t;
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
    const cudaError_t e = p.codes ? cudaLaunchKernelEx(&cfg, diag_backward_kernel<IO, GATE, WEIGHT, LT, true>, p)
                                  : cudaLaunchKernelEx(&cfg, diag_backward_kernel<IO, GATE, WEIGHT, LT, false>, p);
    return e;
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

cudaError_t launch_diag_backward(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream) {
    cudaError_t e;
    switch (io) {
        case GDN_F32: e = by_kind<float>(p, gate, weighting, stream); break;
        case GDN_BF16: e = by_kind<__nv_bfloat16>(p, gate, weighting, stream); break;
        default: e = by_kind<__half>(p, gate, weighting, stream);
    }
    if (e != cudaSuccess || p.parts == 1 || !(p.dA_log || p.da_bias || p.db_bias)) return e;
    diag_sum_parts<<<dim3((p.channels + 255) / 256, 3), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
