// ssm.cu -- the selective state-space scan on the FP32 ALUs: the packed causal convolution
// before it, the token-sequential scan (every type and shape), and the single-token step.
//
//   d_t = clamp(softplus(dt_t + dt_bias)),  a_t = e^{-e^{A_log} d_t}
//   S   = a_t S + d_t B_t (x) x_t           S [d_state][head_dim] per (sequence, head), fp32
//   y_t = (S^T C_t + D x_t) silu(z_t)
// Head h reads B and C of group h / (heads / groups).
#include <type_traits>

#include "ssm_internal.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ causal convolution
// A thread takes V channels and a run of kRun token rows, the last K - 1 rows kept in
// registers; the rows are loaded kAhead at a time, so that enough of them are in flight.
// Products of two 16-bit values are exact in fp32, so the sum's order alone decides its
// value: bias first, then the taps in order.  Bound by reading and writing the rows; the
// arithmetic (13 instructions a value) takes nearly as long.
constexpr int kRun = 32, kAhead = 4;

template <typename IO, int V> struct alignas(sizeof(IO) * V) Pack {
    IO v[V];
};

// silu of V values, each rounded to IO as silu_exact rounds.  For 16-bit types the fast form
// serves unless one of them is within 32 fp32 steps of the border between two 16-bit values: below
// |v| = 8 it is within 12 of the exact form (6 from the exponent's rounding, 2 in the exponential,
// 1 in the reciprocal, the rest in the roundings between).
template <typename IO, int V> __device__ __forceinline__ void silu_rounded(float (&v)[V]) {
    if constexpr (sizeof(IO) == 2) {
        constexpr uint32_t kCut = std::is_same<IO, __half>::value ? 0x1fffu : 0xffffu;    // bits that the rounding drops
        float f[V];
        uint32_t near = 0;
        float top = 0.f, least = 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = v[i] * rcp(1.f + ex2(-kLog2e * v[i]));
            near |= ((__float_as_uint(f[i]) + 32u + (kCut + 1) / 2) & kCut) < 64u;
            top = fmaxf(top, fabsf(v[i]));
            if (kCut == 0x1fffu) least = fminf(least, fabsf(f[i]));    // (f16's subnormals round elsewhere)
        }
        if (!near && top < 8.f && (kCut != 0x1fffu || least > 0x1p-13f)) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = f[i];
            return;
        }
    }
    for (int i = 0; i < V; ++i) v[i] = silu_exact(v[i]);
}

template <typename IO, int V> __device__ __forceinline__ void widen(const Pack<IO, V> &a, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = IoType<IO>::ld(&a.v[i]);
}

template <typename IO, int V, int K>
__global__ void __launch_bounds__(128) ssm_conv_kernel(const SsmConvParams p, int64_t run_blocks) {
    using Vec = Pack<IO, V>;
    const int64_t cv = (int64_t)blockIdx.y * 128 + threadIdx.x;      // channel vector
    if (cv * V >= p.C) return;
    const int c0 = (int)cv * V;
    const IO *x = static_cast<const IO *>(p.x) + c0;
    const IO *cin = p.conv_in ? static_cast<const IO *>(p.conv_in) + c0 : nullptr;
    Vec zero;
#pragma unroll
    for (int i = 0; i < V; ++i) IoType<IO>::st(&zero.v[i], 0.f);

    if ((int64_t)blockIdx.x >= run_blocks) {
        // The last K - 1 inputs of one sequence: its own rows, or past ones where it is short.
        const int64_t n = (int64_t)blockIdx.x - run_blocks;
        int64_t t0, t1;
        if (!seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, n, t0, t1)) return;
        IO *out = static_cast<IO *>(p.conv_out) + (n * (K - 1)) * p.C + c0;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int64_t at = t1 - (K - 1) + j;
            Vec v = zero;
            if (at >= t0) v = *reinterpret_cast<const Vec *>(x + at * p.ld_x);
            else if (cin) v = *reinterpret_cast<const Vec *>(cin + (n * (K - 1) + (t1 - t0) + j) * p.C);
            *reinterpret_cast<Vec *>(out + (int64_t)j * p.C) = v;
        }
        return;
    }

    // Where this thread's channels stand in a row of u.
    int64_t uc;
    const int hp = p.heads * p.head_dim, gn = p.groups * p.d_state;
    if (c0 < hp) {
        uc = (int64_t)(c0 / p.head_dim) * p.x_head + c0 % p.head_dim;
    } else {
        const int b = c0 - hp, in = b % gn;
        uc = (b < gn ? p.off_b : p.off_c) + (int64_t)(in / p.d_state) * p.bc_group + in % p.d_state;
    }
    IO *u = static_cast<IO *>(p.u) + uc;
    float w[K][V], bias[V];
    if (p.w != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = IoType<IO>::ld(static_cast<const IO *>(p.w) + (int64_t)(c0 + i) * K + j);
            bias[i] = p.bias ? IoType<IO>::ld(static_cast<const IO *>(p.bias) + c0 + i) : 0.f;
        }
    }

    const int64_t r0 = (int64_t)blockIdx.x * kRun;
    const int64_t r1 = r0 + kRun < p.rows ? r0 + kRun : p.rows;
    // The sequence of row r0: the last whose first row is not behind it.
    int64_t n = 0, t0 = 0, t1 = p.rows;
    if (p.cu_seqlens == nullptr) {
        n = r0 / p.seqlen;
        t0 = n * p.seqlen;
        t1 = t0 + p.seqlen;
    } else {
        int64_t lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (p.cu_seqlens[mid] <= r0) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
        t0 = p.cu_seqlens[n];
        t1 = p.cu_seqlens[n + 1];
        if (t0 < 0 || t0 > r0) t0 = r0;     // malformed offsets: stay inside the rows (the scan reports them)
        if (t1 <= r0) t1 = r0 + 1;
    }
    float past[K > 1 ? K - 1 : 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t at = r0 - (K - 1) + j;
        Vec v = zero;
        if (at >= t0) v = *reinterpret_cast<const Vec *>(x + at * p.ld_x);
        else if (cin) v = *reinterpret_cast<const Vec *>(cin + (n * (K - 1) + (K - 1) + (at - t0)) * p.C);
        widen<IO, V>(v, past[j]);
    }
    Vec in[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (r0 + i < r1) in[i] = *reinterpret_cast<const Vec *>(x + (r0 + i) * p.ld_x);
#pragma unroll 1
    for (int64_t rb = r0; rb < r1; rb += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t r = rb + i;
            if (r >= r1) break;
            if (r >= t1) {                  // the next sequence that has a row
                if (p.cu_seqlens == nullptr) {
                    ++n;
                    t1 += p.seqlen;
                } else {
                    do ++n;
                    while (n + 1 < p.num_seqs && p.cu_seqlens[n + 1] <= r);
                    if (n >= p.num_seqs) return;
                    t1 = p.cu_seqlens[n + 1];
                    if (t1 <= r) t1 = p.rows;
                }
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    widen<IO, V>(cin ? *reinterpret_cast<const Vec *>(cin + (n * (K - 1) + j) * p.C) : zero, past[j]);
            }
            Vec out = in[i];
            float now[V];
            widen<IO, V>(in[i], now);
            if (r + kAhead < r1) in[i] = *reinterpret_cast<const Vec *>(x + (r + kAhead) * p.ld_x);
            if (p.w != nullptr) {
                float acc[V];
                if constexpr (V % 2 == 0) {
#pragma unroll
                    for (int v = 0; v < V; v += 2) {
                        F2 a = {bias[v], bias[v + 1]};
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) a = fma2({w[j][v], w[j][v + 1]}, {past[j][v], past[j][v + 1]}, a);
                        a = fma2({w[K - 1][v], w[K - 1][v + 1]}, {now[v], now[v + 1]}, a);
                        acc[v] = a.x;
                        acc[v + 1] = a.y;
                    }
                } else {
                    acc[0] = bias[0];
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) acc[0] = fmaf(w[j][0], past[j][0], acc[0]);
                    acc[0] = fmaf(w[K - 1][0], now[0], acc[0]);
                }
                if (p.silu) silu_rounded<IO, V>(acc);
#pragma unroll
                for (int v = 0; v < V; ++v) IoType<IO>::st(&out.v[v], acc[v]);
            }
            *reinterpret_cast<Vec *>(u + r * p.ld_u) = out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) past[j][v] = past[j + 1][v];
                if (K > 1) past[K > 1 ? K - 2 : 0][v] = now[v];
            }
        }
    }
}

template <typename IO, int V>
cudaError_t conv_launch(const SsmConvParams &p, cudaStream_t stream) {
    const int64_t runs = (p.rows + kRun - 1) / kRun;
    const int64_t blocks = runs + (p.K > 1 ? p.num_seqs : 0);
    if (blocks == 0) return cudaSuccess;
    const dim3 grid((unsigned)blocks, (unsigned)((p.C / V + 127) / 128));
    switch (p.K) {
        case 1: ssm_conv_kernel<IO, V, 1><<<grid, 128, 0, stream>>>(p, runs); break;
        case 2: ssm_conv_kernel<IO, V, 2><<<grid, 128, 0, stream>>>(p, runs); break;
        case 3: ssm_conv_kernel<IO, V, 3><<<grid, 128, 0, stream>>>(p, runs); break;
        default: ssm_conv_kernel<IO, V, 4><<<grid, 128, 0, stream>>>(p, runs); break;
    }
    return cudaGetLastError();
}

template <typename IO>
cudaError_t conv_dispatch(const SsmConvParams &p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(IO);
    auto ok = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const bool wide = p.head_dim % V == 0 && p.d_state % V == 0 && p.ld_x % V == 0 && p.ld_u % V == 0 && ok(p.x) && ok(p.u) &&
                      ok(p.conv_in) && ok(p.conv_out) && p.x_head % V == 0 && p.off_b % V == 0 && p.off_c % V == 0 &&
                      p.bc_group % V == 0;
    return wide ? conv_launch<IO, V>(p, stream) : conv_launch<IO, 1>(p, stream);
}

// ------------------------------------------------------------------ token-sequential scan
// A CTA of four warps takes 16 columns of one head's state and walks the sequence.  A warp
// holds four columns; a column's d_state rows are dealt to eight lanes, NS to each, in
// registers.  B, C, x and the gates of kTile tokens are staged in shared memory as fp32,
// the next tile's values loaded while this one is computed.  The eight lanes' partial
// readouts of eight tokens are summed by a reduce-scatter (seven shuffles for eight
// tokens), after which lane slice s owns token s.
constexpr int kTile = 8, kCols = 16, kScanThreads = 128;

template <typename IO, int NS>
__global__ void __launch_bounds__(kScanThreads) ssm_scan_kernel(const SsmParams p) {
    constexpr int NP = 8 * NS, V = NS < 4 ? NS : 4;
    constexpr int LOADS = 2 * NP * kTile / kScanThreads;   // B and C values a thread stages
    __shared__ __align__(16) float sb[2][kTile][2][NP];
    __shared__ float sx[2][kTile][kCols], sg[2][kTile][2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = lane >> 2, col = 4 * warp + (lane & 3);
    const int h = blockIdx.y, g = h / (p.heads / p.groups);
    const int64_t n = blockIdx.x;
    const int c0 = blockIdx.z * kCols;
    const bool live = c0 + col < p.head_dim;
    int64_t t0, t1;
    if (!seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, n, t0, t1)) return;
    const int N = p.d_state, P = p.head_dim;
    auto state_at = [&](int i) { return (i / V) * (8 * V) + slice * V + i % V; };
    const size_t sbase = ((size_t)n * p.heads + h) * (size_t)N * P + c0 + col;

    float S[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        S[i] = (p.state_in && live && state_at(i) < N) ? p.state_in[sbase + (size_t)state_at(i) * P] : 0.f;

    const IO *xs = static_cast<const IO *>(p.xs), *dt = static_cast<const IO *>(p.dt);
    const IO *z = static_cast<const IO *>(p.z);
    const float A = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
    float rb[LOADS], rx, rd;
    // Tile loads: value e of a thread is (token, B or C, row), x one (token, column), dt one token.
    auto load = [&](int64_t tb) {
#pragma unroll
        for (int e = 0; e < LOADS; ++e) {
            const int at = tid + e * kScanThreads, tk = at / (2 * NP), bc = (at / NP) & 1, i = at % NP;
            rb[e] = (tb + tk < t1 && i < N)
                        ? IoType<IO>::ld(xs + (tb + tk) * p.ldx + (bc ? p.off_c : p.off_b) + (int64_t)g * p.bc_group + i)
                        : 0.f;
        }
        const int tk = tid / kCols, c = tid % kCols;
        rx = (tb + tk < t1 && c0 + c < P) ? IoType<IO>::ld(xs + (tb + tk) * p.ldx + (int64_t)h * p.x_head + c0 + c) : 0.f;
        rd = (tid < kTile && tb + tid < t1) ? IoType<IO>::ld(dt + (tb + tid) * p.ld_dt + h) : 0.f;
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int e = 0; e < LOADS; ++e) {
            const int at = tid + e * kScanThreads;
            sb[buf][at / (2 * NP)][(at / NP) & 1][at % NP] = rb[e];
        }
        sx[buf][tid / kCols][tid % kCols] = rx;
        if (tid < kTile) {
            const float d = ssm_step(rd, bias, p.dt_min, p.dt_max);
            sg[buf][tid][0] = d;
            sg[buf][tid][1] = expf(A * d);
        }
    };
    load(t0);
    put(0);
    __syncthreads();
    int buf = 0;
    for (int64_t tb = t0; tb < t1; tb += kTile, buf ^= 1) {
        const bool more = tb + kTile < t1;
        if (more) load(tb + kTile);
        float y[kTile];
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
            y[k] = 0.f;
            if (tb + k < t1) {
                const float a = sg[buf][k][1], dx = sg[buf][k][0] * sx[buf][k][col];
#pragma unroll
                for (int i = 0; i < NS; i += V) {
                    const int at = (i / V) * (8 * V) + slice * V;
                    alignas(16) float b[V], c[V];
                    if constexpr (V == 4) {
                        *reinterpret_cast<float4 *>(b) = *reinterpret_cast<const float4 *>(&sb[buf][k][0][at]);
                        *reinterpret_cast<float4 *>(c) = *reinterpret_cast<const float4 *>(&sb[buf][k][1][at]);
                    } else {
                        *reinterpret_cast<float2 *>(b) = *reinterpret_cast<const float2 *>(&sb[buf][k][0][at]);
                        *reinterpret_cast<float2 *>(c) = *reinterpret_cast<const float2 *>(&sb[buf][k][1][at]);
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        S[i + v] = fmaf(a, S[i + v], dx * b[v]);
                        y[k] = fmaf(c[v], S[i + v], y[k]);
                    }
                }
            }
        }
        // Reduce-scatter over the eight slices (lane bits 2..4): slice s ends with token s.
#pragma unroll
        for (int bit = 2, half = 4; bit >= 0; --bit, half >>= 1) {
            const bool up = (slice >> bit) & 1;
#pragma unroll
            for (int k = 0; k < half; ++k) {
                const float keep = up ? y[k + half] : y[k], give = up ? y[k] : y[k + half];
                y[k] = keep + __shfl_xor_sync(0xffffffffu, give, 4 << bit);
            }
        }
        const int64_t t = tb + slice;
        if (live && t < t1) {
            float out = fmaf(D, sx[buf][slice][col], y[0]);
            const int64_t yc = (int64_t)h * P + c0 + col;
            if (z) out *= silu_gate(IoType<IO>::ld(z + t * p.ld_z + yc));
            IoType<IO>::st(static_cast<IO *>(p.y) + t * (int64_t)p.heads * P + yc, out);
        }
        if (more) put(buf ^ 1);
        __syncthreads();
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (state_at(i) < N) p.state_out[sbase + (size_t)state_at(i) * P] = S[i];
}

template <typename IO>
cudaError_t scan_dispatch(const SsmParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.num_seqs, (unsigned)p.heads, (unsigned)((p.head_dim + kCols - 1) / kCols));
    if (p.d_state <= 16) ssm_scan_kernel<IO, 2><<<grid, kScanThreads, 0, stream>>>(p);
    else if (p.d_state <= 32) ssm_scan_kernel<IO, 4><<<grid, kScanThreads, 0, stream>>>(p);
    else if (p.d_state <= 64) ssm_scan_kernel<IO, 8><<<grid, kScanThreads, 0, stream>>>(p);
    else if (p.d_state <= 128) ssm_scan_kernel<IO, 16><<<grid, kScanThreads, 0, stream>>>(p);
    else ssm_scan_kernel<IO, 32><<<grid, kScanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ single tokens
// A CTA takes one (row, head): its state [N][P] as float4 quads, a thread's quads all of one
// column quad, kDecQuads of them in flight while the row's convolution and gates are
// computed.  Bound by reading and writing the state.
constexpr int kDecThreads = 256, kDecQuads = 8;

template <typename IO>
__device__ __forceinline__ float conv_token(const SsmDecodeParams &p, const IO *x, const IO *conv, int c) {
    const float in = IoType<IO>::ld(x + c);
    if (p.w == nullptr) return in;
    const IO *w = static_cast<const IO *>(p.w) + (int64_t)c * p.K;
    float acc = p.bias ? IoType<IO>::ld(static_cast<const IO *>(p.bias) + c) : 0.f;
    for (int j = 0; j < p.K - 1; ++j) acc = fmaf(IoType<IO>::ld(w + j), IoType<IO>::ld(conv + (int64_t)j * p.C + c), acc);
    acc = fmaf(IoType<IO>::ld(w + p.K - 1), in, acc);
    IO out;
    IoType<IO>::st(&out, p.silu ? silu_exact(acc) : acc);
    return IoType<IO>::ld(&out);
}

// Pool entry of row b, or -1 (a slot outside the pool, reported).
__device__ __forceinline__ int64_t entry_of(const SsmDecodeParams &p, int64_t b) {
    if (p.slots == nullptr) return b;
    const int64_t s = p.slots[b];
    if (s >= 0 && s < p.pool_size) return s;
    atomicOr(p.status, kDevBadSlot);
    return -1;
}

template <typename IO>
__global__ void __launch_bounds__(kDecThreads, 4) ssm_decode_kernel(const SsmDecodeParams p) {
    __shared__ float sB[256], sC[256], sx[256];
    __shared__ __align__(16) float red[kDecThreads * 4];
    const int tid = threadIdx.x, h = blockIdx.x % p.heads;
    const int64_t b = blockIdx.x / p.heads, e = entry_of(p, b);
    if (e < 0) return;
    const int N = p.d_state, P = p.head_dim, Q = P / 4, RP = kDecThreads / Q;
    const int quad = tid % Q, r0 = tid / Q;
    const bool live = r0 < RP;
    float4 *state = reinterpret_cast<float4 *>(p.state + ((size_t)e * p.heads + h) * (size_t)N * P) + quad;

    float4 S[kDecQuads];
#pragma unroll
    for (int m = 0; m < kDecQuads; ++m) {
        const int n = r0 + RP * m;
        if (live && n < N) S[m] = state[(size_t)n * Q];
    }
    const int g = h / (p.heads / p.groups), hp = p.heads * P, gn = p.groups * N;
    const IO *x = static_cast<const IO *>(p.x) + b * p.ld_x;
    const IO *conv = p.conv ? static_cast<const IO *>(p.conv) + e * (int64_t)(p.K - 1) * p.C : nullptr;
    const float d = ssm_step(IoType<IO>::ld(static_cast<const IO *>(p.dt) + b * p.ld_dt + h), p.dt_bias ? p.dt_bias[h] : 0.f,
                             p.dt_min, p.dt_max);
    const float a = expf(-expf(p.A_log[h]) * d), D = p.D ? p.D[h] : 0.f;
    for (int i = tid; i < P + 2 * N; i += kDecThreads) {
        if (i < P) sx[i] = conv_token(p, x, conv, h * P + i);
        else if (i < P + N) sB[i - P] = conv_token(p, x, conv, hp + g * N + i - P);
        else sC[i - P - N] = conv_token(p, x, conv, hp + gn + g * N + i - P - N);
    }
    __syncthreads();

    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        const float4 dx = make_float4(d * sx[4 * quad], d * sx[4 * quad + 1], d * sx[4 * quad + 2], d * sx[4 * quad + 3]);
        for (int base = 0; base < N; base += RP * kDecQuads) {
            if (base > 0) {
#pragma unroll
                for (int m = 0; m < kDecQuads; ++m) {
                    const int n = base + r0 + RP * m;
                    if (n < N) S[m] = state[(size_t)n * Q];
                }
            }
#pragma unroll
            for (int m = 0; m < kDecQuads; ++m) {
                const int n = base + r0 + RP * m;
                if (n < N) {
                    const float bn = sB[n], cn = sC[n];
                    S[m].x = fmaf(a, S[m].x, bn * dx.x); S[m].y = fmaf(a, S[m].y, bn * dx.y);
                    S[m].z = fmaf(a, S[m].z, bn * dx.z); S[m].w = fmaf(a, S[m].w, bn * dx.w);
                    acc.x = fmaf(cn, S[m].x, acc.x); acc.y = fmaf(cn, S[m].y, acc.y);
                    acc.z = fmaf(cn, S[m].z, acc.z); acc.w = fmaf(cn, S[m].w, acc.w);
                    state[(size_t)n * Q] = S[m];
                }
            }
        }
        reinterpret_cast<float4 *>(red)[tid] = acc;
    }
    __syncthreads();
    if (tid < P) {
        float out = 0.f;
        for (int r = 0; r < RP; ++r) out += red[r * P + tid];
        out = fmaf(D, sx[tid], out);
        const int64_t yc = (int64_t)h * P + tid;
        if (p.z) out *= silu_gate(IoType<IO>::ld(static_cast<const IO *>(p.z) + b * p.ld_z + yc));
        IoType<IO>::st(static_cast<IO *>(p.y) + b * (int64_t)hp + yc, out);
    }
}

// The conv states one token on, after the step has read them: rows move up, x comes last.
// (The step's CTAs all read their group's B and C taps, so it cannot move them itself.)
template <typename IO>
__global__ void __launch_bounds__(256) ssm_conv_shift_kernel(const SsmDecodeParams p) {
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int64_t b = blockIdx.x;
    if (c >= p.C) return;
    const int64_t e = p.slots ? (int64_t)p.slots[b] : b;
    if (e < 0 || e >= p.pool_size) return;
    IO *conv = static_cast<IO *>(p.conv) + e * (int64_t)(p.K - 1) * p.C + c;
    for (int j = 0; j + 1 < p.K - 1; ++j) conv[(int64_t)j * p.C] = conv[(int64_t)(j + 1) * p.C];
    conv[(int64_t)(p.K - 2) * p.C] = static_cast<const IO *>(p.x)[b * p.ld_x + c];
}

template <typename IO>
cudaError_t decode_dispatch(const SsmDecodeParams &p, cudaStream_t stream) {
    ssm_decode_kernel<IO><<<(unsigned)(p.heads * p.batch), kDecThreads, 0, stream>>>(p);
    if (p.w != nullptr && p.K > 1)
        ssm_conv_shift_kernel<IO><<<dim3((unsigned)p.batch, (unsigned)((p.C + 255) / 256)), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_conv(const SsmConvParams &p, gdn_dtype io, cudaStream_t stream) {
    if (io == GDN_F32) return conv_dispatch<float>(p, stream);
    return io == GDN_BF16 ? conv_dispatch<__nv_bfloat16>(p, stream) : conv_dispatch<__half>(p, stream);
}

cudaError_t launch_ssm_scan_simt(const SsmParams &p, gdn_dtype io, cudaStream_t stream) {
    if (io == GDN_F32) return scan_dispatch<float>(p, stream);
    return io == GDN_BF16 ? scan_dispatch<__nv_bfloat16>(p, stream) : scan_dispatch<__half>(p, stream);
}

cudaError_t launch_ssm_decode(const SsmDecodeParams &p, gdn_dtype io, cudaStream_t stream) {
    if (io == GDN_F32) return decode_dispatch<float>(p, stream);
    return io == GDN_BF16 ? decode_dispatch<__nv_bfloat16>(p, stream) : decode_dispatch<__half>(p, stream);
}

}  // namespace gdn
