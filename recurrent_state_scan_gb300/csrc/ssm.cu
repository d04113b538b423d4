// ssm.cu -- the selective state-space scan on the FP32 ALUs: the packed causal convolution
// before it, the token-sequential scan (every type and shape), and the single-token step.
//
//   d_t = clamp(softplus(dt_t + dt_bias)),  a_t = e^{-e^{A_log} d_t}
//   S   = a_t S + d_t B_t (x) x_t           S [d_state][head_dim] per (sequence, head), fp32
//   y_t = (S^T C_t + D x_t) silu(z_t)
// Head h reads B and C of group h / (heads / groups).
#include <type_traits>

#include "ssm_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

constexpr int kSms = 152;

// ------------------------------------------------------------------ causal convolution
// A thread takes V channels and a run of up to kRun token rows, the last K - 1 rows kept in
// registers; the rows are loaded kAhead at a time, so that enough of them are in flight.
// Products of two 16-bit values are exact in fp32, so the sum's order alone decides its
// value: bias first, then the taps in order.  Bound by reading and writing the rows; the
// arithmetic (13 instructions a value) takes nearly as long.
constexpr int kRun = 33, kAhead = 3;

// Rows of a run: as many runs as fill the SMs, six CTAs to each, in whole waves of runs of up to
// `most` rows, in whole stages.  (Runs of 72 rows: 2,002 rows of 1,792 f16 channels took 29 us, in
// runs of 12 by bulk copies below 12 us; 1,045 f32 rows of 704 channels here 27.5 us in runs of 33, 7.6
// in runs of 3, although each run reads K - 1 rows more.  8,192 rows of 4,352 channels take
// 8 us more in runs of 72, a wave and a bit, than in runs of 84, one wave.)
int rows_of_run(int64_t rows, int64_t across, int most, int stage) {
    const int64_t work = rows * across, wave = 6 * kSms, waves = (work + most * wave - 1) / (most * wave);
    const int64_t run = waves == 0 ? stage : (work + waves * wave - 1) / (waves * wave);
    return (int)((run + stage - 1) / stage * stage);
}

template <typename IO, int V> struct alignas(sizeof(IO) * V) Pack {
    IO v[V];
};

// silu of V values, each rounded to IO as silu_exact rounds.  For 16-bit types a fast form serves
// where it is not within 8 fp32 steps of the border between two 16-bit values.  Its exponent -v log2 e is
// carried in two terms (log2 e is kHi and what its fp32 rounding leaves, kLo; the second comes in as e (1 +
// rest ln 2)), so below |v| = 64 it is near silu_exact: at most 5 steps, counted over every fp32 value, of
// which none rounds otherwise in either type.  (The operations' bounds alone, some 6 units of
// 2^-23 for both forms together, come to 12 steps where the result's mantissa is near 2.)
__device__ __noinline__ float4 silu_apart(float4 v) {
    return make_float4(silu_exact(v.x), silu_exact(v.y), silu_exact(v.z), silu_exact(v.w));
}

template <typename IO, int V> __device__ __forceinline__ void silu_rounded(float (&v)[V]) {
    if constexpr (sizeof(IO) == 2 && V == 4) {
        constexpr bool kHalf = std::is_same<IO, __half>::value;
        constexpr uint32_t kCut = kHalf ? 0x1fffu : 0xffffu;    // bits that the rounding drops
        constexpr float kHi = -kLog2e, kLo = -1.925963033e-8f;
        float f[V], top = 0.f, low = 1.f;
        uint32_t off = ~0u;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const F2 x = {v[i], v[i + 1]}, t = mul2(x, both(kHi));
            const F2 rest = fma2(x, both(kLo), fma2(x, both(kHi), mul2(x, both(-kHi))));   // (the last is -t)
            F2 e = {ex2(t.x), ex2(t.y)};
            e = fma2(e, mul2(rest, both(0.69314718f)), e);
            const F2 d = add2(e, both(1.f)), y = mul2(x, {rcp(d.x), rcp(d.y)});
            f[i] = y.x;
            f[i + 1] = y.y;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            off = min(off, (__float_as_uint(f[i]) + 8u + (kCut + 1) / 2) & (kCut & ~15u));   // 0: near a border
            top = fmaxf(top, fabsf(v[i]));
            if (kHalf) low = fminf(low, fabsf(f[i]));    // (f16's subnormals round elsewhere)
        }
        const bool sure = off != 0 && top < 64.f && (!kHalf || low > 0x1p-13f);
        if (!sure) {
            const float4 s = silu_apart(make_float4(v[0], v[1], v[2], v[3]));
            f[0] = s.x; f[1] = s.y; f[2] = s.z; f[3] = s.w;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = silu_exact(v[i]);
    }
}

template <typename IO, int V> __device__ __forceinline__ void widen(const Pack<IO, V> &a, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = IoType<IO>::ld(&a.v[i]);
}

// The last K - 1 inputs of sequence n: its own rows, or past ones where it is short.
template <typename IO, int V, int K>
__device__ __forceinline__ void conv_states(const SsmConvParams &p, int64_t n, int c0) {
    using Vec = Pack<IO, V>;
    int64_t t0, t1;
    if (!seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, n, t0, t1)) return;
    const IO *x = static_cast<const IO *>(p.x) + c0, *cin = p.conv_in ? static_cast<const IO *>(p.conv_in) + c0 : nullptr;
    IO *out = static_cast<IO *>(p.conv_out) + (n * (K - 1)) * p.C + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t at = t1 - (K - 1) + j;
        Vec v;
#pragma unroll
        for (int i = 0; i < V; ++i) IoType<IO>::st(&v.v[i], 0.f);
        if (at >= t0) v = *reinterpret_cast<const Vec *>(x + at * p.ld_x);
        else if (cin) v = *reinterpret_cast<const Vec *>(cin + (n * (K - 1) + (t1 - t0) + j) * p.C);
        *reinterpret_cast<Vec *>(out + (int64_t)j * p.C) = v;
    }
}

// The sequence of a run of rows and the walk along it, for both convolution kernels.
struct Walk {
    int64_t n, t0, t1;      // sequence, its first row, the row behind it
};
__device__ __forceinline__ Walk walk_from(const SsmConvParams &p, int64_t r0) {
    Walk w{0, 0, p.rows};
    if (p.cu_seqlens == nullptr) {
        w.n = r0 / p.seqlen;
        w.t0 = w.n * p.seqlen;
        w.t1 = w.t0 + p.seqlen;
        return w;
    }
    int64_t lo = 0, hi = p.num_seqs - 1;         // the last sequence whose first row is not behind r0
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= r0) lo = mid;
        else hi = mid - 1;
    }
    w.n = lo;
    w.t0 = p.cu_seqlens[lo];
    w.t1 = p.cu_seqlens[lo + 1];
    if (w.t0 < 0 || w.t0 > r0) w.t0 = r0;        // malformed offsets: stay inside the rows (the scan reports them)
    if (w.t1 <= r0) w.t1 = r0 + 1;
    return w;
}
// The next sequence that has row r; false: none.
__device__ __forceinline__ bool walk_on(const SsmConvParams &p, Walk &w, int64_t r) {
    if (p.cu_seqlens == nullptr) {
        ++w.n;
        w.t1 += p.seqlen;
        return true;
    }
    do ++w.n;
    while (w.n + 1 < p.num_seqs && p.cu_seqlens[w.n + 1] <= r);
    if (w.n >= p.num_seqs) return false;
    w.t1 = p.cu_seqlens[w.n + 1];
    if (w.t1 <= r) w.t1 = p.rows;
    return true;
}
// Where channel c0 of a row of x stands in a row of u.
__device__ __forceinline__ int64_t u_channel(const SsmConvParams &p, int c0) {
    const int hp = p.heads * p.head_dim, gn = p.groups * p.d_state;
    if (c0 < hp) return (int64_t)(c0 / p.head_dim) * p.x_head + c0 % p.head_dim;
    const int b = c0 - hp, in = b % gn;
    return (b < gn ? p.off_b : p.off_c) + (int64_t)(in / p.d_state) * p.bc_group + in % p.d_state;
}

template <typename IO, int V, int K>
__global__ void __launch_bounds__(128) ssm_conv_kernel(const SsmConvParams p, int64_t run_blocks, int run) {
    using Vec = Pack<IO, V>;
    const int64_t cv = (int64_t)blockIdx.y * 128 + threadIdx.x;      // channel vector
    if (cv * V >= p.C) return;
    const int c0 = (int)cv * V;
    if ((int64_t)blockIdx.x >= run_blocks) {
        conv_states<IO, V, K>(p, (int64_t)blockIdx.x - run_blocks, c0);
        return;
    }
    const IO *x = static_cast<const IO *>(p.x) + c0;
    const IO *cin = p.conv_in ? static_cast<const IO *>(p.conv_in) + c0 : nullptr;
    Vec zero;
#pragma unroll
    for (int i = 0; i < V; ++i) IoType<IO>::st(&zero.v[i], 0.f);
    IO *u = static_cast<IO *>(p.u) + u_channel(p, c0);
    float w[K][V], bias[V];
    if (p.w != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = IoType<IO>::ld(static_cast<const IO *>(p.w) + (int64_t)(c0 + i) * K + j);
            bias[i] = p.bias ? IoType<IO>::ld(static_cast<const IO *>(p.bias) + c0 + i) : 0.f;
        }
    }

    const int64_t r0 = (int64_t)blockIdx.x * run;
    const int64_t r1 = r0 + run < p.rows ? r0 + run : p.rows;
    Walk seq = walk_from(p, r0);
    float past[K > 1 ? K - 1 : 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t at = r0 - (K - 1) + j;
        Vec v = zero;
        if (at >= seq.t0) v = *reinterpret_cast<const Vec *>(x + at * p.ld_x);
        else if (cin) v = *reinterpret_cast<const Vec *>(cin + (seq.n * (K - 1) + (K - 1) + (at - seq.t0)) * p.C);
        widen<IO, V>(v, past[j]);
    }
    const int left = (int)(r1 - r0);            // rows of this run, and of its first sequence
    int turn = seq.t1 - r0 < left ? (int)(seq.t1 - r0) : left;
    const IO *px = x + r0 * p.ld_x;
    u += r0 * p.ld_u;
    Vec in[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i, px += p.ld_x)
        if (i < left) in[i] = *reinterpret_cast<const Vec *>(px);
#pragma unroll 1
    for (int done = 0; done < left; done += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, px += p.ld_x, u += p.ld_u) {
            if (done + i >= left) break;
            if (done + i >= turn) {             // the next sequence that has a row
                if (!walk_on(p, seq, r0 + done + i)) return;
                turn = seq.t1 - r0 < left ? (int)(seq.t1 - r0) : left;
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    widen<IO, V>(cin ? *reinterpret_cast<const Vec *>(cin + (seq.n * (K - 1) + j) * p.C) : zero, past[j]);
            }
            Vec out = in[i];
            float now[V];
            widen<IO, V>(in[i], now);
            if (done + i + kAhead < left) in[i] = *reinterpret_cast<const Vec *>(px);
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
            *reinterpret_cast<Vec *>(u) = out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) past[j][v] = past[j + 1][v];
                if (K > 1) past[K > 1 ? K - 2 : 0][v] = now[v];
            }
        }
    }
}

// The convolution of 16-bit rows that bulk copies can take (16-byte rows and channel runs): a CTA
// takes 512 channels of a run of up to kBulkRun rows, which arrive kStageRows at a time in a ring of
// kBulkRing stages; a thread reads its four channels of each row once, the last K - 1 rows kept in
// registers, and writes them straight out.  (The kernel above, with its loads in registers, holds
// 18 KB in flight to an SM, and took 91 us for 8,192 rows of 4,352 channels; this one 150 KB: 40 us.)
// Bound by issue (66% of the slots, mostly the silu's), at 3.6 TB/s there and 4.2 TB/s for 16,384
// rows of 6,144 channels (95 us).  A barrier to a stage costs no more than counting its readers.
constexpr int kStageRows = 6, kBulkRing = 4, kBulkRun = 96, kBulkChannels = 512;

template <typename IO, int K>
__global__ void __launch_bounds__(128, 6) ssm_conv_bulk_kernel(const SsmConvParams p, int64_t run_blocks, int run) {
    using namespace tc;
    constexpr int V = 4;
    using Vec = Pack<IO, V>;
    __shared__ __align__(128) IO ring[kBulkRing][kStageRows][kBulkChannels];
    __shared__ uint64_t full[kBulkRing];
    const int tid = threadIdx.x, cta0 = blockIdx.y * kBulkChannels, c0 = cta0 + V * tid;
    if ((int64_t)blockIdx.x >= run_blocks) {
        if (c0 < p.C) conv_states<IO, V, K>(p, (int64_t)blockIdx.x - run_blocks, c0);
        return;
    }
    const int64_t r0 = (int64_t)blockIdx.x * run;
    const int left = (int)(p.rows - r0 < run ? p.rows - r0 : run), stages = (left + kStageRows - 1) / kStageRows;
    const uint32_t bytes = 2u * (uint32_t)(p.C - cta0 < kBulkChannels ? p.C - cta0 : kBulkChannels);
    if (tid == 0) {
        for (int i = 0; i < kBulkRing; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto fetch = [&](int s) {
        const int rows = left - s * kStageRows < kStageRows ? left - s * kStageRows : kStageRows;
        const IO *from = static_cast<const IO *>(p.x) + (r0 + s * kStageRows) * p.ld_x + cta0;
        mbar_arrive_expect_tx(&full[s % kBulkRing], rows * bytes);
        for (int i = 0; i < rows; ++i) bulk_load(ring[s % kBulkRing][i], from + i * p.ld_x, bytes, &full[s % kBulkRing]);
    };
    if (tid == 0)
        for (int s = 0; s < kBulkRing && s < stages; ++s) fetch(s);

    const bool live = c0 < p.C;
    const IO *x = static_cast<const IO *>(p.x) + c0, *cin = p.conv_in ? static_cast<const IO *>(p.conv_in) + c0 : nullptr;
    Walk at = walk_from(p, r0);
    float w[K][V], bias[V], past[K > 1 ? K - 1 : 1][V];
    IO *u = static_cast<IO *>(p.u) + r0 * p.ld_u;
    if (live) {
        u += u_channel(p, c0);
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = IoType<IO>::ld(static_cast<const IO *>(p.w) + (int64_t)(c0 + i) * K + j);
            bias[i] = p.bias ? IoType<IO>::ld(static_cast<const IO *>(p.bias) + c0 + i) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int64_t r = r0 - (K - 1) + j;
#pragma unroll
            for (int v = 0; v < V; ++v) past[j][v] = 0.f;
            if (r >= at.t0) widen<IO, V>(*reinterpret_cast<const Vec *>(x + r * p.ld_x), past[j]);
            else if (cin) widen<IO, V>(*reinterpret_cast<const Vec *>(cin + (at.n * (K - 1) + (K - 1) + (r - at.t0)) * p.C), past[j]);
        }
    }
    int turn = at.t1 - r0 < left ? (int)(at.t1 - r0) : left;
    bool ok = true, more = true;       // more: the offsets lead to a sequence for the next row
    auto taps = [&](const float (*in)[V], float (&acc)[V]) {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            F2 a = {bias[v], bias[v + 1]};
#pragma unroll
            for (int j = 0; j < K; ++j) a = fma2({w[j][v], w[j][v + 1]}, {in[j][v], in[j][v + 1]}, a);
            acc[v] = a.x;
            acc[v + 1] = a.y;
        }
    };
    auto emit = [&](float (&acc)[V], IO *to) {
        if (p.silu) silu_rounded<IO, V>(acc);
        Vec out;
#pragma unroll
        for (int v = 0; v < V; ++v) IoType<IO>::st(&out.v[v], acc[v]);
        *reinterpret_cast<Vec *>(to) = out;
    };
#pragma unroll 1
    for (int s = 0; s < stages; ++s) {
        ok = mbar_wait(&full[s % kBulkRing], (s / kBulkRing) & 1, 4000000000LL) && ok;
        const IO(*stage)[kBulkChannels] = ring[s % kBulkRing];
        const int first = s * kStageRows;
        if (live && ok && more && first + kStageRows <= turn) {
            // A whole stage of one sequence (turn is not behind the run).
            float in[K - 1 + kStageRows][V];
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) in[j][v] = past[j][v];
#pragma unroll
            for (int i = 0; i < kStageRows; ++i) widen<IO, V>(*reinterpret_cast<const Vec *>(&stage[i][V * tid]), in[K - 1 + i]);
#pragma unroll
            for (int i = 0; i < kStageRows; ++i, u += p.ld_u) {
                float acc[V];
                taps(&in[i], acc);
                emit(acc, u);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) past[j][v] = in[kStageRows + j][v];
        } else if (live && ok && more) {
#pragma unroll 1
            for (int i = 0; i < kStageRows; ++i, u += p.ld_u) {
                const int r = first + i;
                if (r >= left) break;
                if (r >= turn) {
                    if (!(more = walk_on(p, at, r0 + r))) break;
                    turn = at.t1 - r0 < left ? (int)(at.t1 - r0) : left;
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) {
#pragma unroll
                        for (int v = 0; v < V; ++v) past[j][v] = 0.f;
                        if (cin) widen<IO, V>(*reinterpret_cast<const Vec *>(cin + (at.n * (K - 1) + j) * p.C), past[j]);
                    }
                }
                float in[K][V], acc[V];
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) in[j][v] = past[j][v];
                widen<IO, V>(*reinterpret_cast<const Vec *>(&stage[i][V * tid]), in[K - 1]);
                taps(in, acc);
                emit(acc, u);
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) past[j][v] = in[j + 1][v];
            }
        }
        __syncthreads();        // the stage has been read
        if (tid == 0 && s + kBulkRing < stages) fetch(s + kBulkRing);
    }
    if (!ok && tid == 0) atomicOr(p.status, kDevTimeout);
}

template <typename IO, int V>
cudaError_t conv_launch(const SsmConvParams &p, cudaStream_t stream) {
    const int64_t across = (p.C / V + 127) / 128;
    const int run = rows_of_run(p.rows, across, kRun, kAhead);
    const int64_t runs = (p.rows + run - 1) / run;
    const int64_t blocks = runs + (p.K > 1 ? p.num_seqs : 0);
    if (blocks == 0) return cudaSuccess;
    const dim3 grid((unsigned)blocks, (unsigned)across);
    switch (p.K) {
        case 1: ssm_conv_kernel<IO, V, 1><<<grid, 128, 0, stream>>>(p, runs, run); break;
        case 2: ssm_conv_kernel<IO, V, 2><<<grid, 128, 0, stream>>>(p, runs, run); break;
        case 3: ssm_conv_kernel<IO, V, 3><<<grid, 128, 0, stream>>>(p, runs, run); break;
        default: ssm_conv_kernel<IO, V, 4><<<grid, 128, 0, stream>>>(p, runs, run); break;
    }
    return cudaGetLastError();
}

template <typename IO>
cudaError_t conv_dispatch(const SsmConvParams &p, cudaStream_t stream) {
    constexpr int V = 4;
    auto ok = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & (V * sizeof(IO) - 1)) == 0; };
    const bool wide = p.head_dim % V == 0 && p.d_state % V == 0 && p.ld_x % V == 0 && p.ld_u % V == 0 && ok(p.x) && ok(p.u) &&
                      ok(p.conv_in) && ok(p.conv_out) && p.x_head % V == 0 && p.off_b % V == 0 && p.off_c % V == 0 &&
                      p.bc_group % V == 0;
    if constexpr (sizeof(IO) == 2) {
        auto by16 = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
        if (wide && p.w != nullptr && p.rows > 0 && p.C % 8 == 0 && p.ld_x % 8 == 0 && by16(p.x)) {
            const int64_t across = (p.C + kBulkChannels - 1) / kBulkChannels;
            const int run = rows_of_run(p.rows, across, kBulkRun, kStageRows);
            const int64_t runs = (p.rows + run - 1) / run;
            const dim3 grid((unsigned)(runs + (p.K > 1 ? p.num_seqs : 0)), (unsigned)across);
            switch (p.K) {
                case 1: ssm_conv_bulk_kernel<IO, 1><<<grid, 128, 0, stream>>>(p, runs, run); break;
                case 2: ssm_conv_bulk_kernel<IO, 2><<<grid, 128, 0, stream>>>(p, runs, run); break;
                case 3: ssm_conv_bulk_kernel<IO, 3><<<grid, 128, 0, stream>>>(p, runs, run); break;
                default: ssm_conv_bulk_kernel<IO, 4><<<grid, 128, 0, stream>>>(p, runs, run); break;
            }
            return cudaGetLastError();
        }
    }
    return wide ? conv_launch<IO, V>(p, stream) : conv_launch<IO, 1>(p, stream);
}

// ------------------------------------------------------------------ token-sequential scan
// A CTA of four warps takes 16 columns of one head's state and walks the sequence.  A warp
// holds four columns; a column's d_state rows are dealt to eight lanes, NS to each, in
// registers, two rows to a packed instruction.  B, C, x, z and the gates of two batches of eight
// tokens (one, where d_state > 128 leaves no room) are fetched while the two before them are
// computed, as raw bits: widened at the load they were waited for there (133 us, then 207).  The
// eight lanes' partial readouts of a batch are summed by a reduce-scatter (seven shuffles for
// eight tokens), after which lane slice s owns token s.
// Bound by issue and latency: 2 x 1,001 f16 tokens of 24 heads of 64 columns x 128 rows take
// 139 us, 260 cycles a token, on SMs with four or eight warps each; there is no more parallelism
// than columns without cutting time.
constexpr int kBatch = 8, kCols = 16, kScanThreads = 128;

template <typename IO, int NS>
__global__ void __launch_bounds__(kScanThreads) ssm_scan_kernel(const SsmParams p) {
    constexpr int NP = 8 * NS, V = NS < 4 ? NS : 4, kTile = NS > 16 ? kBatch : 2 * kBatch, kXs = kTile * kCols / kScanThreads;
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

    F2 S[NS / 2];
#pragma unroll
    for (int i = 0; i < NS; i += 2) {
        auto at = [&](int j) { return p.state_in && live && state_at(j) < N ? p.state_in[sbase + (size_t)state_at(j) * P] : 0.f; };
        S[i / 2] = {at(i), at(i + 1)};
    }

    const IO *xs = static_cast<const IO *>(p.xs), *dt = static_cast<const IO *>(p.dt);
    const IO *z = static_cast<const IO *>(p.z);
    const float A = ssm_rate(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
    IO rb[LOADS], rx[kXs], rd, rz[kTile / kBatch];      // (widened where they are used: nothing waits for them in load)
    const IO none = IO(0.f);
    const int64_t yc = (int64_t)h * P + c0 + col;
    // Tile loads: value e of a thread is (token, B or C, row), x one (token, column), dt one token.
    auto load = [&](int64_t tb) {
#pragma unroll
        for (int e = 0; e < LOADS; ++e) {
            const int at = tid + e * kScanThreads, tk = at / (2 * NP), bc = (at / NP) & 1, i = at % NP;
            rb[e] = (tb + tk < t1 && i < N)
                        ? xs[(tb + tk) * p.ldx + (bc ? p.off_c : p.off_b) + (int64_t)g * p.bc_group + i]
                        : none;
        }
#pragma unroll
        for (int e = 0; e < kXs; ++e) {
            const int tk = (tid + e * kScanThreads) / kCols, c = tid % kCols;
            rx[e] = (tb + tk < t1 && c0 + c < P) ? xs[(tb + tk) * p.ldx + (int64_t)h * p.x_head + c0 + c] : none;
        }
        rd = (tid < kTile && tb + tid < t1) ? dt[(tb + tid) * p.ld_dt + h] : none;
#pragma unroll
        for (int e = 0; e < kTile / kBatch; ++e) {
            const int64_t t = tb + e * kBatch + slice;
            rz[e] = z && live && t < t1 ? z[t * p.ld_z + yc] : none;
        }
    };
    auto put = [&](int64_t tb, int buf) {      // tokens behind the sequence change nothing: d = 0, decay 1
#pragma unroll
        for (int e = 0; e < LOADS; ++e) {
            const int at = tid + e * kScanThreads;
            sb[buf][at / (2 * NP)][(at / NP) & 1][at % NP] = IoType<IO>::ld(&rb[e]);
        }
#pragma unroll
        for (int e = 0; e < kXs; ++e) sx[buf][(tid + e * kScanThreads) / kCols][tid % kCols] = IoType<IO>::ld(&rx[e]);
        if (tid < kTile) {
            const float d = tb + tid < t1 ? ssm_step(IoType<IO>::ld(&rd), bias, p.dt_min, p.dt_max) : 0.f;
            sg[buf][tid][0] = d;
            sg[buf][tid][1] = ssm_decay(A * d);
        }
    };
    load(t0);
    put(t0, 0);
    __syncthreads();
    int buf = 0;
    for (int64_t tb = t0; tb < t1; tb += kTile, buf ^= 1) {
        const bool more = tb + kTile < t1;
        IO zv[kTile / kBatch];
#pragma unroll
        for (int e = 0; e < kTile / kBatch; ++e) zv[e] = rz[e];
        if (more) load(tb + kTile);
#pragma unroll
        for (int e = 0; e < kTile / kBatch; ++e) {
            if (e > 0 && tb + e * kBatch >= t1) break;
            float y[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int tk = e * kBatch + k;
                const F2 a = both(sg[buf][tk][1]), dx = both(sg[buf][tk][0] * sx[buf][tk][col]);
                F2 sum = both(0.f);
#pragma unroll
                for (int i = 0; i < NS; i += V) {
                    const int at = (i / V) * (8 * V) + slice * V;
                    F2 b[V / 2], c[V / 2];
                    if constexpr (V == 4) {
                        const float4 bv = *reinterpret_cast<const float4 *>(&sb[buf][tk][0][at]);
                        const float4 cv = *reinterpret_cast<const float4 *>(&sb[buf][tk][1][at]);
                        b[0] = {bv.x, bv.y}; b[1] = {bv.z, bv.w}; c[0] = {cv.x, cv.y}; c[1] = {cv.z, cv.w};
                    } else {
                        const float2 bv = *reinterpret_cast<const float2 *>(&sb[buf][tk][0][at]);
                        const float2 cv = *reinterpret_cast<const float2 *>(&sb[buf][tk][1][at]);
                        b[0] = {bv.x, bv.y}; c[0] = {cv.x, cv.y};
                    }
#pragma unroll
                    for (int v = 0; v < V / 2; ++v) {
                        F2 &s = S[i / 2 + v];
                        s = fma2(a, s, mul2(dx, b[v]));
                        sum = fma2(c[v], s, sum);
                    }
                }
                y[k] = sum.x + sum.y;
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
            const int64_t t = tb + e * kBatch + slice;
            if (live && t < t1) {
                float out = fmaf(D, sx[buf][e * kBatch + slice][col], y[0]);
                if (z) out *= silu_gate<IO>(IoType<IO>::ld(&zv[e]));
                IoType<IO>::st(static_cast<IO *>(p.y) + t * (int64_t)p.heads * P + yc, out);
            }
        }
        if (more) put(tb + kTile, buf ^ 1);
        __syncthreads();
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NS; i += 2) {
        if (state_at(i) < N) p.state_out[sbase + (size_t)state_at(i) * P] = S[i / 2].x;
        if (state_at(i + 1) < N) p.state_out[sbase + (size_t)state_at(i + 1) * P] = S[i / 2].y;
    }
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
    const float a = ssm_decay(ssm_rate(p.A_log[h]) * d), D = p.D ? p.D[h] : 0.f;
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
        if (p.z) out *= silu_gate<IO>(IoType<IO>::ld(static_cast<const IO *>(p.z) + b * p.ld_z + yc));
        IoType<IO>::st(static_cast<IO *>(p.y) + b * (int64_t)hp + yc, out);
    }
}

// The same for states of up to kStreamState values, by a persistent CTA: a contiguous run of
// (row, head) units, whose states pass through a ring of kRing stages in shared memory by bulk
// copies in both directions.  The convolved B and C of a (row, group) are kept for all of its
// heads, and the next unit's inputs are loaded while this one is computed.  Two CTAs to an SM
// keep 128 KB of loads in flight.  Bound by reading and writing the states: 256 rows of 64 heads of
// 64 x 128 take 169 us (6.4 TB/s of a copy's 6.8); the call took 253 us with the kernel above, and takes
// 179 with this one.
constexpr int kStreamState = 8192, kRing = 3, kSlots = 3;

template <typename IO>
__global__ void __launch_bounds__(kDecThreads, 2) ssm_decode_stream_kernel(const SsmDecodeParams p, int64_t units) {
    using namespace tc;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sB[256], sC[256], sx[256];
    __shared__ __align__(16) float red[kDecThreads * 4];
    __shared__ uint64_t full[kRing];
    const int tid = threadIdx.x;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    const int count = (int)(u1 - u0);
    const int N = p.d_state, P = p.head_dim, Q = P / 4, RP = kDecThreads / Q, hpg = p.heads / p.groups;
    const int hp = p.heads * P, gn = p.groups * N, quad = tid % Q, r0 = tid / Q;
    const uint32_t bytes = (uint32_t)N * P * 4;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    auto state_of = [&](int64_t u) -> float * {      // null: a slot outside the pool
        const int64_t b = u / p.heads, e = p.slots ? (int64_t)p.slots[b] : b;
        return e < 0 || e >= p.pool_size ? nullptr : p.state + (e * p.heads + u % p.heads) * (int64_t)N * P;
    };
    auto fetch = [&](int i) {                        // (one thread) unit i's state into its stage
        const float *from = state_of(u0 + i);
        if (from == nullptr) {
            mbar_arrive(&full[i % kRing]);
            return;
        }
        mbar_arrive_expect_tx(&full[i % kRing], bytes);
        bulk_load(ring + (size_t)(i % kRing) * bytes, from, bytes, &full[i % kRing]);
    };

    // Inputs of the next unit, as they come: up to kSlots channels of [x | B | C] to a thread.
    IO raw[kSlots][4], w[kSlots][4], bias[kSlots], raw_dt;
    float A = 0.f, db = 0.f, D = 0.f;
    IoType<IO>::st(&raw_dt, 0.f);
    int have = 0;                                    // channels of this thread among them
    bool fresh = false;                              // the unit begins another (row, group)
    auto gather = [&](int64_t u) {
        const int64_t b = u / p.heads;
        const int h = (int)(u % p.heads), g = h / hpg;
        fresh = u == u0 || h % hpg == 0;
        const int64_t e = p.slots ? (int64_t)p.slots[b] : b;
        have = 0;
        raw_dt = static_cast<const IO *>(p.dt)[b * p.ld_dt + h];
        A = p.A_log[h];
        db = p.dt_bias ? p.dt_bias[h] : 0.f;
        D = p.D ? p.D[h] : 0.f;
        if (e < 0 || e >= p.pool_size) return;
        const IO *x = static_cast<const IO *>(p.x) + b * p.ld_x;
        const IO *conv = p.conv ? static_cast<const IO *>(p.conv) + e * (int64_t)(p.K - 1) * p.C : nullptr;
        const int n = fresh ? P + 2 * N : P;
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int i = tid + j * kDecThreads;
            if (i >= n) break;
            const int c = i < P ? h * P + i : i < P + N ? hp + g * N + i - P : hp + gn + g * N + i - P - N;
            raw[j][3] = x[c];
            if (p.w != nullptr) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {        // (the last tap stands last)
                    const int tap = k - (4 - p.K);
                    if (tap >= 0) w[j][k] = static_cast<const IO *>(p.w)[(int64_t)c * p.K + tap];
                    if (tap >= 0 && k < 3) raw[j][k] = conv[(int64_t)tap * p.C + c];
                }
                if (p.bias) bias[j] = static_cast<const IO *>(p.bias)[c];
            }
            have = j + 1;
        }
    };
    float d = 0.f, a = 0.f, skip = 0.f;
    auto settle = [&]() {                            // the gathered inputs into place
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            if (j >= have) break;
            const int i = tid + j * kDecThreads;
            float v = IoType<IO>::ld(&raw[j][3]);
            if (p.w != nullptr) {
                float acc = p.bias ? IoType<IO>::ld(&bias[j]) : 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k >= 4 - p.K) acc = fmaf(IoType<IO>::ld(&w[j][k]), IoType<IO>::ld(&raw[j][k]), acc);
                IO out;
                IoType<IO>::st(&out, p.silu ? silu_exact(acc) : acc);
                v = IoType<IO>::ld(&out);
            }
            (i < P ? sx[i] : i < P + N ? sB[i - P] : sC[i - P - N]) = v;
        }
        d = ssm_step(IoType<IO>::ld(&raw_dt), db, p.dt_min, p.dt_max);
        a = ssm_decay(ssm_rate(A) * d);
        skip = D;
    };

    __syncthreads();
    if (tid == 0)
        for (int i = 0; i < kRing - 1 && i < count; ++i) fetch(i);
    if (count > 0) {
        gather(u0);
        settle();
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
        const int64_t u = u0 + i, b = u / p.heads;
        const int h = (int)(u % p.heads);
        float *state = state_of(u);
        const bool live = state != nullptr;
        if (tid == 0 && i + kRing - 1 < count) {
            bulk_wait_read();                        // the stage's state has gone out
            fetch(i + kRing - 1);
        }
        if (i + 1 < count) gather(u + 1);
        const int64_t yc = (int64_t)h * P + tid;
        IO zr;                                       // (widened where it is used: nothing waits for it here)
        IoType<IO>::st(&zr, 0.f);
        if (p.z && tid < P) zr = static_cast<const IO *>(p.z)[b * p.ld_z + yc];
        const bool ok = mbar_wait(&full[i % kRing], (i / kRing) & 1, 4000000000LL);
        if (!ok) atomicOr(p.status, kDevTimeout);
        float4 *S = reinterpret_cast<float4 *>(ring + (size_t)(i % kRing) * bytes) + quad;
        if (live && ok && r0 < RP) {
            const float4 dx = make_float4(d * sx[4 * quad], d * sx[4 * quad + 1], d * sx[4 * quad + 2], d * sx[4 * quad + 3]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int n = r0; n < N; n += RP) {
                const float bn = sB[n], cn = sC[n];
                float4 v = S[(size_t)n * Q];
                v.x = fmaf(a, v.x, bn * dx.x); v.y = fmaf(a, v.y, bn * dx.y);
                v.z = fmaf(a, v.z, bn * dx.z); v.w = fmaf(a, v.w, bn * dx.w);
                acc.x = fmaf(cn, v.x, acc.x); acc.y = fmaf(cn, v.y, acc.y);
                acc.z = fmaf(cn, v.z, acc.z); acc.w = fmaf(cn, v.w, acc.w);
                S[(size_t)n * Q] = v;
            }
            reinterpret_cast<float4 *>(red)[tid] = acc;
        }
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            if (live && ok) bulk_store(state, ring + (size_t)(i % kRing) * bytes, bytes);
            else if (!live) atomicOr(p.status, kDevBadSlot);
            bulk_commit();
        }
        if (live && tid < P) {
            float out = 0.f;
            for (int r = 0; r < RP; ++r) out += red[r * P + tid];
            out = fmaf(skip, sx[tid], out);
            if (p.z) out *= silu_gate<IO>(IoType<IO>::ld(&zr));
            IoType<IO>::st(static_cast<IO *>(p.y) + b * (int64_t)hp + yc, out);
        }
        __syncthreads();                             // sx, sB, sC and red are free
        if (i + 1 < count) settle();
        __syncthreads();
    }
    if (tid == 0) bulk_wait_all();
}

// The conv states one token on, after the step has read them: rows move up, x comes last.
// (The step's CTAs all read their group's B and C taps, so it cannot move them itself.)  V channels
// to a thread: 16 bytes where the rows allow it (256 rows of 6,144 channels: 14.8 us singly,
// 6.6 us so).
template <typename IO, int V>
__global__ void __launch_bounds__(256) ssm_conv_shift_kernel(const SsmDecodeParams p) {
    using Vec = Pack<IO, V>;
    const int c = V * (blockIdx.y * 256 + threadIdx.x);
    const int64_t b = blockIdx.x;
    if (c >= p.C) return;
    const int64_t e = p.slots ? (int64_t)p.slots[b] : b;
    if (e < 0 || e >= p.pool_size) return;
    IO *conv = static_cast<IO *>(p.conv) + e * (int64_t)(p.K - 1) * p.C + c;
    auto row = [&](int j) { return reinterpret_cast<Vec *>(conv + (int64_t)j * p.C); };
    const Vec x = *reinterpret_cast<const Vec *>(static_cast<const IO *>(p.x) + b * p.ld_x + c);
    Vec a = x, d = x;
    if (p.K > 2) a = *row(1);
    if (p.K > 3) d = *row(2);
    if (p.K > 2) *row(0) = a;
    if (p.K > 3) *row(1) = d;
    *row(p.K - 2) = x;
}

template <typename IO>
cudaError_t decode_dispatch(const SsmDecodeParams &p, cudaStream_t stream) {
    const int64_t units = (int64_t)p.heads * p.batch;
    if (p.d_state * p.head_dim <= kStreamState) {
        const int smem = kRing * p.d_state * p.head_dim * 4;
        const cudaError_t e = cudaFuncSetAttribute(ssm_decode_stream_kernel<IO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kRing * kStreamState * 4);
        if (e != cudaSuccess) return e;
        const unsigned grid = (unsigned)(units < 2 * kSms ? units : 2 * kSms);
        ssm_decode_stream_kernel<IO><<<grid, kDecThreads, smem, stream>>>(p, units);
    } else {
        ssm_decode_kernel<IO><<<(unsigned)units, kDecThreads, 0, stream>>>(p);
    }
    if (p.w != nullptr && p.K > 1) {
        constexpr int V = 16 / sizeof(IO);
        const bool wide = p.C % V == 0 && p.ld_x % V == 0 && (reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.conv)) % 16 == 0;
        const dim3 grid((unsigned)p.batch, (unsigned)((p.C + 255) / 256)), few((unsigned)p.batch, (unsigned)((p.C / V + 255) / 256));
        if (wide) ssm_conv_shift_kernel<IO, V><<<few, 256, 0, stream>>>(p);
        else ssm_conv_shift_kernel<IO, 1><<<grid, 256, 0, stream>>>(p);
    }
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
