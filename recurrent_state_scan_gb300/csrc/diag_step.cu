// diag_step.cu -- single tokens of the diagonal recurrence, and rows as 8-bit codes.
#include "diag_internal.cuh"

namespace gdn {
namespace {

// One token per row: h = alpha h + w i x in place, y = h rounded.  Bound by the state's and the rows' bytes (16 a
// channel in 16 bits) and, at the sizes of a batch of requests, by latency: 256 rows of 4,096 channels take 7.8 us on an idle GPU,
// 2.5 by their bytes.  A thread takes four channels, and rows of a large batch in turn with one set of parameters.
template <typename IO, int GATE, int WEIGHT, bool VEC>
__global__ void __launch_bounds__(128) diag_decode_kernel(const __grid_constant__ DiagDecodeParams p) {
    constexpr int N = VEC ? 2 : 1;          // pairs of channels
    const int64_t C = p.channels, c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 2 * N;
    if (c >= C) return;
    DiagLane l[N];
#pragma unroll
    for (int k = 0; k < N; ++k) l[k] = diag_lane(p.A_log, p.a_bias, p.b_bias, (int)c + 2 * k, (int)C);
    for (int64_t row = blockIdx.y; row < p.batch; row += gridDim.y) {
        const int64_t e = p.slots ? p.slots[row] : row;
        if (e < 0 || e >= p.pool_size) {
            if (c == 0) atomicOr(p.status, kDevBadSlot);
            continue;
        }
        float *state = p.state + e * C + c;
        const IO *x = (const IO *)p.x + row * p.ld_x + c, *a = (const IO *)p.a + row * p.ld_a + c;
        const IO *b = (const IO *)p.b + row * p.ld_b + c;
        IO *y = (IO *)p.y + row * p.ld_y + c;
        F2 xv[N], av[N], bv[N], h[N];
        if (VEC) {
            using Raw = typename Pair<IO>::Raw;
            struct __align__(2 * sizeof(Raw)) Two {
                Raw v[2];
            };
            const Two rx = *reinterpret_cast<const Two *>(x), ra = *reinterpret_cast<const Two *>(a);
            Two rb{};
            if (p.has_b) rb = *reinterpret_cast<const Two *>(b);
            const float4 s = *reinterpret_cast<const float4 *>(state);
            h[0] = {s.x, s.y};
            h[N - 1] = {s.z, s.w};
#pragma unroll
            for (int k = 0; k < N; ++k) {
                xv[k] = Pair<IO>::wide(rx.v[k]);
                av[k] = Pair<IO>::wide(ra.v[k]);
                bv[k] = Pair<IO>::wide(rb.v[k]);
            }
        } else {
            const bool two = c + 1 < C;
            xv[0] = {IoType<IO>::ld(x), two ? IoType<IO>::ld(x + 1) : 0.f};
            av[0] = {IoType<IO>::ld(a), two ? IoType<IO>::ld(a + 1) : 0.f};
            bv[0] = both(0.f);
            if (p.has_b) bv[0] = {IoType<IO>::ld(b), two ? IoType<IO>::ld(b + 1) : 0.f};
            h[0] = {state[0], two ? state[1] : 0.f};
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const DiagDecay d = diag_decay<false>(diag_exponent<GATE>(av[k], l[k]));
            F2 v = p.has_b ? mul2(diag_sigmoid(bv[k], l[k].nbbias), xv[k]) : xv[k];
            v = WEIGHT == GDN_DIAG_PLAIN ? v : mul2(diag_weigh<WEIGHT>(d.n), v);
            h[k] = fma2(d.alpha, h[k], v);
        }
        if (VEC) {
            *reinterpret_cast<float4 *>(state) = make_float4(h[0].x, h[0].y, h[N - 1].x, h[N - 1].y);
            typename Pair<IO>::Raw r[2] = {Pair<IO>::narrow(h[0]), Pair<IO>::narrow(h[N - 1])};
            if (sizeof(IO) == 4) {
                *reinterpret_cast<float4 *>(y) = make_float4(h[0].x, h[0].y, h[N - 1].x, h[N - 1].y);
            } else {
                *reinterpret_cast<uint2 *>(y) = *reinterpret_cast<const uint2 *>(r);
            }
        } else {
            state[0] = h[0].x;
            IoType<IO>::st(y, h[0].x);
            if (c + 1 < C) {
                state[1] = h[0].y;
                IoType<IO>::st(y + 1, h[0].y);
            }
        }
    }
}

template <typename IO, int GATE, int WEIGHT> cudaError_t launch(const DiagDecodeParams &p, cudaStream_t stream) {
    const int64_t per = 128 * (p.vec ? 4 : 2), blocks = (p.channels + per - 1) / per;
    int64_t rows = (152 * 16 + blocks - 1) / blocks;
    if (rows > p.batch) rows = p.batch;
    const dim3 grid((unsigned)blocks, (unsigned)rows);
    if (p.vec) diag_decode_kernel<IO, GATE, WEIGHT, true><<<grid, 128, 0, stream>>>(p);
    else diag_decode_kernel<IO, GATE, WEIGHT, false><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename IO> cudaError_t by_kind(const DiagDecodeParams &p, int gate, int weighting, cudaStream_t s) {
    if (gate == GDN_DIAG_SOFTPLUS)
        return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_NORM>(p, s)
               : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_COMPLEMENT>(p, s)
                                                  : launch<IO, GDN_DIAG_SOFTPLUS, GDN_DIAG_PLAIN>(p, s);
    return weighting == GDN_DIAG_NORM         ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_NORM>(p, s)
           : weighting == GDN_DIAG_COMPLEMENT ? launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_COMPLEMENT>(p, s)
                                              : launch<IO, GDN_DIAG_SIGMOID, GDN_DIAG_PLAIN>(p, s);
}

// ------------------------------------------------------------------ 8-bit codes
// By eight channels: 16 bytes of 16-bit rows (32 of fp32) to a lane, eight lanes to a block, R rows of four blocks to a warp, so
// that R loads are on their way together; codes go out eight to a lane.  Bound by memory: 16,384 bf16 rows of 4,096 channels are
// packed in 38 us and read back in 29 (a value to a thread: 118 and 102), 30 each by their bytes.
constexpr int R = 4;
template <typename IO> struct Eight {
    F2 v[4];
    static __device__ __forceinline__ Eight load(const IO *p) {
        Eight e;
        if (sizeof(IO) == 4) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
            e.v[0] = {a.x, a.y}, e.v[1] = {a.z, a.w}, e.v[2] = {b.x, b.y}, e.v[3] = {b.z, b.w};
        } else {
            const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p));
            const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) e.v[i] = Pair<IO>::wide(*reinterpret_cast<const typename Pair<IO>::Raw *>(&r[i]));
        }
        return e;
    }
    __device__ __forceinline__ void store(IO *p) const {
        if (sizeof(IO) == 4) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        } else {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const typename Pair<IO>::Raw n = Pair<IO>::narrow(v[i]);
                r[i] = *reinterpret_cast<const uint32_t *>(&n);
            }
            *reinterpret_cast<uint4 *>(p) = make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
};

template <typename IO>
__global__ void __launch_bounds__(256) pack_wide_kernel(int64_t rows, int C, const IO *x, int64_t ld, int8_t *codes, uint8_t *steps) {
    const int lane = threadIdx.x % 32, c = (blockIdx.x * 32 + lane) * 8, blocks = (C + kDiagSlice - 1) / kDiagSlice;
    const int64_t r0 = ((int64_t)blockIdx.y * 8 + threadIdx.x / 32) * R;
    const bool in = c < C;
    Eight<IO> e[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        e[r] = Eight<IO>{};
        if (in && r0 + r < rows) e[r] = Eight<IO>::load(x + (r0 + r) * ld + c);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, magnitude(e[r].v[i]));
        m = max(m, __shfl_xor_sync(~0u, m, 1));
        m = max(m, __shfl_xor_sync(~0u, m, 2));
        m = max(m, __shfl_xor_sync(~0u, m, 4));
        const uint32_t s = code_step(m);
        if (!in || r0 + r >= rows) continue;
        const uint32_t a = codes_of(e[r].v[0], s), b = codes_of(e[r].v[1], s), d = codes_of(e[r].v[2], s), f = codes_of(e[r].v[3], s);
        *reinterpret_cast<uint2 *>(codes + (r0 + r) * C + c) = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(d, f, 0x5410));
        if (lane % 8 == 0) steps[(r0 + r) * blocks + c / kDiagSlice] = (uint8_t)s;
    }
}

// Any width and address: a warp takes one block of one row, two channels to a lane.
template <typename IO>
__global__ void __launch_bounds__(256) pack_kernel(int64_t rows, int64_t C, const IO *x, int64_t ld, int8_t *codes, uint8_t *steps) {
    const int lane = threadIdx.x % 32;
    const int64_t blocks = (C + kDiagSlice - 1) / kDiagSlice, all = rows * blocks, warps = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < all; i += warps) {
        const int64_t row = i / blocks, k = i - row * blocks, c = k * kDiagSlice + 2 * lane;
        const IO *p = x + row * ld + c;
        const F2 v = {c < C ? IoType<IO>::ld(p) : 0.f, c + 1 < C ? IoType<IO>::ld(p + 1) : 0.f};
        const uint32_t e = code_step(__reduce_max_sync(~0u, magnitude(v)));
        const uint32_t q = codes_of(v, e);
        if (c < C) codes[row * C + c] = (int8_t)(q & 255);
        if (c + 1 < C) codes[row * C + c + 1] = (int8_t)(q >> 8);
        if (lane == 0) steps[i] = (uint8_t)e;
    }
}

// The value in the type that it is read back in: f16's range is the only one that a code can pass.
template <typename IO> __device__ __forceinline__ float held(float v) { return v; }
template <> __device__ __forceinline__ float held<__half>(float v) { return v > 65504.f ? 65504.f : v < -65504.f ? -65504.f : v; }

template <typename IO>
__global__ void __launch_bounds__(256) unpack_wide_kernel(int64_t rows, int C, const int8_t *codes, const uint8_t *steps, IO *y, int64_t ld) {
    const int lane = threadIdx.x % 32, c = (blockIdx.x * 32 + lane) * 8, blocks = (C + kDiagSlice - 1) / kDiagSlice;
    const int64_t r0 = ((int64_t)blockIdx.y * 8 + threadIdx.x / 32) * R;
    if (c >= C) return;
    uint2 q[R];
    uint32_t s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        q[r] = make_uint2(0, 0);
        s[r] = 16;
        if (r0 + r < rows) {
            q[r] = __ldcs(reinterpret_cast<const uint2 *>(codes + (r0 + r) * C + c));
            s[r] = steps[(r0 + r) * blocks + c / kDiagSlice];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r0 + r >= rows) break;
        const F2 step = both(code_scale(s[r]));
        Eight<IO> e;
        e.v[0] = mul2(code_values(q[r].x & 0xffff), step);
        e.v[1] = mul2(code_values(q[r].x >> 16), step);
        e.v[2] = mul2(code_values(q[r].y & 0xffff), step);
        e.v[3] = mul2(code_values(q[r].y >> 16), step);
#pragma unroll
        for (int i = 0; i < 4; ++i) e.v[i] = {held<IO>(e.v[i].x), held<IO>(e.v[i].y)};
        e.store(y + (r0 + r) * ld + c);
    }
}

template <typename IO>
__global__ void __launch_bounds__(256) unpack_kernel(int64_t rows, int64_t C, const int8_t *codes, const uint8_t *steps, IO *y, int64_t ld) {
    const int lane = threadIdx.x % 32;
    const int64_t blocks = (C + kDiagSlice - 1) / kDiagSlice, all = rows * blocks, warps = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < all; i += warps) {
        const int64_t row = i / blocks, k = i - row * blocks, c = k * kDiagSlice + 2 * lane;
        const float s = code_scale(steps[i]);
        IO *p = y + row * ld + c;
        if (c < C) IoType<IO>::st(p, held<IO>(s * codes[row * C + c]));
        if (c + 1 < C) IoType<IO>::st(p + 1, held<IO>(s * codes[row * C + c + 1]));
    }
}

unsigned code_blocks(int64_t rows, int64_t C) {
    const int64_t n = (rows * ((C + kDiagSlice - 1) / kDiagSlice) + 7) / 8, most = 152 * 8 * 4;
    return (unsigned)(n < most ? n : most);
}

}  // namespace

cudaError_t launch_diag_decode(const DiagDecodeParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream) {
    switch (io) {
        case GDN_F32: return by_kind<float>(p, gate, weighting, stream);
        case GDN_BF16: return by_kind<__nv_bfloat16>(p, gate, weighting, stream);
        default: return by_kind<__half>(p, gate, weighting, stream);
    }
}

// Whether rows are taken by eight channels: widths, strides and addresses have to allow it, and a grid's second extent the rows.
bool code_wide(int64_t rows, int64_t C, const void *x, int64_t ld, const void *codes) {
    return C % 8 == 0 && C <= INT32_MAX - 256 && ld % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 8 == 0 &&
           (rows + 8 * R - 1) / (8 * R) <= 65535;
}
dim3 code_grid(int64_t rows, int64_t C) { return dim3((unsigned)((C + 255) / 256), (unsigned)((rows + 8 * R - 1) / (8 * R))); }

template <typename IO>
void pack(int64_t rows, int64_t C, const void *x, int64_t ld, int8_t *codes, uint8_t *steps, bool wide, cudaStream_t stream) {
    if (wide) pack_wide_kernel<IO><<<code_grid(rows, C), 256, 0, stream>>>(rows, (int)C, (const IO *)x, ld, codes, steps);
    else pack_kernel<IO><<<code_blocks(rows, C), 256, 0, stream>>>(rows, C, (const IO *)x, ld, codes, steps);
}
template <typename IO>
void unpack(int64_t rows, int64_t C, const int8_t *codes, const uint8_t *steps, void *y, int64_t ld, bool wide, cudaStream_t stream) {
    if (wide) unpack_wide_kernel<IO><<<code_grid(rows, C), 256, 0, stream>>>(rows, (int)C, codes, steps, (IO *)y, ld);
    else unpack_kernel<IO><<<code_blocks(rows, C), 256, 0, stream>>>(rows, C, codes, steps, (IO *)y, ld);
}

cudaError_t launch_checkpoint_pack(gdn_dtype io, int64_t rows, int64_t C, const void *x, int64_t ld, int8_t *codes, uint8_t *steps,
                                   cudaStream_t stream) {
    const bool wide = code_wide(rows, C, x, ld, codes);
    switch (io) {
        case GDN_F32: pack<float>(rows, C, x, ld, codes, steps, wide, stream); break;
        case GDN_BF16: pack<__nv_bfloat16>(rows, C, x, ld, codes, steps, wide, stream); break;
        default: pack<__half>(rows, C, x, ld, codes, steps, wide, stream);
    }
    return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(gdn_dtype io, int64_t rows, int64_t C, const int8_t *codes, const uint8_t *steps, void *y, int64_t ld,
                                     cudaStream_t stream) {
    const bool wide = code_wide(rows, C, y, ld, codes);
    switch (io) {
        case GDN_F32: unpack<float>(rows, C, codes, steps, y, ld, wide, stream); break;
        case GDN_BF16: unpack<__nv_bfloat16>(rows, C, codes, steps, y, ld, wide, stream); break;
        default: unpack<__half>(rows, C, codes, steps, y, ld, wide, stream);
    }
    return cudaGetLastError();
}

}  // namespace gdn
