// diag_internal.cuh -- what the diagonal recurrence's translation units share: its arguments, its gates,
// the 8-bit codes, the sequences' edges among a warp's rows, and the walk over the tiles.
#pragma once

#include "ssm_internal.cuh"

namespace gdn {

constexpr int kDiagTile = 64;    // token rows of an item of the walk, and with codes between two kept states
constexpr int kDiagRows = 16;    // of one warp, and without codes between two kept states
constexpr int kDiagSlice = 64;   // channels of an item, and of a block of the 8-bit codes

// One call (validated arguments).  Token rows are those of the whole call: t of sequence b at
// b * seqlen + t, or the packed index.  Row strides in elements.
struct DiagParams {
    const void *x, *a, *b;
    bool has_b;                          // else the input gate is 1
    int64_t ld_x, ld_a, ld_b, ld_y;      // ld_y: y's and dy's rows
    const float *A_log, *a_bias, *b_bias;   // the biases may be null
    const float *state_in;               // may be null (zeros); may alias state_out
    float *state_out;
    void *y;
    const int32_t *cu_seqlens;           // may be null
    int64_t seqlen, rows;
    int32_t num_seqs, channels;
    int32_t wide;                        // bytes that every input row can be copied by: 16, a pair's, or 0: by the element
    bool pairs;                          // every output row can be written two channels at a time
    int *status;
    // What the forward pass keeps for the backward pass.
    float *kept;                         // h before rows, [.][slices * 64], or null: with codes before every 64th, else every 16th
    int8_t *codes;                       // [x | a | b][slice][rows, in whole tiles][64] or null
    uint8_t *steps;                      // [x | a | b][slice][rows, in whole tiles]
    // The backward pass.
    const void *dy;
    const float *dstate_out;             // may be null (zeros)
    void *dx, *da, *db;
    int64_t ld_dx, ld_da, ld_db;
    float *dA_log, *da_bias, *db_bias, *dstate_in;   // each may be null
    float *partial;                      // [tiles][3][channels]: a tile's sums of the parameters' gradients
    // The walk over the tiles (see DiagWalk).
    uint32_t *ticket;
    unsigned long long *words;           // [slice][tile][4][32]: what the tiles hand on
    float *table;                        // [5][slices * 64]: the channels' parameters (DiagLane), or null
    uint32_t magic, magic_shift;         // item / slices as (item * magic) >> magic_shift, for items below 2^31
    long long budget;                    // cycles that a wait for an earlier tile may take
};

struct DiagDecodeParams {
    const void *x, *a, *b;
    bool has_b;
    int64_t ld_x, ld_a, ld_b, ld_y;
    const float *A_log, *a_bias, *b_bias;
    float *state;                        // [pool][channels], in place
    int64_t pool_size;
    const int32_t *slots;                // may be null
    void *y;
    int32_t batch, channels;
    bool vec;                            // four channels at a time
    int *status;
};

int diag_slices(int channels);
int64_t diag_tiles(int64_t rows);
// Bytes of a walk's workspace (0: one tile a slice, nothing to hand on).
size_t diag_walk_bytes(int64_t rows, int channels);
void diag_walk_layout(DiagParams &p, void *workspace);
// Launches a walk's kernel behind its first one, as a dependent of it: its CTAs start while that one still runs, and
// DiagWalk::first waits for it.
template <typename Kernel>
cudaError_t diag_launch(Kernel kernel, unsigned grid, int threads, size_t shared, const DiagParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.table ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
// The walk's first kernel: clears the counter and the words and makes the table.
cudaError_t diag_begin(const DiagParams &p, cudaStream_t stream);
// CTAs of a walk: one for each item, up to `per_sm` on each of 152 SMs (a single row of tiles: always one for each).
unsigned diag_grid(const DiagParams &p, int per_sm);
template <typename IO> cudaError_t diag_prefill_by_kind(const DiagParams &p, int gate, int weighting, cudaStream_t s);
template <typename IO> cudaError_t diag_backward_by_kind(const DiagParams &p, int gate, int weighting, cudaStream_t s);
cudaError_t launch_diag_prefill(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream);
cudaError_t launch_diag_backward(const DiagParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream);
cudaError_t launch_diag_decode(const DiagDecodeParams &p, gdn_dtype io, int gate, int weighting, cudaStream_t stream);
cudaError_t launch_checkpoint_pack(gdn_dtype io, int64_t rows, int64_t channels, const void *x, int64_t ld, int8_t *codes,
                                   uint8_t *steps, cudaStream_t stream);
cudaError_t launch_checkpoint_unpack(gdn_dtype io, int64_t rows, int64_t channels, const int8_t *codes, const uint8_t *steps,
                                     void *y, int64_t ld, cudaStream_t stream);

#ifdef __CUDACC__
// ------------------------------------------------------------------ gates
// n = 1 - e^-G and alpha = e^-G for a decay's exponent G >= 0.  Slow decays are multiplied in thousands of times and weigh their
// input by n, so both have to keep their digits: up to 1/4 by G + G^2 r(G), r the Chebyshev fit of (1 - e^-G - G) / G^2
// (1.2e-8 of the result), alpha being its difference from 1 rounded once; beyond by the exponential, n within 4e-7 of itself.
// NEAR: no G is beyond.
struct DiagDecay {
    F2 n, alpha;
};
template <bool NEAR> __device__ __forceinline__ DiagDecay diag_decay(F2 G) {
    F2 r = fma2(G, both(0x1.f6d2c6p-8f), both(-0x1.548062p-5f));
    r = fma2(r, G, both(0x1.5552b2p-3f));
    r = fma2(r, G, both(-0x1.fffffep-2f));
    const F2 n = fma2(mul2(G, G), r, G), a = fma2(n, both(-1.f), both(1.f));
    if (NEAR) return {n, a};
    const F2 t = mul2(G, both(-kLog2e)), e = {ex2(t.x), ex2(t.y)}, far = fma2(e, both(-1.f), both(1.f));
    const bool x = G.x < 0.25f, y = G.y < 0.25f;
    return {{x ? n.x : far.x, y ? n.y : far.y}, {x ? a.x : e.x, y ? a.y : e.y}};
}
// sigmoid(v + bias); `nbias` is -bias log2 e.  e^-v beyond fp32's range gives 0.  (`k`: for v in units of a power of two, its
// multiple of -log2 e, by which the product rounds alike.)
__device__ __forceinline__ F2 diag_sigmoid(F2 v, F2 nbias, float k = -kLog2e) {
    const F2 t = fma2(v, both(k), nbias);
    const F2 d = add2({ex2(t.x), ex2(t.y)}, both(1.f));
    return {rcp(d.x), rcp(d.y)};
}
// e = e^-(v + bias), of which the gate is s = diag_opening(e), as diag_sigmoid has it, and 1 - s = e s, which keeps its digits however
// far the gate is open (as a difference from 1 it has lost half of them at v = 8, all at 16).  Where e has become infinite and s 0, the
// saturated product is 0 in place of 1: what it multiplies is 0 there.
__device__ __forceinline__ F2 diag_closing(F2 v, F2 nbias, float k = -kLog2e) {
    const F2 t = fma2(v, both(k), nbias);
    return {ex2(t.x), ex2(t.y)};
}
__device__ __forceinline__ F2 diag_opening(F2 e) {
    const F2 d = add2(e, both(1.f));
    return {rcp(d.x), rcp(d.y)};
}
__device__ __forceinline__ F2 diag_closed(F2 e, F2 s) {
    F2 r;
    asm("mul.sat.f32 %0, %1, %2;" : "=f"(r.x) : "f"(e.x), "f"(s.x));
    asm("mul.sat.f32 %0, %1, %2;" : "=f"(r.y) : "f"(e.y), "f"(s.y));
    return r;
}
// The sigmoid's negative, by the same steps.
__device__ __forceinline__ F2 diag_minus_sigmoid(F2 v, F2 nbias, float k = -kLog2e) {
    const F2 t = fma2(v, both(k), nbias);
    const F2 d = fma2({ex2(t.x), ex2(t.y)}, both(-1.f), both(-1.f));
    return {rcp(d.x), rcp(d.y)};
}
// softplus(z) = max(z, 0) + log(1 + e), e = e^-|z|.  log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by
// s + s^3 q(s^2), q the Chebyshev fit of the series of atanh (1.6e-8 of the result): digits are kept however
// small e is.
__device__ __forceinline__ F2 diag_softplus(F2 z) {
    const F2 e = {ex2(-kLog2e * fabsf(z.x)), ex2(-kLog2e * fabsf(z.y))}, d = add2(e, both(2.f));
    const F2 s = mul2(e, {rcp(d.x), rcp(d.y)}), q = mul2(s, s);
    F2 p = fma2(both(0x1.131faap-3f), q, both(0x1.211da0p-3f));
    p = fma2(p, q, both(0x1.99adb6p-3f));
    p = fma2(p, q, both(0x1.55554cp-2f));
    const F2 l = fma2(mul2(s, q), p, s);
    return fma2(l, both(2.f), {z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y});   // (a NaN stays one)
}

// The parameters of a lane's two channels.
struct DiagLane {
    F2 rate, ninverse, abias, nabias, nbbias;   // e^A_log, -1 / e^A_log (or 0), a_bias, -a_bias log2 e, -b_bias log2 e
};
// The input's weight, and for the backward pass and `norm` (sqrt(1 - alpha^2)) 1 / w, which counts as 0 where the weight is 0.
template <int WEIGHT> __device__ __forceinline__ F2 diag_weigh(F2 n) {
    if (WEIGHT == GDN_DIAG_COMPLEMENT) return n;
    if (WEIGHT == GDN_DIAG_PLAIN) return both(1.f);
    const F2 q = mul2(n, fma2(n, both(-1.f), both(2.f)));
    F2 w;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(w.x) : "f"(q.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(w.y) : "f"(q.y));
    return w;
}
__device__ __forceinline__ F2 diag_unweigh(F2 n) {
    const F2 q = mul2(n, fma2(n, both(-1.f), both(2.f)));
    F2 r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(q.x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(q.y));
    return {q.x < 0x1p-126f ? 0.f : r.x, q.y < 0x1p-126f ? 0.f : r.y};
}
// (`by`: for a in units of a power of two, which it then holds as a factor.)
template <int GATE> constexpr float kGateUnit = GATE == GDN_DIAG_SIGMOID ? -kLog2e : 1.f;
template <int GATE> __device__ __forceinline__ F2 diag_exponent(F2 a, const DiagLane &l, float by = kGateUnit<GATE>) {
    return mul2(l.rate, GATE == GDN_DIAG_SIGMOID ? diag_sigmoid(a, l.nabias, by) : diag_softplus(fma2(a, both(by), l.abias)));
}

__device__ __forceinline__ DiagLane diag_lane(const float *A_log, const float *a_bias, const float *b_bias, int c, int C) {
    DiagLane l{};
    const bool one = c < C, two = c + 1 < C;
    l.rate = {one ? -ssm_rate(A_log[c]) : 0.f, two ? -ssm_rate(A_log[c + 1]) : 0.f};
    // (Held finite for rates below the normal numbers, A_log < -87, whose products with the gate are below 2^-126 whatever it is.)
    l.ninverse = {l.rate.x != 0.f ? fmaxf(-1.f / l.rate.x, -0x1p127f) : 0.f, l.rate.y != 0.f ? fmaxf(-1.f / l.rate.y, -0x1p127f) : 0.f};
    if (a_bias) l.abias = {one ? a_bias[c] : 0.f, two ? a_bias[c + 1] : 0.f};
    F2 bb = both(0.f);
    if (b_bias) bb = {one ? b_bias[c] : 0.f, two ? b_bias[c + 1] : 0.f};
    l.nabias = mul2(l.abias, both(-kLog2e));
    l.nbbias = mul2(bb, both(-kLog2e));
    return l;
}
// The same as they lie in the walk's table, [5][slices * 64], or in a copy of a slice's part of it, [5][64].
__device__ __forceinline__ DiagLane diag_lane(const float *table, int row, int lane) {
    const float2 *t = reinterpret_cast<const float2 *>(table) + lane;
    row /= 2;
    const float2 v[5] = {t[0], t[row], t[2 * row], t[3 * row], t[4 * row]};
    return {{v[0].x, v[0].y}, {v[1].x, v[1].y}, {v[2].x, v[2].y}, {v[3].x, v[3].y}, {v[4].x, v[4].y}};
}
// From the walk's table, which its first kernel makes, or without one from the parameters themselves.
__device__ __forceinline__ DiagLane diag_lane(const DiagParams &p, int c, int slices) {
    if (p.table == nullptr) return diag_lane(p.A_log, p.a_bias, p.b_bias, c, p.channels);
    return diag_lane(p.table + (c & ~(kDiagSlice - 1)), slices * kDiagSlice, (c & (kDiagSlice - 1)) / 2);
}
// Whether no channel of a warp's can pass diag_decay's polynomial: a sigmoid gate's exponent is the rate at most.
template <int GATE> __device__ __forceinline__ bool diag_near(const DiagLane &l) {
    return GATE == GDN_DIAG_SIGMOID && __all_sync(~0u, l.rate.x < 0.25f && l.rate.y < 0.25f);
}

// ------------------------------------------------------------------ rows, two channels at a time
template <typename IO> struct IoBits {
    static constexpr bool kHalf = false;
};
template <> struct IoBits<__half> {
    static constexpr bool kHalf = true;
};
template <typename IO> struct Pair;      // a lane's two channels of one row, as they lie in memory
template <> struct Pair<float> {
    using Raw = float2;
    static __device__ __forceinline__ F2 wide(Raw v) { return {v.x, v.y}; }
    static __device__ __forceinline__ Raw narrow(F2 v) { return make_float2(v.x, v.y); }
};
template <> struct Pair<__nv_bfloat16> {
    using Raw = uint32_t;
    static __device__ __forceinline__ F2 wide(Raw v) { return {__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)}; }
    static __device__ __forceinline__ Raw narrow(F2 v) {
        Raw r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
        return r;
    }
};
template <> struct Pair<__half> {
    using Raw = uint32_t;
    static __device__ __forceinline__ F2 wide(Raw v) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&v);
        const float2 f = __half22float2(h);
        return {f.x, f.y};
    }
    static __device__ __forceinline__ Raw narrow(F2 v) {
        Raw r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
        return r;
    }
};

// The bits of -infinity and of infinity, over four bytes: rows that a call does not have are staged as x and b 0 and a -infinity,
// and are then the identity (alpha 1, input 0) without a test; an input gate that it does not have as b infinity.
template <typename IO> __device__ __forceinline__ uint32_t infinity_bits(bool negative) {
    const uint32_t b = sizeof(IO) == 4 ? 0x7f800000u : sizeof(IO) == 2 && IoBits<IO>::kHalf ? 0x7c007c00u : 0x7f807f80u;
    return negative ? b | (sizeof(IO) == 4 ? 0x80000000u : 0x80008000u) : b;
}

// Copies N rows of a slice to shared memory, [N][64], by one warp for itself, asynchronously where `wide` allows.  Rows from
// `rows` on become `outside`, channels behind C zeros.
template <typename IO, int N> struct Stager {
    static constexpr int kRow = kDiagSlice * sizeof(IO) / 16, kStep = 32 / kRow;    // 16-byte pieces of a row; rows at a time
    const IO *base;         // this lane's piece of row 0 of slice 0
    int64_t ld;
    __device__ __forceinline__ Stager(const void *from, int64_t ld_, int lane)
        : base(static_cast<const IO *>(from) + (lane / kRow) * ld_ + lane % kRow * (16 / (int)sizeof(IO))), ld(ld_) {}

    __device__ __forceinline__ void rows(IO *to, int r0, int rows, int c0, int C, int wide, uint32_t outside, int lane) const {
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to)) + lane * 16;
        const IO *from = base + (int64_t)r0 * ld + c0;
        if (wide == 16 && r0 + N <= rows && c0 + kDiagSlice <= C) {
#pragma unroll
            for (int i = 0; i < N / kStep; ++i) {
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst + i * 512), "l"(from) : "memory");
                from += kStep * ld;
            }
            return;
        }
        some_rows(to, from, r0, rows, c0, C, wide, outside, lane);
    }
    __device__ __noinline__ void some_rows(IO *to, const IO *from, int r0, int rows, int c0, int C, int wide, uint32_t outside, int lane) const {
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
        if (wide == 16) {
            const int left = (C - c0) * (int)sizeof(IO) - lane % kRow * 16, bytes = left < 0 ? 0 : left > 16 ? 16 : left;
            if (bytes == 0) from = base;
            for (int i = 0; i < N / kStep; ++i, from += bytes ? kStep * ld : 0) {
                if (r0 + lane / kRow + i * kStep < rows)
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst + lane * 16 + i * 512), "l"(from), "r"(bytes) : "memory");
                else
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + lane * 16 + i * 512), "r"(outside) : "memory");
            }
            return;
        }
        using Raw = typename Pair<IO>::Raw;
        const int c = c0 + 2 * lane;
        from = base - (lane / kRow) * ld - lane % kRow * (16 / (int)sizeof(IO)) + (int64_t)r0 * ld + c;
        for (int t = 0; t < N; ++t, from += ld) {
            IO *q = to + t * kDiagSlice + 2 * lane;
            if (r0 + t >= rows) {
                uint32_t *v = reinterpret_cast<uint32_t *>(q);
                v[0] = outside;
                if (sizeof(IO) == 4) v[1] = outside;
            } else if (wide == (int)sizeof(Raw) && c + 1 < C) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst + (t * 32 + lane) * (uint32_t)sizeof(Raw)), "l"(from), "n"(sizeof(Raw)) : "memory");
            } else {
                q[0] = c < C ? from[0] : IO(0.f);
                q[1] = c + 1 < C ? from[1] : IO(0.f);
            }
        }
    }
};
// Has 16 rows of a slice of two arrays (the second may be null) fetched into L2, by one warp: no address outside them.
template <typename IO>
__device__ __forceinline__ void fetch_rows(const void *one, int64_t ld_one, const void *two, int64_t ld_two, int r0, int rows, int c0, int C, int lane) {
    const int row = r0 + lane % 16;
    const IO *from = lane < 16 ? static_cast<const IO *>(one) + row * ld_one : static_cast<const IO *>(two) + row * ld_two;
    if (row >= rows || (lane >= 16 && two == nullptr)) return;
#pragma unroll
    for (int c = c0; c < c0 + kDiagSlice; c += 128 / (int)sizeof(IO))
        if (c < C) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + c));
}
// Fills N staged rows with four bytes.
template <typename IO, int N> __device__ __forceinline__ void fill_rows(IO *to, uint32_t bits, int lane) {
    for (int i = lane; i < N * kDiagSlice * (int)sizeof(IO) / 4; i += 32) reinterpret_cast<uint32_t *>(to)[i] = bits;
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
}
template <typename IO> __device__ __forceinline__ F2 staged(const IO *rows, int t, int lane) {
    return Pair<IO>::wide(reinterpret_cast<const typename Pair<IO>::Raw *>(rows)[t * 32 + lane]);
}
template <typename IO>
__device__ __forceinline__ void store_pair(IO *p, F2 v, int c, int C, bool fast) {
    if (fast) {
        *reinterpret_cast<typename Pair<IO>::Raw *>(p) = Pair<IO>::narrow(v);
    } else {
        if (c < C) IoType<IO>::st(p, v.x);
        if (c + 1 < C) IoType<IO>::st(p + 1, v.y);
    }
}
__device__ __forceinline__ F2 load_state(const float *p, int c, int C) {
    return {c < C ? p[c] : 0.f, c + 1 < C ? p[c + 1] : 0.f};
}
__device__ __forceinline__ void store_state(float *p, F2 v, int c, int C) {
    if (c < C) p[c] = v.x;
    if (c + 1 < C) p[c + 1] = v.y;
}

// ------------------------------------------------------------------ 8-bit codes
// The step of a block whose largest magnitude has the bits `most`: 2^(e - 133), e in [16, 254], the least
// power of two that keeps rint(most / step) at 127 or below; 255: the block holds an infinity or a NaN.
// (Adding 2^16 carries into the exponent from 255/128 of a power of two on.)
__device__ __forceinline__ uint32_t code_step(uint32_t most) {
    if (most >= 0x7f800000u) return 255u;
    const uint32_t e = (most + 0x10000u) >> 23;
    return e < 16u ? 16u : e > 254u ? 254u : e;
}
__device__ __forceinline__ float code_scale(uint32_t e) { return e == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((e - 6u) << 23); }
__device__ __forceinline__ float code_inverse(uint32_t e) { return e == 255u ? 0.f : __uint_as_float((260u - e) << 23); }
// Two codes as the bytes of an integer: v / step, exact, plus 1.5 x 2^23 is rounded to the nearest integer, whose low byte is the
// code.  Only at the step 254 could values next to fp32's largest reach 128.
__device__ __forceinline__ uint32_t code_bytes(F2 v, float inverse) {
    const F2 q = fma2(v, both(inverse), both(12582912.f));
    return __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040);
}
__device__ __forceinline__ F2 code_range(F2 v, float inverse) {
    const float top = 127.f / inverse;
    return {fminf(fmaxf(v.x, -top), top), fminf(fmaxf(v.y, -top), top)};
}
__device__ __forceinline__ uint32_t codes_of(F2 v, uint32_t e) {
    const float inverse = code_inverse(e);
    return code_bytes(e == 254u ? code_range(v, inverse) : v, inverse);
}
// The two codes in the low bytes of q as numbers: a byte plus 128 in the low byte of 2^23 is 2^23 + 128 more than the code.
__device__ __forceinline__ F2 code_values(uint32_t q) {
    q ^= 0x8080u;
    const F2 v = {__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7540)), __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7541))};
    return add2(v, both(-8388736.f));
}
__device__ __forceinline__ uint32_t magnitude(F2 v) {
    const uint32_t a = __float_as_uint(v.x) & 0x7fffffffu, b = __float_as_uint(v.y) & 0x7fffffffu;
    return a > b ? a : b;
}

// What the diagonal recurrence keeps of a gate's arguments: -infinity, which holds the gate shut, takes no part in its block's step
// and has the code -128, which no other value has.  Coded rows with an infinity among them are coded again so, by one warp: few are,
// and looking for them among the values cost the forward pass of 16,384 rows 20 us of 182 (the one test that is left: 5).
constexpr float kShutCode = -128.f;
template <typename IO> __device__ __noinline__ void code_gate_rows(const IO *rows, int8_t *codes, uint8_t *steps, int live, int lane) {
    __syncwarp();
    for (int t = 0; t < live && t < kDiagRows; ++t) {
        const F2 v = staged(rows, t, lane);
        const bool x = __float_as_uint(v.x) == 0xff800000u, y = __float_as_uint(v.y) == 0xff800000u;
        const uint32_t e = code_step(__reduce_max_sync(~0u, magnitude({x ? 0.f : v.x, y ? 0.f : v.y})));
        const uint32_t mask = (x ? 0xffu : 0u) | (y ? 0xff00u : 0u);
        reinterpret_cast<uint16_t *>(codes)[t * 32 + lane] = (uint16_t)((codes_of(v, e) & ~mask) | (mask & 0x8080u));
        if (lane == 0) steps[t] = (uint8_t)e;
    }
}
// Whether any of twice 16 rows of 64 codes is -128, by one warp.
__device__ __forceinline__ bool any_shut(const int8_t *a, const int8_t *b, int lane) {
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4 *>(i < 2 ? a : b)[i % 2 * 32 + lane];
        for (const uint32_t v : {q.x, q.y, q.z, q.w}) some |= v & ~((v & 0x7f7f7f7fu) + 0x7f7f7f7fu);       // (the sign bit alone)
    }
    return __any_sync(~0u, (some & 0x80808080u) != 0);
}

// 16 staged rows of 64 channels in 16 bits as codes [16][64] and steps [16], the first `live` of them, by one warp: half a row to
// a lane, 16 bytes at a time (its pieces in an order that starts at the row, so that eight lanes meet all banks).  Returns whether
// a row's largest magnitude is infinity.
template <typename IO> __device__ __forceinline__ bool code_rows(const IO *rows, int8_t *codes, uint8_t *steps, int live, int lane) {
    const int r = lane / 2, half = lane % 2;
    const uint4 *from = reinterpret_cast<const uint4 *>(rows) + r * 8 + half * 4;
    uint4 q[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = from[(i + r) % 4];
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(q[i].x & 0x7fff7fffu, q[i].y & 0x7fff7fffu), __vmaxu2(q[i].z & 0x7fff7fffu, q[i].w & 0x7fff7fffu)));
    }
    m = __vmaxu2(m, __shfl_xor_sync(~0u, m, 1));
    m = max(m & 0xffffu, m >> 16);
    const bool infinite = __any_sync(~0u, m == (infinity_bits<IO>(false) & 0xffffu));
    const uint32_t e = code_step(IoBits<IO>::kHalf ? __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) : m << 16);
    const float inverse = code_inverse(e);
    const bool top = __any_sync(~0u, e == 254u);
    uint2 c[4];
    auto two = [&](uint32_t a) {
        const F2 v = Pair<IO>::wide(a);
        return top ? codes_of(v, e) : code_bytes(v, inverse);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = make_uint2(__byte_perm(two(q[i].x), two(q[i].y), 0x5410), __byte_perm(two(q[i].z), two(q[i].w), 0x5410));
    // Back in order: piece i is at (i + r) % 4.
    if (r & 1) {
        const uint2 t = c[3];
        c[3] = c[2], c[2] = c[1], c[1] = c[0], c[0] = t;
    }
    if (r & 2) {
        const uint2 t = c[0], u = c[1];
        c[0] = c[2], c[1] = c[3], c[2] = t, c[3] = u;
    }
    if (r < live) {
        uint4 *to = reinterpret_cast<uint4 *>(codes) + r * 4 + half * 2;
        to[0] = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
        to[1] = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
        if (half == 0) steps[r] = (uint8_t)e;
    }
    return infinite;
}

// ------------------------------------------------------------------ the sequences among the rows
// Row where sequence n begins (n = num_seqs: the end of the rows).
__device__ __forceinline__ uint32_t seq_begin(const DiagParams &p, int n) {
    return p.cu_seqlens ? (uint32_t)p.cu_seqlens[n] : (uint32_t)(n * p.seqlen);
}
// Whether cu_seqlens is what it has to be, looked at by all threads of the CTA alike; if not, the call does nothing.
__device__ __forceinline__ bool offsets_ok(const DiagParams &p) {
    if (p.cu_seqlens == nullptr) return true;
    bool bad = false;
    for (int n = threadIdx.x; n <= p.num_seqs; n += blockDim.x) {
        const int v = p.cu_seqlens[n];
        bad |= n == 0 ? v != 0 : v < p.cu_seqlens[n - 1];
        if (n == p.num_seqs) bad |= v != p.rows;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(p.status, kDevBadCuSeqlens);
        return false;
    }
    return true;
}
// First n in [lo, num_seqs] whose sequence begins at `row` or behind it (num_seqs: none), by one warp.
__device__ __forceinline__ int first_at(const DiagParams &p, uint32_t row, int lo, int lane) {
    if (p.cu_seqlens == nullptr) {
        if (p.seqlen == 0) return row == 0 ? lo : p.num_seqs;
        const int64_t n = (row + p.seqlen - 1) / p.seqlen;
        return n > p.num_seqs ? p.num_seqs : (int)(n < lo ? lo : n);
    }
    int size = p.num_seqs - lo;             // candidates [lo, lo + size); behind them num_seqs, which always is
    while (size > 0) {
        const int step = (size + 31) / 32, at = lo + (lane + 1) * step - 1;
        const bool below = at < lo + size && (uint32_t)p.cu_seqlens[at] < row;
        const int n = __popc(__ballot_sync(~0u, below));
        lo += n * step;
        size = n == 32 ? 0 : step == 1 ? 0 : min(step - 1, size - n * step);
    }
    return lo < p.num_seqs ? lo : p.num_seqs;
}
// 32 sequences' first rows, one to a lane, kept while a warp walks along the rows.
struct EdgeWindow {
    int n0;
    uint32_t at;        // row where sequence n0 + lane begins (behind num_seqs: none)
    uint32_t lo, hi;    // no edge is at rows [lo, hi)
};
__device__ __forceinline__ EdgeWindow edge_window(const DiagParams &p, int n0, int lane) {
    return {n0, n0 + lane <= p.num_seqs ? seq_begin(p, n0 + lane) : 0xffffffffu, 0u, 0u};
}
// The edges between sequences at rows [w0, w0 + N], one bit each, and for each of them the first and the last
// n that begins there (in between: sequences without tokens).  `base`: the least n that counts; `behind`: how far
// ahead of the rows the window is laid (for a walk towards the first rows).
template <int N>
__device__ __forceinline__ uint32_t find_edges(const DiagParams &p, EdgeWindow &win, uint32_t w0, int base, int behind, int *first, int *last,
                                               int lane) {
    if (w0 >= win.lo && w0 + N < win.hi) return 0u;
    const uint32_t top = __shfl_sync(~0u, win.at, 31), bottom = __shfl_sync(~0u, win.at, 0);
    if (top < w0 || (behind > 0 && bottom >= w0 && win.n0 > base)) {
        const int n = first_at(p, w0, base, lane) - behind;
        win = edge_window(p, n > base ? n : base, lane);
    }
    uint32_t mask = 0;
    for (EdgeWindow v = win;;) {
        const uint32_t d = v.at - w0;
        const bool in = v.at >= w0 && d <= (uint32_t)N;
        if (__any_sync(~0u, in)) {
            const uint32_t bit = in ? 1u << d : 0u;
            const uint32_t before = __shfl_up_sync(~0u, bit, 1), after = __shfl_down_sync(~0u, bit, 1);
            if (in && !(mask & bit) && (lane == 0 || before != bit)) first[d] = v.n0 + lane;
            if (in && (lane == 31 || after != bit)) last[d] = v.n0 + lane;
            mask |= __reduce_or_sync(~0u, bit);
        }
        if (__shfl_sync(~0u, v.at, 31) > w0 + N) break;        // (none behind num_seqs: 2^32 - 1)
        v = edge_window(p, v.n0 + 32, lane);
    }
    if (mask == 0 && __shfl_sync(~0u, win.at, 31) > w0 + N) {
        win.lo = __reduce_max_sync(~0u, win.at < w0 ? win.at + 1 : 0u);
        if (__shfl_sync(~0u, win.at, 0) >= w0 && win.n0 > base) win.lo = w0;
        win.hi = __reduce_min_sync(~0u, win.at > w0 + N ? win.at : 0xffffffffu);
    }
    __syncwarp();
    return mask;
}

// ------------------------------------------------------------------ maps
// A stretch of tokens as the map h -> (hi + lo) h + H: the product of its decays in two fp32 numbers, because the
// chain of these maps over a long sequence has to keep slow decays (hi alone drifts: 65,536 equal tokens of
// 1 - 3e-5 by up to 2e-3) as well as the digits of fast ones.  hi = -1 marks a stretch that holds an edge, the
// same for all lanes: nothing of what came before is left behind it, an infinity or a NaN neither.  In the forward pass hi is 0 only
// where a token's decay is: it is held at 2^-149 where only the product has become 0, so that an infinite h stays infinite over
// the stretch as it does token by token.
constexpr float kLeast = 0x1p-149f;
struct DiagProduct {
    F2 hi, lo;
};
__device__ __forceinline__ DiagProduct diag_product(F2 sum_G, bool edge) {
    const DiagDecay d = diag_decay<false>(sum_G);
    DiagProduct o;
    // Where 1 - n was rounded, what that lost; a far decay is hi itself.
    const F2 lost = add2(fma2(d.alpha, both(-1.f), both(1.f)), {-d.n.x, -d.n.y});
    o.hi = edge ? both(-1.f) : d.alpha;
    o.lo = {sum_G.x < 0.25f ? lost.x : 0.f, sum_G.y < 0.25f ? lost.y : 0.f};
    return o;
}
__device__ __forceinline__ F2 diag_apply(DiagProduct p, F2 H, F2 h) {
    const F2 r = fma2(p.hi, h, fma2(p.lo, h, H)), far = fma2(p.hi, h, H);       // (lo times an infinite h has a sign of its own, or is NaN)
    const bool edge = p.hi.x < 0.f;
    return {edge ? H.x : isinf(h.x) ? far.x : r.x, edge ? H.y : isinf(h.y) ? far.y : r.y};
}
__device__ __forceinline__ DiagProduct diag_join(DiagProduct p, DiagProduct q) {
    DiagProduct o;
    o.hi = mul2(p.hi, q.hi);
    const F2 lost = fma2(p.hi, q.hi, {-o.hi.x, -o.hi.y});
    o.lo = fma2(p.hi, q.lo, fma2(p.lo, q.hi, lost));
    if (o.hi.x == 0.f && p.hi.x != 0.f && q.hi.x != 0.f) o.hi.x = kLeast;
    if (o.hi.y == 0.f && p.hi.y != 0.f && q.hi.y != 0.f) o.hi.y = kLeast;
    if (p.hi.x < 0.f || q.hi.x < 0.f) o.hi = both(-1.f);
    return o;
}
// Maps in shared memory, one to a lane.
struct DiagMaps {
    float4 product[32];
    float2 shift[32];
};
__device__ __forceinline__ DiagProduct get_product(const DiagMaps &m, int lane) {
    const float4 v = m.product[lane];
    return {{v.x, v.y}, {v.z, v.w}};
}
__device__ __forceinline__ F2 get_pair(const float2 *v, int lane) { return {v[lane].x, v[lane].y}; }
__device__ __forceinline__ void put_map(DiagMaps &m, int lane, DiagProduct p, F2 H) {
    m.product[lane] = make_float4(p.hi.x, p.hi.y, p.lo.x, p.lo.y);
    m.shift[lane] = make_float2(H.x, H.y);
}

// ------------------------------------------------------------------ the walk over the tiles
// Barriers between the warps that take rows and the one that hands maps on.
template <int THREADS> __device__ __forceinline__ void side_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory"); }
template <int THREADS> __device__ __forceinline__ void side_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory"); }

// CTAs take (tile, slice) items off one counter, tile by tile in the order of the walk.  An item hands on its map as soon as it
// has it, and what is behind it (h after the tile, G before it) once it knows what came in: that is found from the nearest
// earlier item that has handed on the latter, and the maps between, applied in the order of the rows: the same arithmetic from
// whichever item it starts, so results do not depend on timing.  The earliest unfinished item never waits, and its CTA is
// running, so every wait ends.
// What is handed on are 64-bit words, two channels each, that say themselves whether they are there (kNone: not yet), so that
// neither side needs a fence: with flags and release stores an item cost its CTA 8,500 cycles, so 3,000.
constexpr unsigned long long kNone = ~0ull;
struct DiagWalk {
    const DiagParams &p;
    int tiles, slices, lane;

    __device__ __forceinline__ uint32_t items() const { return (uint32_t)tiles * (uint32_t)slices; }
    __device__ __forceinline__ int tile_of(uint32_t item) const { return (int)((uint64_t)item * p.magic >> p.magic_shift); }
    // The next item: only CTAs that run hold any.  (A single row of tiles has nothing to wait for: an item for each CTA.)
    __device__ __forceinline__ uint32_t ticket() const { return tiles > 1 ? atomicAdd(p.ticket, 1u) : items(); }
    // For the walk's first kernel to end; every thread, before it ends itself too: what comes behind the call waits for this kernel
    // alone, and may have the workspace for its own.
    static __device__ __forceinline__ void wait_for_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
    __device__ __forceinline__ uint32_t first(uint32_t &shared) const {
        wait_for_first();
        if (threadIdx.x == 0) shared = tiles > 1 ? atomicAdd(p.ticket, 1u) : blockIdx.x;
        __syncthreads();
        const uint32_t item = shared;
        __syncthreads();
        return item;
    }
    __device__ __forceinline__ unsigned long long *at(int j, int slice) const { return p.words + ((int64_t)slice * tiles + j) * 128 + lane; }
    static __device__ __forceinline__ void put(unsigned long long *to, F2 v) {
        unsigned long long w = bits(v);
        if (w == kNone) w = 0x7fffffff7fffffffull;          // (a NaN like any other)
        asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(to), "l"(w) : "memory");
    }
    static __device__ __forceinline__ unsigned long long get(const unsigned long long *from) {
        unsigned long long w;
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(from) : "memory");
        return w;
    }
    __device__ __forceinline__ void hand_on_map(int j, int slice, DiagProduct m, F2 H) const {
        unsigned long long *to = at(j, slice);
        put(to, m.hi);
        put(to + 32, m.lo);
        put(to + 64, H);
    }
    __device__ __forceinline__ void hand_on(int j, int slice, F2 h) const { put(at(j, slice) + 96, h); }
    // What comes in to the j-th tile of a slice, by one warp.  A wait that runs out is reported, and takes 0.
    __device__ __forceinline__ F2 come_in(int j, int slice) const {
        if (j == 0) return both(0.f);
        constexpr int D = 4;                                // tiles back (3 to 12 tried: the traffic of more costs what they find)
        const unsigned long long *from = at(j, slice);
        unsigned long long hi[D], lo[D], H[D], after[D];
        int maps;
        const long long t0 = clock64();
        for (;;) {
#pragma unroll
            for (int q = 0; q < D; ++q) {
                const unsigned long long *w = from - (q + 1) * 128;
                const bool is = j > q;                      // (before the first tile: 0)
                after[q] = is ? get(w + 96) : 0ull;
                hi[q] = is ? get(w) : 0ull;
                lo[q] = is ? get(w + 32) : 0ull;
                H[q] = is ? get(w + 64) : 0ull;
            }
            uint32_t done = 0, some = 0;
#pragma unroll
            for (int q = 0; q < D; ++q) {
                done |= (uint32_t)__all_sync(~0u, after[q] != kNone) << q;
                some |= (uint32_t)__all_sync(~0u, hi[q] != kNone && lo[q] != kNone && H[q] != kNone) << q;
            }
            maps = __ffs(done) - 1;
            if (done != 0 && (~some & ((1u << maps) - 1)) == 0) break;
            if (__any_sync(~0u, clock64() - t0 > p.budget)) {
                if (lane == 0) atomicOr(p.status, kDevTimeout);
                return both(0.f);
            }
        }
        F2 h = both(0.f);
#pragma unroll
        for (int q = D - 1; q >= 0; --q) {
            if (q == maps) h = pair(after[q]);
            if (q < maps) h = diag_apply({pair(hi[q]), pair(lo[q])}, pair(H[q]), h);
        }
        return h;
    }
};
#endif  // __CUDACC__

}  // namespace gdn
