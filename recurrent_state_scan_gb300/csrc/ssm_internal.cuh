// ssm_internal.cuh -- what the state-space scan's translation units share.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// One call of the selective state-space scan (validated arguments).  `rows` of x, dt and z
// are token rows (t of sequence b at b * seqlen + t, or the packed index).
struct SsmParams {
    // The rows the scan reads: x of head h at xs + h * x_head, B of group g at
    // xs + off_b + g * bc_group, C at xs + off_c + g * bc_group, row stride ldx (elements).
    const void *xs;
    int64_t ldx;
    int32_t x_head, off_b, off_c, bc_group;
    const void *dt, *z;          // z may be null
    int64_t ld_dt, ld_z;
    const float *A_log, *dt_bias, *D;   // dt_bias, D may be null
    float dt_min, dt_max;
    const float *state_in;       // may be null (zeros); may alias state_out
    float *state_out;
    void *y;                     // [rows, H, P]
    const int32_t *cu_seqlens;   // may be null
    int64_t seqlen, rows;
    int32_t num_seqs, heads, groups, head_dim, d_state;
    int *status;
};

// The causal convolution of the mixed rows [x | B | C] before the scan, packed-aware:
// u [rows][..] in the layout SsmParams describes (ld_u, x_head, off_b, off_c, bc_group).
struct SsmConvParams {
    const void *x;
    int64_t ld_x;
    const void *w, *bias;        // [C][K], [C] or null
    const void *conv_in;         // [n][K - 1][C] or null (zeros)
    void *conv_out;              // [n][K - 1][C]
    void *u;
    int64_t ld_u;
    int32_t x_head, off_b, off_c, bc_group;
    const int32_t *cu_seqlens;
    int64_t seqlen, rows;
    int32_t num_seqs, heads, groups, head_dim, d_state;
    int32_t C, K, silu;          // K = 1 with a null w: a copy (rows re-laid for the scan)
    int *status;
};

struct SsmDecodeParams {
    const void *x, *dt, *z;
    int64_t ld_x, ld_dt, ld_z;
    const void *w, *bias;        // w null: x is used as it is
    void *conv;                  // [pool][K - 1][C], advanced in place
    const float *A_log, *dt_bias, *D;
    float dt_min, dt_max;
    float *state;                // [pool][H][N][P], advanced in place
    int64_t pool_size;
    const int32_t *slots;        // may be null: row b is entry b
    void *y;
    int32_t batch, heads, groups, head_dim, d_state, C, K, silu;
    int *status;
};

cudaError_t launch_ssm_conv(const SsmConvParams &p, gdn_dtype io, cudaStream_t stream);
cudaError_t launch_ssm_scan_simt(const SsmParams &p, gdn_dtype io, cudaStream_t stream);
// The tensor-core scan: its types and sizes, the rows it can read by TMA, its launches (and whether
// it runs in time segments), the bytes of its segments' states and items (16-byte aligned; 0:
// none), and the launch.
bool ssm_tc_shape_ok(gdn_dtype io, int head_dim, int d_state);
bool ssm_tc_rows_ok(const SsmParams &p);
int ssm_tc_launches(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int heads, int groups, int head_dim, bool *segments);
size_t ssm_tc_workspace(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int heads, int groups, int head_dim,
                        int d_state);
cudaError_t launch_ssm_tc(const SsmParams &p, void *workspace, cudaStream_t stream);
cudaError_t launch_ssm_decode(const SsmDecodeParams &p, gdn_dtype io, cudaStream_t stream);

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two fp32 operations in one instruction.
struct F2 {
    float x, y;
};
__device__ __forceinline__ uint64_t bits(F2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ F2 pair(uint64_t v) {
    F2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ F2 both(float a) { return {a, a}; }

// silu as the convolution stores it: the correctly scaled exponential and a true divide,
// so that its rounding to a 16-bit type does not hang on an approximation's last bits.
__device__ __forceinline__ float silu_exact(float v) { return v / (1.0f + expf(-v)); }
// silu of the gate z by e^-|z|, which neither overflows nor loses a gate far below zero.  An f32 output
// meets no other rounding, so there to fp32's own precision; a 16-bit one by the fast intrinsics, within
// 2^-16 of it.
template <typename IO> __device__ __forceinline__ float silu_gate(float v) {
    const float e = sizeof(IO) == 4 ? expf(-fabsf(v)) : __expf(-fabsf(v)), num = v < 0.0f ? e : 1.0f;
    return v * (sizeof(IO) == 4 ? num / (1.0f + e) : __fdividef(num, 1.0f + e));
}

// The step d = clamp(softplus(dt + dt_bias), dt_min, dt_max); a NaN stays one.
__device__ __forceinline__ float ssm_step(float dt, float bias, float lo, float hi) {
    const float d = softplus_f(dt + bias);
    return d < lo ? lo : d > hi ? hi : d;
}
// -e^{A_log}, held finite (and so that its product with log2 e is): a step of 0 then has a decay of 1, not a NaN,
// past A_log = 88 too.
__device__ __forceinline__ float ssm_rate(float A_log) {
    const float e = expf(A_log);
    return e > 0x1p126f ? -0x1p126f : -e;
}
// e^g.  A slow decay is multiplied in thousands of times, so its rounding has to be fair: expf alone
// drifts (2,000 tokens of e^-0.0003: 1.4e-5 off, 1.0e-6 so).  A fast one has to keep its own digits,
// which 1 + expm1f loses (e^-10 0.05% off, e^-17 and below nothing).
__device__ __forceinline__ float ssm_decay(float g) { return g > -0.5f ? 1.f + expm1f(g) : expf(g); }

}  // namespace gdn
