// ssm_api.cu -- gdn_ssm_prefill and gdn_ssm_decode: argument checks and dispatch.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "ssm_internal.cuh"

namespace gdn {
namespace {

gdn_status fail(gdn_status status, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return report_error(status, msg);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a != nullptr && b != nullptr && a0 < b0 + nb && b0 < a0 + na;
}

// What the checks work out on the way.
struct Geometry {
    size_t es;
    int64_t rows, C, hp, ld_x, ld_dt, ld_z;
    size_t conv_bytes;   // of one conv state entry
};

gdn_status check(const gdn_ssm_shape *s, const gdn_ssm_params *q, bool varlen, Geometry &g) {
    if (s == nullptr || q == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape or params is NULL");
    if (s->io_dtype != GDN_F32 && s->io_dtype != GDN_BF16 && s->io_dtype != GDN_F16)
        return fail(GDN_ERR_INVALID_ARG, "io_dtype %d is not F32/BF16/F16", s->io_dtype);
    if (s->seqlen < 0 || s->num_seqs < 0 || s->batch < 0)
        return fail(GDN_ERR_INVALID_ARG, "batch, seqlen and num_seqs must be >= 0");
    if (varlen ? s->batch != 1 : s->batch != s->num_seqs)
        return fail(GDN_ERR_INVALID_ARG, "batch must be 1 with cu_seqlens, and equal num_seqs without (batch %d, num_seqs %d)",
                    s->batch, s->num_seqs);
    if (s->heads <= 0 || s->groups <= 0 || s->heads % s->groups != 0)
        return fail(GDN_ERR_INVALID_ARG, "heads (%d) must be a positive multiple of groups (%d)", s->heads, s->groups);
    if (s->head_dim <= 0 || s->d_state <= 0)
        return fail(GDN_ERR_INVALID_ARG, "head_dim (%d) and d_state (%d) must be positive", s->head_dim, s->d_state);
    if (s->head_dim > 256 || s->head_dim % 4 != 0 || s->d_state > 256 || s->heads > 65535)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim %d (a multiple of 4 up to 256), d_state %d (up to 256) or heads %d (up to 65535) is not built",
                    s->head_dim, s->d_state, s->heads);
    if (q->conv_kernel < 0 || q->conv_kernel > 4) return fail(GDN_ERR_INVALID_ARG, "conv_kernel %d is not in 0..4", q->conv_kernel);
    if (q->conv_activation != GDN_ACT_NONE && q->conv_activation != GDN_ACT_SILU)
        return fail(GDN_ERR_INVALID_ARG, "the convolution's activation is NONE or SILU");
    if (!(q->dt_min >= 0.0f) || !(q->dt_max >= q->dt_min) || isinf(q->dt_min))
        return fail(GDN_ERR_INVALID_ARG, "0 <= dt_min <= dt_max is needed, dt_min finite");
    g.es = s->io_dtype == GDN_F32 ? 4 : 2;
    g.rows = s->seqlen;
    if (!varlen && g.rows <= INT32_MAX) g.rows *= s->batch;      // (the product of larger ones could pass 64 bits)
    if (g.rows > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%lld token rows are not built", (long long)g.rows);
    g.hp = (int64_t)s->heads * s->head_dim;
    g.C = g.hp + 2LL * s->groups * s->d_state;
    if (g.C > 65535LL * 256)       // (a grid's second extent, of the single-token conv states' 256 channels)
        return fail(GDN_ERR_UNSUPPORTED, "mixed rows of %lld elements are not built", (long long)g.C);
    g.ld_x = s->xbc_stride ? s->xbc_stride : g.C;
    g.ld_dt = s->dt_stride ? s->dt_stride : s->heads;
    g.ld_z = s->z_stride ? s->z_stride : g.hp;
    if (g.ld_x < g.C || g.ld_dt < s->heads || g.ld_z < g.hp)
        return fail(GDN_ERR_INVALID_ARG, "a row stride is below its row's width");
    g.conv_bytes = q->conv_kernel > 1 ? (size_t)(q->conv_kernel - 1) * g.C * g.es : 0;
    return GDN_OK;
}

gdn_status check_rows(int32_t heads, const gdn_ssm_params *q, const Geometry &g, const void *xbc, const void *dt, const void *z,
                      const void *w, const void *bias, const float *A_log, const float *dt_bias, const float *D,
                      const void *y) {
    if (g.rows == 0) return GDN_OK;
    if (!xbc || !dt || !A_log || !y) return fail(GDN_ERR_INVALID_ARG, "xbc, dt, A_log or y is NULL");
    if (q->conv_kernel && !w) return fail(GDN_ERR_INVALID_ARG, "conv_weight is NULL");
    const void *io[] = {xbc, dt, z, y, q->conv_kernel ? w : nullptr, q->conv_kernel ? bias : nullptr};
    for (const void *p : io)
        if (!aligned(p, g.es)) return fail(GDN_ERR_INVALID_ARG, "pointer is not %zu-byte aligned", g.es);
    if (!aligned(A_log, 4) || !aligned(dt_bias, 4) || !aligned(D, 4))
        return fail(GDN_ERR_INVALID_ARG, "A_log, dt_bias and D must be 4-byte aligned");
    const size_t yb = (size_t)g.rows * g.hp * g.es;
    if (overlaps(y, yb, xbc, ((size_t)(g.rows - 1) * g.ld_x + g.C) * g.es) ||
        overlaps(y, yb, z, ((size_t)(g.rows - 1) * g.ld_z + g.hp) * g.es) ||
        overlaps(y, yb, dt, ((size_t)(g.rows - 1) * g.ld_dt + heads) * g.es))
        return fail(GDN_ERR_INVALID_ARG, "y overlaps xbc, z or dt");
    return GDN_OK;
}

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

// The convolved (or re-laid) rows in the workspace: heads and groups on 8-element boundaries.
int64_t u_stride(const gdn_ssm_shape *s) { return s->heads * round8(s->head_dim) + 2 * s->groups * round8(s->d_state); }

bool tc_shape(const gdn_ssm_shape *s, const Geometry &g) {
    return g.rows > 0 && s->num_seqs > 0 && ssm_tc_shape_ok((gdn_dtype)s->io_dtype, s->head_dim, s->d_state);
}

// Workspace bytes: first the rows the scan reads, where it cannot read xbc itself (behind the
// convolution; on the tensor cores also where TMA cannot take xbc's strides, whose rows are then
// copied), then the tensor-core scan's segments.
struct Layout {
    size_t u, total;
};
Layout layout(const gdn_ssm_shape *s, const gdn_ssm_params *q, const Geometry &g, bool varlen) {
    const bool tc = tc_shape(s, g);
    const bool relay = tc && (g.ld_x % 8 != 0 || s->d_state % 8 != 0);
    Layout l{};
    if (q->conv_kernel || relay) l.u = ((size_t)g.rows * u_stride(s) * g.es + 255) / 256 * 256;
    l.total = l.u + (tc ? ssm_tc_workspace(varlen, s->seqlen, g.rows, s->num_seqs, s->heads, s->groups, s->head_dim, s->d_state) : 0);
    return l;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_ssm_prefill_workspace_bytes(const gdn_ssm_shape *shape, const gdn_ssm_params *params) {
    Geometry g;
    if (shape == nullptr || params == nullptr || check(shape, params, shape->batch == 1, g) != GDN_OK) return 0;
    return layout(shape, params, g, shape->batch == 1).total;
}

gdn_status gdn_ssm_prefill_plan(const gdn_ssm_shape *shape, const gdn_ssm_params *params, int32_t *path, int32_t *launches) {
    Geometry g;
    const bool varlen = shape != nullptr && shape->batch == 1 && shape->num_seqs != 1;
    const gdn_status st = check(shape, params, varlen, g);
    if (st != GDN_OK) return st;
    const bool tc = tc_shape(shape, g);
    bool seg = false;
    const int scans = tc ? ssm_tc_launches(varlen, shape->seqlen, g.rows, shape->num_seqs, shape->heads, shape->groups, shape->head_dim, &seg) : 1;
    if (path) *path = tc ? (seg ? 3 : 2) : 1;
    // The convolution's pass: rows to make, or (without any) conv states to carry over.
    const bool conv = layout(shape, params, g, varlen).u > 0 || params->conv_kernel > 1;
    if (launches) *launches = shape->num_seqs > 0 ? conv + scans : 0;
    return GDN_OK;
}

gdn_status gdn_ssm_prefill(const gdn_ssm_shape *shape, const gdn_ssm_params *params, const void *xbc, const void *dt,
                           const void *z, const void *conv_weight, const void *conv_bias, const void *conv_state_in,
                           void *conv_state_out, const float *A_log, const float *dt_bias, const float *D,
                           const float *state_in, const int32_t *cu_seqlens, void *y, float *state_out, void *workspace,
                           size_t workspace_bytes, void *stream) {
    Geometry g;
    gdn_status st = check(shape, params, cu_seqlens != nullptr, g);
    if (st != GDN_OK) return st;
    st = check_rows(shape->heads, params, g, xbc, dt, z, conv_weight, conv_bias, A_log, dt_bias, D, y);
    if (st != GDN_OK) return st;
    if (shape->num_seqs == 0) return GDN_OK;
    if (state_out == nullptr || A_log == nullptr) return fail(GDN_ERR_INVALID_ARG, "state_out or A_log is NULL");
    if (!aligned(state_out, 16) || !aligned(state_in, 16)) return fail(GDN_ERR_INVALID_ARG, "state_in/state_out must be 16-byte aligned");
    if (!aligned(cu_seqlens, 4)) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
    const size_t sb = (size_t)shape->num_seqs * shape->heads * shape->d_state * shape->head_dim * 4;
    if (state_in != state_out && overlaps(state_in, sb, state_out, sb))
        return fail(GDN_ERR_INVALID_ARG, "state_out overlaps state_in without being it");
    const size_t cb = g.conv_bytes * shape->num_seqs;
    if (cb > 0) {
        if (conv_state_out == nullptr) return fail(GDN_ERR_INVALID_ARG, "conv_state_out is NULL");
        if (!aligned(conv_state_in, g.es) || !aligned(conv_state_out, g.es))
            return fail(GDN_ERR_INVALID_ARG, "the conv states must be %zu-byte aligned", g.es);
        if (overlaps(conv_state_in, cb, conv_state_out, cb))
            return fail(GDN_ERR_INVALID_ARG, "conv_state_out overlaps conv_state_in (the update cannot be in place)");
    }
    const Layout ws = layout(shape, params, g, cu_seqlens != nullptr);
    if (ws.total > 0) {
        if (workspace == nullptr || workspace_bytes < ws.total)
            return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu this call needs",
                        workspace == nullptr ? (size_t)0 : workspace_bytes, ws.total);
        if (!aligned(workspace, 16)) return fail(GDN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    }
    int *word = nullptr;
    st = device_check_word(&word);
    if (st != GDN_OK) return st;
    const gdn_dtype io = (gdn_dtype)shape->io_dtype;
    const cudaStream_t cs = (cudaStream_t)stream;

    SsmParams p{};
    p.xs = xbc; p.ldx = g.ld_x; p.x_head = shape->head_dim;
    p.off_b = (int32_t)g.hp; p.off_c = (int32_t)(g.hp + (int64_t)shape->groups * shape->d_state); p.bc_group = shape->d_state;
    p.dt = dt; p.z = z; p.ld_dt = g.ld_dt; p.ld_z = g.ld_z;
    p.A_log = A_log; p.dt_bias = dt_bias; p.D = D; p.dt_min = params->dt_min; p.dt_max = params->dt_max;
    p.state_in = state_in; p.state_out = state_out; p.y = y; p.cu_seqlens = cu_seqlens;
    p.seqlen = shape->seqlen; p.rows = g.rows; p.num_seqs = shape->num_seqs; p.heads = shape->heads;
    p.groups = shape->groups; p.head_dim = shape->head_dim; p.d_state = shape->d_state; p.status = word;
    if (params->conv_kernel || ws.u > 0) {
        SsmConvParams c{};
        c.x = xbc; c.ld_x = g.ld_x; c.w = params->conv_kernel ? conv_weight : nullptr; c.bias = conv_bias;
        c.conv_in = params->conv_kernel > 1 ? conv_state_in : nullptr; c.conv_out = conv_state_out;
        c.u = workspace; c.ld_u = u_stride(shape); c.x_head = (int32_t)round8(shape->head_dim);
        c.bc_group = (int32_t)round8(shape->d_state);
        c.off_b = shape->heads * c.x_head; c.off_c = c.off_b + shape->groups * c.bc_group;
        c.cu_seqlens = cu_seqlens; c.seqlen = p.seqlen; c.rows = p.rows; c.num_seqs = p.num_seqs; c.heads = p.heads;
        c.groups = p.groups; c.head_dim = p.head_dim; c.d_state = p.d_state; c.C = (int32_t)g.C;
        c.K = params->conv_kernel ? params->conv_kernel : 1;
        c.silu = params->conv_activation == GDN_ACT_SILU; c.status = word;
        const cudaError_t e = launch_ssm_conv(c, io, cs);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "state-space convolution launch: %s", cudaGetErrorString(e));
        p.xs = c.u; p.ldx = c.ld_u; p.x_head = c.x_head; p.off_b = c.off_b; p.off_c = c.off_c; p.bc_group = c.bc_group;
    }
    // An xbc or y off 16 bytes (which no shape tells) leaves the tensor cores.
    const bool tc = tc_shape(shape, g) && ssm_tc_rows_ok(p);
    const cudaError_t e = tc ? launch_ssm_tc(p, static_cast<uint8_t *>(workspace) + ws.u, cs) : launch_ssm_scan_simt(p, io, cs);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "state-space scan launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

gdn_status gdn_ssm_decode(const gdn_ssm_shape *shape, const gdn_ssm_params *params, const void *xbc, const void *dt,
                          const void *z, const void *conv_weight, const void *conv_bias, void *conv_state,
                          const float *A_log, const float *dt_bias, const float *D, float *state, int64_t pool_size,
                          const int32_t *slots, void *y, void *stream) {
    Geometry g;
    gdn_status st = check(shape, params, false, g);
    if (st != GDN_OK) return st;
    if (shape->seqlen != 1) return fail(GDN_ERR_INVALID_ARG, "decode takes seqlen 1 (got %lld)", (long long)shape->seqlen);
    st = check_rows(shape->heads, params, g, xbc, dt, z, conv_weight, conv_bias, A_log, dt_bias, D, y);
    if (st != GDN_OK) return st;
    if (shape->batch == 0) return GDN_OK;
    if ((int64_t)shape->batch * shape->heads > INT32_MAX)
        return fail(GDN_ERR_UNSUPPORTED, "batch x heads above 2^31 is not built");
    if (state == nullptr || !aligned(state, 16)) return fail(GDN_ERR_INVALID_ARG, "state is NULL or not 16-byte aligned");
    if (slots != nullptr && pool_size <= 0) return fail(GDN_ERR_INVALID_ARG, "pool_size %lld <= 0", (long long)pool_size);
    if (!aligned(slots, 4)) return fail(GDN_ERR_INVALID_ARG, "slots must be 4-byte aligned");
    if (g.conv_bytes > 0 && (conv_state == nullptr || !aligned(conv_state, g.es)))
        return fail(GDN_ERR_INVALID_ARG, "conv_state is NULL or misaligned");
    int *word = nullptr;
    st = device_check_word(&word);
    if (st != GDN_OK) return st;
    SsmDecodeParams p{};
    p.x = xbc; p.dt = dt; p.z = z; p.ld_x = g.ld_x; p.ld_dt = g.ld_dt; p.ld_z = g.ld_z;
    p.w = params->conv_kernel ? conv_weight : nullptr; p.bias = conv_bias;
    p.conv = g.conv_bytes > 0 ? conv_state : nullptr;
    p.A_log = A_log; p.dt_bias = dt_bias; p.D = D; p.dt_min = params->dt_min; p.dt_max = params->dt_max;
    p.state = state; p.slots = slots; p.pool_size = slots ? pool_size : shape->batch; p.y = y;
    p.batch = shape->batch; p.heads = shape->heads; p.groups = shape->groups; p.head_dim = shape->head_dim;
    p.d_state = shape->d_state; p.C = (int32_t)g.C; p.K = params->conv_kernel;
    p.silu = params->conv_activation == GDN_ACT_SILU; p.status = word;
    const cudaError_t e = launch_ssm_decode(p, (gdn_dtype)shape->io_dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "state-space step launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

}  // extern "C"
