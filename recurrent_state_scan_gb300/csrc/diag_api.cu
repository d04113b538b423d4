// diag_api.cu -- gdn_diag_prefill, gdn_diag_backward, gdn_diag_decode, gdn_checkpoint_pack and _unpack: argument
// checks and dispatch.
#include <stdarg.h>
#include <stdio.h>

#include "diag_internal.cuh"

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

// Bytes that a tensor of evenly spaced rows takes: `rows` of `width` bytes, `apart` bytes from one to the next.
struct Span {
    const char *name;
    const void *p;
    int64_t rows, width, apart;
};

bool overlap(const Span &s, const Span &t) {
    if (!s.p || !t.p || s.rows <= 0 || t.rows <= 0 || s.width <= 0 || t.width <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(s.p), b = reinterpret_cast<uintptr_t>(t.p);
    const uintptr_t na = (uintptr_t)(s.rows - 1) * s.apart + s.width, nb = (uintptr_t)(t.rows - 1) * t.apart + t.width;
    if (!(a < b + nb && b < a + na)) return false;
    if (s.apart != t.apart) return true;
    // Slices of one wider row lie beside one another.
    const uintptr_t d = a < b ? (b - a) % s.apart : (s.apart - (a - b) % s.apart) % s.apart;     // of t's rows behind s's
    return !(d >= (uintptr_t)s.width && d + t.width <= (uintptr_t)s.apart);
}

gdn_status none_overlap(const Span *outs, int n, const Span *ins, int m) {
    for (int i = 0; i < n; ++i) {
        for (int k = 0; k < m; ++k)
            if (overlap(outs[i], ins[k])) return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[k].name);
        for (int k = i + 1; k < n; ++k)
            if (overlap(outs[i], outs[k])) return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return GDN_OK;
}

// What the checks work out on the way.
struct Geometry {
    size_t es;
    int64_t rows, C, n;
    int64_t x, a, b, y, dx, da, db;     // row strides
    size_t kept_states, kept;           // bytes: of the kept states, of all that is kept
};

gdn_status check(const gdn_diag_shape *s, bool varlen, Geometry &g) {
    if (s == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
    if (s->io_dtype != GDN_F32 && s->io_dtype != GDN_BF16 && s->io_dtype != GDN_F16)
        return fail(GDN_ERR_INVALID_ARG, "io_dtype %d is not F32/BF16/F16", s->io_dtype);
    if (s->seqlen < 0 || s->num_seqs < 0 || s->batch < 0)
        return fail(GDN_ERR_INVALID_ARG, "batch, seqlen and num_seqs must be >= 0");
    if (varlen ? s->batch != 1 : s->batch != s->num_seqs)
        return fail(GDN_ERR_INVALID_ARG, "batch must be 1 with cu_seqlens, and equal num_seqs without (batch %d, num_seqs %d)",
                    s->batch, s->num_seqs);
    // (What looks through cu_seqlens adds up to 1,024 to an index, and 32 parts of what is left of them.)
    if (varlen && s->num_seqs > INT32_MAX / 2) return fail(GDN_ERR_UNSUPPORTED, "%d sequences are not built", s->num_seqs);
    if (s->channels <= 0) return fail(GDN_ERR_INVALID_ARG, "channels (%d) must be positive", s->channels);
    if (s->channels > 65535 * kDiagSlice) return fail(GDN_ERR_UNSUPPORTED, "%d channels are not built", s->channels);
    if (s->gate != GDN_DIAG_SOFTPLUS && s->gate != GDN_DIAG_SIGMOID)
        return fail(GDN_ERR_INVALID_ARG, "gate %d is not SOFTPLUS or SIGMOID", s->gate);
    if (s->weighting != GDN_DIAG_PLAIN && s->weighting != GDN_DIAG_COMPLEMENT && s->weighting != GDN_DIAG_NORM)
        return fail(GDN_ERR_INVALID_ARG, "weighting %d is not PLAIN, COMPLEMENT or NORM", s->weighting);
    if (s->input_gate != 0 && s->input_gate != 1) return fail(GDN_ERR_INVALID_ARG, "input_gate must be 0 or 1");
    if (s->keep != GDN_DIAG_KEEP_NONE && s->keep != GDN_DIAG_KEEP_STATES && s->keep != GDN_DIAG_KEEP_8BIT)
        return fail(GDN_ERR_INVALID_ARG, "keep %d is not NONE, STATES or 8BIT", s->keep);
    g.es = s->io_dtype == GDN_F32 ? 4 : 2;
    g.rows = s->seqlen;
    if (!varlen && g.rows <= INT32_MAX) g.rows *= s->batch;      // (the product of larger ones could pass 64 bits)
    if (s->batch == 0) g.rows = 0;
    if (g.rows > INT32_MAX - kDiagTile * 16) return fail(GDN_ERR_UNSUPPORTED, "%lld token rows are not built", (long long)g.rows);
    g.C = s->channels;
    g.n = s->num_seqs;
    const int64_t given[] = {s->x_stride, s->a_stride, s->b_stride, s->y_stride, s->dx_stride, s->da_stride, s->db_stride};
    int64_t *to[] = {&g.x, &g.a, &g.b, &g.y, &g.dx, &g.da, &g.db};
    for (int i = 0; i < 7; ++i) {
        *to[i] = given[i] ? given[i] : g.C;
        if (*to[i] < g.C) return fail(GDN_ERR_INVALID_ARG, "a row stride is below its row's width");
        if (g.rows > 1 && *to[i] > INT64_MAX / 8 / g.rows) return fail(GDN_ERR_UNSUPPORTED, "rows that far apart are not built");
    }
    const size_t slices = diag_slices(s->channels), tiles = (size_t)(g.rows + kDiagTile - 1) / kDiagTile;
    if (tiles * slices > INT32_MAX / 2)
        return fail(GDN_ERR_UNSUPPORTED, "%lld rows of %d channels are not built", (long long)g.rows, s->channels);
    const size_t held = s->keep == GDN_DIAG_KEEP_8BIT ? tiles : s->keep == GDN_DIAG_KEEP_STATES ? tiles * (kDiagTile / kDiagRows) : 0;
    g.kept_states = held * slices * kDiagSlice * 4;
    g.kept = g.kept_states;
    if (s->keep == GDN_DIAG_KEEP_8BIT) g.kept += (size_t)(2 + s->input_gate) * slices * tiles * kDiagTile * (kDiagSlice + 1);
    return GDN_OK;
}

Span io_rows(const char *name, const void *p, const Geometry &g, int64_t ld) {
    return {name, p, g.rows, (int64_t)(g.C * g.es), (int64_t)(ld * g.es)};
}
Span flat(const char *name, const void *p, size_t bytes) { return {name, p, 1, (int64_t)bytes, (int64_t)bytes}; }

gdn_status check_io(const Geometry &g, std::initializer_list<Span> spans) {
    if (g.rows == 0) return GDN_OK;
    for (const Span &s : spans) {
        if (s.p == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", s.name);
        if (!aligned(s.p, g.es)) return fail(GDN_ERR_INVALID_ARG, "%s is not %zu-byte aligned", s.name, g.es);
    }
    return GDN_OK;
}
gdn_status check_floats(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned(p, 4)) return fail(GDN_ERR_INVALID_ARG, "an fp32 or int32 pointer is not 4-byte aligned");
    return GDN_OK;
}
gdn_status check_kept(const Geometry &g, const void *kept, size_t bytes) {
    if (g.kept == 0) return GDN_OK;
    if (kept == nullptr || bytes < g.kept)
        return fail(GDN_ERR_INVALID_ARG, "kept of %zu bytes is below the %zu this call needs", kept == nullptr ? (size_t)0 : bytes, g.kept);
    if (!aligned(kept, 16)) return fail(GDN_ERR_INVALID_ARG, "kept must be 16-byte aligned");
    return GDN_OK;
}

// Whether rows can be taken `n` elements at a time.
bool by(int n, const Geometry &g, std::initializer_list<Span> spans) {
    for (const Span &s : spans)
        if (s.p != nullptr && (!aligned(s.p, n * g.es) || (s.rows > 1 && s.apart % (int64_t)(n * g.es) != 0))) return false;
    return true;
}

// Workspaces: the walk over the tiles, and in the backward pass the tiles' sums of the parameters' gradients.
size_t walk_bytes(const Geometry &g) { return diag_walk_bytes(g.rows, (int)g.C); }
size_t back_bytes(const Geometry &g) {
    const int64_t tiles = diag_tiles(g.rows);
    return tiles > 1 ? walk_bytes(g) + (size_t)tiles * 3 * g.C * 4 : 0;
}
gdn_status check_workspace(const void *workspace, size_t bytes, size_t need) {
    if (need == 0) return GDN_OK;
    if (workspace == nullptr || bytes < need)
        return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu this call needs", workspace == nullptr ? (size_t)0 : bytes, need);
    if (!aligned(workspace, 16)) return fail(GDN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    return GDN_OK;
}

void set_widths(DiagParams &p, const Geometry &g, std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
    p.wide = by(16 / (int)g.es, g, ins) ? 16 : by(2, g, ins) ? 2 * (int)g.es : 0;
    p.pairs = by(2, g, outs);
}

DiagParams params(const gdn_diag_shape *s, const Geometry &g, void *kept) {
    DiagParams p{};
    p.has_b = s->input_gate != 0;
    p.ld_x = g.x; p.ld_a = g.a; p.ld_b = g.b; p.ld_y = g.y; p.ld_dx = g.dx; p.ld_da = g.da; p.ld_db = g.db;
    p.seqlen = s->seqlen; p.rows = g.rows; p.num_seqs = s->num_seqs; p.channels = s->channels;
    const long long budget = __atomic_load_n(&g_wait_budget, __ATOMIC_RELAXED);
    p.budget = budget > 0 ? budget : 4000000000ll;      // (about two seconds)
    if (s->keep != GDN_DIAG_KEEP_NONE) p.kept = static_cast<float *>(kept);
    if (s->keep == GDN_DIAG_KEEP_8BIT) {
        p.codes = static_cast<int8_t *>(kept) + g.kept_states;
        p.steps = reinterpret_cast<uint8_t *>(p.codes) + (g.kept - g.kept_states) / (kDiagSlice + 1) * kDiagSlice;
    }
    return p;
}

gdn_status check_codes(int32_t io, int64_t rows, int64_t C, int64_t &ld, Geometry &g) {
    if (io != GDN_F32 && io != GDN_BF16 && io != GDN_F16) return fail(GDN_ERR_INVALID_ARG, "io_dtype %d is not F32/BF16/F16", io);
    if (rows < 0 || C < 0) return fail(GDN_ERR_INVALID_ARG, "rows and channels must be >= 0");
    if (ld == 0) ld = C;
    if (ld < C) return fail(GDN_ERR_INVALID_ARG, "a row stride is below its row's width");
    if (rows > 0 && ld > INT64_MAX / 8 / rows) return fail(GDN_ERR_UNSUPPORTED, "rows that far apart are not built");
    g.es = io == GDN_F32 ? 4 : 2;
    g.rows = C == 0 ? 0 : rows;
    g.C = C;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_diag_kept_bytes(const gdn_diag_shape *shape) {
    Geometry g;
    return shape != nullptr && check(shape, shape->batch != shape->num_seqs, g) == GDN_OK ? g.kept : 0;
}

size_t gdn_diag_prefill_workspace_bytes(const gdn_diag_shape *shape) {
    Geometry g;
    return shape != nullptr && check(shape, shape->batch != shape->num_seqs, g) == GDN_OK ? walk_bytes(g) : 0;
}

size_t gdn_diag_backward_workspace_bytes(const gdn_diag_shape *shape) {
    Geometry g;
    if (shape == nullptr || check(shape, shape->batch != shape->num_seqs, g) != GDN_OK) return 0;
    return back_bytes(g);
}

gdn_status gdn_diag_prefill(const gdn_diag_shape *shape, const void *x, const void *a, const void *b, const float *A_log,
                            const float *a_bias, const float *b_bias, const float *state_in, const int32_t *cu_seqlens, void *y,
                            float *state_out, void *kept, size_t kept_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    Geometry g;
    gdn_status st = check(shape, cu_seqlens != nullptr, g);
    if (st != GDN_OK) return st;
    const bool has_b = shape->input_gate != 0;
    const Span sx = io_rows("x", x, g, g.x), sa = io_rows("a", a, g, g.a), sb = io_rows("b", has_b ? b : nullptr, g, g.b),
               sy = io_rows("y", y, g, g.y);
    st = has_b ? check_io(g, {sx, sa, sb, sy}) : check_io(g, {sx, sa, sy});
    if (st == GDN_OK) st = check_floats({A_log, a_bias, b_bias, state_in, state_out, cu_seqlens});
    if (st == GDN_OK) st = check_kept(g, kept, kept_bytes);
    if (st != GDN_OK) return st;
    if (g.n == 0 && g.rows == 0) return GDN_OK;
    if (A_log == nullptr || state_out == nullptr) return fail(GDN_ERR_INVALID_ARG, "A_log or state_out is NULL");
    const size_t sbytes = (size_t)g.n * g.C * 4;
    const Span si = flat("state_in", state_in == state_out ? nullptr : state_in, sbytes);
    const size_t need = walk_bytes(g);
    const Span outs[] = {sy, flat("state_out", state_out, sbytes), flat("kept", g.kept ? kept : nullptr, g.kept),
                         flat("workspace", need ? workspace : nullptr, need)};
    const size_t cbytes = (size_t)g.C * 4;
    const Span ins[] = {sx, sa, sb, si, flat("A_log", A_log, cbytes), flat("a_bias", a_bias, cbytes),
                        flat("b_bias", has_b ? b_bias : nullptr, cbytes), flat("cu_seqlens", cu_seqlens, ((size_t)g.n + 1) * 4)};
    st = check_workspace(workspace, workspace_bytes, need);
    if (st == GDN_OK) st = none_overlap(outs, 4, ins, 8);
    if (st != GDN_OK) return st;
    DiagParams p = params(shape, g, kept);
    diag_walk_layout(p, workspace);
    st = device_check_word(&p.status);
    if (st != GDN_OK) return st;
    p.x = x; p.a = a; p.b = b; p.y = y;
    p.A_log = A_log; p.a_bias = a_bias; p.b_bias = has_b ? b_bias : nullptr;
    p.state_in = state_in; p.state_out = state_out; p.cu_seqlens = cu_seqlens;
    set_widths(p, g, {sx, sa, sb}, {sy});
    const cudaError_t e = launch_diag_prefill(p, (gdn_dtype)shape->io_dtype, shape->gate, shape->weighting, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "diagonal recurrence launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

gdn_status gdn_diag_backward(const gdn_diag_shape *shape, const void *x, const void *a, const void *b, const float *A_log,
                             const float *a_bias, const float *b_bias, const float *state_in, const int32_t *cu_seqlens,
                             const void *kept, size_t kept_bytes, const void *dy, const float *dstate_out, void *dx, void *da, void *db,
                             float *dA_log, float *da_bias, float *db_bias, float *dstate_in, void *workspace,
                             size_t workspace_bytes, void *stream) {
    Geometry g;
    gdn_status st = check(shape, cu_seqlens != nullptr, g);
    if (st != GDN_OK) return st;
    if (shape->keep == GDN_DIAG_KEEP_NONE) return fail(GDN_ERR_INVALID_ARG, "the backward pass needs what the forward pass kept (keep is NONE)");
    const bool has_b = shape->input_gate != 0, codes = shape->keep == GDN_DIAG_KEEP_8BIT;
    const Span sx = io_rows("x", codes ? nullptr : x, g, g.x), sa = io_rows("a", codes ? nullptr : a, g, g.a),
               sb = io_rows("b", codes || !has_b ? nullptr : b, g, g.b), sdy = io_rows("dy", dy, g, g.y),
               sdx = io_rows("dx", dx, g, g.dx), sda = io_rows("da", da, g, g.da), sdb = io_rows("db", has_b ? db : nullptr, g, g.db);
    st = check_io(g, {sdy, sdx, sda});
    if (st == GDN_OK && has_b) st = check_io(g, {sdb});
    if (st == GDN_OK && !codes) st = has_b ? check_io(g, {sx, sa, sb}) : check_io(g, {sx, sa});
    if (st == GDN_OK) st = check_floats({A_log, a_bias, b_bias, state_in, cu_seqlens, dstate_out, dA_log, da_bias, db_bias, dstate_in});
    if (st == GDN_OK) st = check_kept(g, kept, kept_bytes);
    if (st != GDN_OK) return st;
    if (A_log == nullptr) return fail(GDN_ERR_INVALID_ARG, "A_log is NULL");
    const size_t sbytes = (size_t)g.n * g.C * 4, cbytes = (size_t)g.C * 4;
    DiagParams p = params(shape, g, const_cast<void *>(kept));
    const size_t need = back_bytes(g);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != GDN_OK) return st;
    diag_walk_layout(p, workspace);
    if (need > 0) p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + walk_bytes(g));
    const Span outs[] = {sdx, sda, sdb, flat("dA_log", dA_log, cbytes), flat("da_bias", da_bias, cbytes),
                         flat("db_bias", has_b ? db_bias : nullptr, cbytes), flat("dstate_in", dstate_in, sbytes),
                         flat("workspace", need ? workspace : nullptr, need)};
    const Span ins[] = {sx, sa, sb, sdy, flat("A_log", A_log, cbytes), flat("a_bias", a_bias, cbytes),
                        flat("b_bias", has_b ? b_bias : nullptr, cbytes), flat("state_in", state_in, sbytes),
                        flat("dstate_out", dstate_out, sbytes), flat("kept", kept, g.kept),
                        flat("cu_seqlens", cu_seqlens, ((size_t)g.n + 1) * 4)};
    st = none_overlap(outs, 8, ins, 11);
    if (st != GDN_OK) return st;
    st = device_check_word(&p.status);
    if (st != GDN_OK) return st;
    p.x = x; p.a = a; p.b = b; p.dy = dy; p.dx = dx; p.da = da; p.db = db;
    p.A_log = A_log; p.a_bias = a_bias; p.b_bias = has_b ? b_bias : nullptr;
    p.state_in = state_in; p.cu_seqlens = cu_seqlens; p.dstate_out = dstate_out; p.dstate_in = dstate_in;
    p.dA_log = dA_log; p.da_bias = da_bias; p.db_bias = has_b ? db_bias : nullptr;
    set_widths(p, g, {sx, sa, sb, sdy}, {sdx, sda, sdb});
    const cudaError_t e = launch_diag_backward(p, (gdn_dtype)shape->io_dtype, shape->gate, shape->weighting, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "diagonal recurrence's backward launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

gdn_status gdn_diag_decode(const gdn_diag_shape *shape, const void *x, const void *a, const void *b, const float *A_log,
                           const float *a_bias, const float *b_bias, float *state, int64_t pool_size, const int32_t *slots, void *y,
                           void *stream) {
    Geometry g;
    gdn_status st = check(shape, false, g);
    if (st != GDN_OK) return st;
    if (shape->seqlen != 1) return fail(GDN_ERR_INVALID_ARG, "decode takes seqlen 1 (got %lld)", (long long)shape->seqlen);
    const bool has_b = shape->input_gate != 0;
    const Span sx = io_rows("x", x, g, g.x), sa = io_rows("a", a, g, g.a), sb = io_rows("b", has_b ? b : nullptr, g, g.b),
               sy = io_rows("y", y, g, g.y);
    st = has_b ? check_io(g, {sx, sa, sb, sy}) : check_io(g, {sx, sa, sy});
    if (st == GDN_OK) st = check_floats({A_log, a_bias, b_bias, state, slots});
    if (st != GDN_OK) return st;
    if (g.rows == 0) return GDN_OK;
    if (A_log == nullptr || state == nullptr) return fail(GDN_ERR_INVALID_ARG, "A_log or state is NULL");
    if (slots != nullptr && pool_size <= 0) return fail(GDN_ERR_INVALID_ARG, "pool_size %lld <= 0", (long long)pool_size);
    const int64_t pool = slots ? pool_size : g.n;
    if (pool > INT64_MAX / 8 / g.C) return fail(GDN_ERR_INVALID_ARG, "pool_size %lld is beyond an address's range", (long long)pool);
    const size_t cbytes = (size_t)g.C * 4;
    const Span outs[] = {sy, flat("state", state, (size_t)pool * g.C * 4)};
    const Span ins[] = {sx, sa, sb, flat("A_log", A_log, cbytes), flat("a_bias", a_bias, cbytes),
                        flat("b_bias", has_b ? b_bias : nullptr, cbytes), flat("slots", slots, (size_t)g.n * 4)};
    st = none_overlap(outs, 2, ins, 7);
    if (st != GDN_OK) return st;
    DiagDecodeParams p{};
    st = device_check_word(&p.status);
    if (st != GDN_OK) return st;
    p.x = x; p.a = a; p.b = b; p.has_b = has_b; p.y = y;
    p.ld_x = g.x; p.ld_a = g.a; p.ld_b = g.b; p.ld_y = g.y;
    p.A_log = A_log; p.a_bias = a_bias; p.b_bias = has_b ? b_bias : nullptr;
    p.state = state; p.pool_size = pool; p.slots = slots;
    p.batch = shape->batch; p.channels = shape->channels;
    p.vec = g.C % 4 == 0 && aligned(state, 16) && by(4, g, {sx, sa, sb, sy});
    const cudaError_t e = launch_diag_decode(p, (gdn_dtype)shape->io_dtype, shape->gate, shape->weighting, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "diagonal recurrence's step launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

gdn_status gdn_checkpoint_pack(int32_t io_dtype, int64_t rows, int64_t channels, const void *x, int64_t x_stride, int8_t *codes,
                               uint8_t *steps, void *stream) {
    Geometry g;
    gdn_status st = check_codes(io_dtype, rows, channels, x_stride, g);
    if (st != GDN_OK) return st;
    const Span sx = io_rows("x", x, g, x_stride);
    st = check_io(g, {sx});
    if (st != GDN_OK || g.rows == 0) return st;
    if (codes == nullptr || steps == nullptr) return fail(GDN_ERR_INVALID_ARG, "codes or steps is NULL");
    const Span outs[] = {flat("codes", codes, (size_t)(rows * channels)),
                         flat("steps", steps, (size_t)(rows * ((channels + kDiagSlice - 1) / kDiagSlice)))};
    st = none_overlap(outs, 2, &sx, 1);
    if (st != GDN_OK) return st;
    const cudaError_t e = launch_checkpoint_pack((gdn_dtype)io_dtype, rows, channels, x, x_stride, codes, steps, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "checkpoint pack launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

gdn_status gdn_checkpoint_unpack(int32_t io_dtype, int64_t rows, int64_t channels, const int8_t *codes, const uint8_t *steps, void *y,
                                 int64_t y_stride, void *stream) {
    Geometry g;
    gdn_status st = check_codes(io_dtype, rows, channels, y_stride, g);
    if (st != GDN_OK) return st;
    const Span sy = io_rows("y", y, g, y_stride);
    st = check_io(g, {sy});
    if (st != GDN_OK || g.rows == 0) return st;
    if (codes == nullptr || steps == nullptr) return fail(GDN_ERR_INVALID_ARG, "codes or steps is NULL");
    const Span ins[] = {flat("codes", codes, (size_t)(rows * channels)),
                        flat("steps", steps, (size_t)(rows * ((channels + kDiagSlice - 1) / kDiagSlice)))};
    st = none_overlap(&sy, 1, ins, 2);
    if (st != GDN_OK) return st;
    const cudaError_t e = launch_checkpoint_unpack((gdn_dtype)io_dtype, rows, channels, codes, steps, y, y_stride, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "checkpoint unpack launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

}  // extern "C"
