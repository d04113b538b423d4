// rotary.cu -- rotary positions on one or two head tensors (q and k, or C and B of a
// state-space layer) in one launch, and the frequencies of its scaled forms.
//
//   theta = position * inv_freq[i],  (a, b) -> scale (a cos - b sin, b cos + a sin)
// over the pairs (a, b) of dimensions (2i, 2i + 1) or (i, i + rot / 2) of the rotated part;
// the other dimensions are copied.  The inverse turns by -theta (the transpose, so also
// the gradient).
#include <math.h>
#include <stdio.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

// The angle of a far position does not survive an fp32 product, and fp64 is slow here.  So a
// frequency is held as a 64-bit binary fraction of a turn, F = inv_freq / 2 pi mod 1, and
// position * F mod 2^64 is the angle with its whole turns gone, exactly: the product's error
// is position * 2^-54 turns.  sincospif then takes the nearest 32 bits.
//
// A CTA takes `tile` token rows: it fills a table of their cosines and sines, then streams the
// heads.  A thread's item is a place in the row -- two vectors of V values (the V pairs) or one of
// the copied rest -- that it follows down the rows, kRows of them in flight.  Bound by reading and
// writing the heads: 117 us for 32,768 rows of 40 heads of 128 (5.7 TB/s); with four rows in flight,
// and so half as many warps to an SM, it took 163 us.
constexpr int kThreads = 256, kRows = 2, kMaxPairs = 128, kMaxTile = 32;

struct RotaryParams {
    const void *in[2];
    void *out[2];
    int64_t in_row[2], in_head[2], out_row[2], out_head[2];   // element strides
    int32_t heads[2];
    const float *inv_freq;
    const int32_t *positions, *cu_seqlens;   // either may be null
    int64_t rows, seqlen;
    int32_t num_seqs, dim, rot, offset, inverse, tile;
    int32_t across, down;                    // the CTA's threads: items of a row x rows
    float scale;
    int *status;
};

template <typename IO, int V> struct alignas(sizeof(IO) * V) Vec {
    IO v[V];
};

__device__ __forceinline__ int64_t row_position(const RotaryParams &p, int64_t r) {
    if (p.positions) return p.positions[r];
    if (!p.cu_seqlens) return r % p.seqlen;
    int64_t lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    int64_t t0, t1;
    if (!seq_range(p.cu_seqlens, p.rows, p.num_seqs, p.status, lo, t0, t1)) return 0;
    return r - t0;
}

template <typename IO, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const RotaryParams p) {
    __shared__ uint64_t turns[kMaxPairs];
    extern __shared__ __align__(16) float2 cs[];     // [tile][V][pairs / V]: lanes side by side read side by side
    __shared__ int64_t pos[kMaxTile];
    const int tid = threadIdx.x, half = p.rot / 2;
    const int64_t r0 = (int64_t)blockIdx.x * p.tile;
    const int rows = (int)(p.rows - r0 < p.tile ? p.rows - r0 : p.tile);
    for (int i = tid; i < half; i += blockDim.x) {
        const double t = (double)p.inv_freq[i] * 0.15915494309189533577;   // 1 / 2 pi
        turns[i] = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
    }
    for (int i = tid; i < rows; i += blockDim.x) pos[i] = row_position(p, r0 + i);
    __syncthreads();
    const int pairs = half / V;
    for (int e = tid; e < rows * half; e += blockDim.x) {
        const int r = e / half, f = e - r * half;
        const int64_t angle = (int64_t)((uint64_t)pos[r] * turns[f]);      // 2^-64 turns, in [-1/2, 1/2)
        float s, c;
        sincospif((float)(angle >> 32) * 0x1p-31f, &s, &c);
        cs[r * half + (f % V) * pairs + f / V] = make_float2(c * p.scale, p.inverse ? -s * p.scale : s * p.scale);
    }
    __syncthreads();

    const int items = pairs + (p.dim - p.rot) / V, per_row = (p.heads[0] + p.heads[1]) * items;
    const int down = tid / p.across;
    if (down >= p.down) return;
    for (int it = tid - down * p.across; it < per_row; it += p.across) {
        const int hd = it / items, j = it - hd * items;
        const int which = hd >= p.heads[0], h = hd - (which ? p.heads[0] : 0);
        const bool turn = j < pairs;
        const int e = (j - pairs) * V;
        const int d = turn ? p.offset + (kInterleaved ? 2 : 1) * V * j : e < p.offset ? e : e + p.rot;
        const IO *src = static_cast<const IO *>(p.in[which]) + r0 * p.in_row[which] + h * p.in_head[which] + d;
        IO *dst = static_cast<IO *>(p.out[which]) + r0 * p.out_row[which] + h * p.out_head[which] + d;
        const int next = kInterleaved ? V : half;
        for (int rb = down; rb < rows; rb += kRows * p.down) {
            Vec<IO, V> a[kRows], b[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = rb + k * p.down;
                if (r < rows) {
                    a[k] = *reinterpret_cast<const Vec<IO, V> *>(src + r * p.in_row[which]);
                    if (turn) b[k] = *reinterpret_cast<const Vec<IO, V> *>(src + r * p.in_row[which] + next);
                }
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = rb + k * p.down;
                if (r >= rows) break;
                if (turn) {
                    float x[2 * V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        x[i] = IoType<IO>::ld(&a[k].v[i]);
                        x[V + i] = IoType<IO>::ld(&b[k].v[i]);
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 t = cs[r * half + i * pairs + j];
                        float &u = x[kInterleaved ? 2 * i : i], &v = x[kInterleaved ? 2 * i + 1 : V + i];
                        const float w = u * t.x - v * t.y;
                        v = v * t.x + u * t.y;
                        u = w;
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        IoType<IO>::st(&a[k].v[i], x[i]);
                        IoType<IO>::st(&b[k].v[i], x[V + i]);
                    }
                    *reinterpret_cast<Vec<IO, V> *>(dst + r * p.out_row[which] + next) = b[k];
                }
                *reinterpret_cast<Vec<IO, V> *>(dst + r * p.out_row[which]) = a[k];
            }
        }
    }
}

template <typename IO>
cudaError_t rotary_launch(RotaryParams p, bool interleaved, bool wide, cudaStream_t stream) {
    const int V = wide ? 16 / (int)sizeof(IO) : 1;
    // Threads: a row's items in as few equal turns as fit the CTA, rows side by side where they are few.
    const int per_row = (p.heads[0] + p.heads[1]) * (p.rot / 2 / V + (p.dim - p.rot) / V);
    const int turns = (per_row + kThreads - 1) / kThreads;
    p.across = (per_row + turns - 1) / turns;
    // Rows to a CTA: four rounds of four CTAs to an SM where there are so many, up to kMaxTile rows.
    p.tile = (int32_t)(p.rows / 2432);
    p.tile = p.tile < 1 ? 1 : p.tile > kMaxTile ? kMaxTile : p.tile;
    p.down = kThreads / p.across;
    if (p.down > p.tile) p.down = p.tile;
    const unsigned grid = (unsigned)((p.rows + p.tile - 1) / p.tile), threads = (unsigned)((p.across * p.down + 31) / 32 * 32);
    const size_t smem = (size_t)p.tile * (p.rot / 2) * sizeof(float2);
    if (wide && interleaved) rotary_kernel<IO, 16 / sizeof(IO), true><<<grid, threads, smem, stream>>>(p);
    else if (wide) rotary_kernel<IO, 16 / sizeof(IO), false><<<grid, threads, smem, stream>>>(p);
    else if (interleaved) rotary_kernel<IO, 1, true><<<grid, threads, smem, stream>>>(p);
    else rotary_kernel<IO, 1, false><<<grid, threads, smem, stream>>>(p);
    return cudaGetLastError();
}

gdn_status refuse(const char *fmt, long long a = 0, long long b = 0) {
    char msg[256];
    snprintf(msg, sizeof(msg), fmt, a, b);
    return report_error(GDN_ERR_INVALID_ARG, msg);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_rotary(const gdn_rotary_shape *s, const void *q, const void *k, const float *inv_freq,
                                 const int32_t *positions, const int32_t *cu_seqlens, void *q_out, void *k_out,
                                 void *stream) {
    if (s == nullptr) return refuse("shape is NULL");
    if (s->io_dtype != GDN_F32 && s->io_dtype != GDN_BF16 && s->io_dtype != GDN_F16)
        return refuse("io_dtype %lld is not F32/BF16/F16", s->io_dtype);
    if (s->batch < 0 || s->seqlen < 0 || s->num_seqs < 0) return refuse("batch, seqlen and num_seqs must be >= 0");
    if (cu_seqlens ? s->batch != 1 : s->num_seqs != s->batch)
        return refuse("batch must be 1 with cu_seqlens, and equal num_seqs without");
    if (s->heads_q < 0 || s->heads_k < 0 || s->heads_q > 65535 || s->heads_k > 65535)
        return refuse("head counts must be in 0..65535");
    if (s->head_dim < 2 || s->head_dim > 1024) return refuse("head_dim %lld is not in 2..1024", s->head_dim);
    if (s->rot_dim < 2 || s->rot_dim % 2 || s->rot_dim > 2 * kMaxPairs)
        return refuse("rot_dim %lld is not an even number in 2..%lld", s->rot_dim, 2 * kMaxPairs);
    if (s->rot_offset < 0 || s->rot_offset > s->head_dim || s->rot_offset + s->rot_dim > s->head_dim)
        return refuse("the rotated part [%lld, + rot_dim) leaves head_dim %lld", s->rot_offset, s->head_dim);
    if (!(s->scale == s->scale) || isinf(s->scale)) return refuse("scale is not finite");
    const int64_t rows = s->seqlen > INT32_MAX ? s->seqlen : s->batch * s->seqlen;   // (the product of larger ones could pass 64 bits)
    const size_t es = s->io_dtype == GDN_F32 ? 4 : 2;
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int32_t heads[2] = {s->heads_q, s->heads_k};
    const int64_t in_row[2] = {s->q_row_stride, s->k_row_stride}, in_head[2] = {s->q_head_stride, s->k_head_stride};
    const int64_t out_row[2] = {s->q_out_row_stride, s->k_out_row_stride},
                  out_head[2] = {s->q_out_head_stride, s->k_out_head_stride};
    if (rows == 0 || heads[0] + heads[1] == 0 || s->num_seqs == 0) return GDN_OK;
    if (rows > INT32_MAX) return refuse("%lld rows are above 2^31 - 1", rows);
    if (inv_freq == nullptr) return refuse("inv_freq is NULL");
    if (reinterpret_cast<uintptr_t>(inv_freq) % 4 || reinterpret_cast<uintptr_t>(positions) % 4 ||
        reinterpret_cast<uintptr_t>(cu_seqlens) % 4)
        return refuse("inv_freq, positions and cu_seqlens must be 4-byte aligned");
    const int64_t W = 16 / (int64_t)es;
    bool wide = s->head_dim % W == 0 && (s->rot_dim / 2) % W == 0 && s->rot_offset % W == 0;
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        if (in[i] == nullptr || out[i] == nullptr) return refuse("q, k or an output is NULL");
        if (reinterpret_cast<uintptr_t>(in[i]) % es || reinterpret_cast<uintptr_t>(out[i]) % es)
            return refuse("pointer is not %lld-byte aligned", (long long)es);
        if (in_head[i] < s->head_dim || out_head[i] < s->head_dim || in_row[i] < (heads[i] - 1) * in_head[i] + s->head_dim ||
            out_row[i] < (heads[i] - 1) * out_head[i] + s->head_dim)
            return refuse("strides let heads or rows overlap");
        if (in[i] == out[i] && (in_row[i] != out_row[i] || in_head[i] != out_head[i]))
            return refuse("an in-place call needs the same strides in and out");
        wide = wide && reinterpret_cast<uintptr_t>(in[i]) % 16 == 0 && reinterpret_cast<uintptr_t>(out[i]) % 16 == 0 &&
               in_row[i] % W == 0 && in_head[i] % W == 0 && out_row[i] % W == 0 && out_head[i] % W == 0;
    }
    int *word = nullptr;
    const gdn_status st = device_check_word(&word);
    if (st != GDN_OK) return st;
    RotaryParams p{};
    for (int i = 0; i < 2; ++i) {
        p.in[i] = in[i]; p.out[i] = out[i]; p.heads[i] = heads[i];
        p.in_row[i] = in_row[i]; p.in_head[i] = in_head[i]; p.out_row[i] = out_row[i]; p.out_head[i] = out_head[i];
    }
    p.inv_freq = inv_freq; p.positions = positions; p.cu_seqlens = cu_seqlens;
    p.rows = rows; p.seqlen = s->seqlen; p.num_seqs = s->num_seqs;
    p.dim = s->head_dim; p.rot = s->rot_dim; p.offset = s->rot_offset; p.inverse = s->inverse != 0;
    p.scale = s->scale; p.status = word;
    cudaError_t e;
    const bool il = s->interleaved != 0;
    if (s->io_dtype == GDN_F32) e = rotary_launch<float>(p, il, wide, (cudaStream_t)stream);
    else if (s->io_dtype == GDN_BF16) e = rotary_launch<__nv_bfloat16>(p, il, wide, (cudaStream_t)stream);
    else e = rotary_launch<__half>(p, il, wide, (cudaStream_t)stream);
    if (e == cudaSuccess) return GDN_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "rotary launch: %s", cudaGetErrorString(e));
    return report_error(GDN_ERR_CUDA, msg);
}

extern "C" gdn_status gdn_rotary_frequencies(const gdn_rotary_scaling *f, int32_t rot_dim, float *inv_freq, float *scale) {
    if (f == nullptr || inv_freq == nullptr) return refuse("scaling or inv_freq is NULL");
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 2 * kMaxPairs)
        return refuse("rot_dim %lld is not an even number in 2..%lld", rot_dim, 2 * kMaxPairs);
    if (!(f->base > 1.0) || isinf(f->base)) return refuse("base must be finite and above 1");
    if (f->kind < GDN_ROTARY_PLAIN || f->kind > GDN_ROTARY_WAVELENGTH) return refuse("kind %lld is not a gdn_rotary_kind", f->kind);
    const bool bands = f->kind == GDN_ROTARY_BANDS || f->kind == GDN_ROTARY_WAVELENGTH;
    if (f->kind != GDN_ROTARY_PLAIN && (!(f->factor >= 1.0) || isinf(f->factor))) return refuse("factor must be finite and >= 1");
    if (f->kind == GDN_ROTARY_BASE && rot_dim == 2) return refuse("a scaled base needs rot_dim > 2");
    if (bands && (!(f->trained_length > 0.0) || isinf(f->trained_length) || !(f->low > 0.0) || !(f->high > f->low) || isinf(f->high)))
        return refuse("bands need a finite trained_length > 0 and 0 < low < high");
    const double pi2 = 6.283185307179586476925, dim = rot_dim;
    const double base = f->kind == GDN_ROTARY_BASE ? f->base * pow(f->factor, dim / (dim - 2)) : f->base;
    // Bands: the dimension index at which a frequency makes `turns` turns over the trained length.
    auto index = [&](double turns) { return dim * log(f->trained_length / (turns * pi2)) / (2 * log(f->base)); };
    double lo = 0, hi = 0;
    if (f->kind == GDN_ROTARY_BANDS) {
        lo = fmax(floor(index(f->high)), 0.0);
        hi = fmin(ceil(index(f->low)), dim - 1);
        if (hi <= lo) hi = lo + 0.001;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = pow(base, -2.0 * i / dim);
        double keep = 1.0;     // share of the unscaled frequency
        if (f->kind == GDN_ROTARY_LINEAR) keep = 0.0;
        if (f->kind == GDN_ROTARY_BANDS) keep = 1.0 - fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
        if (f->kind == GDN_ROTARY_WAVELENGTH)
            keep = fmin(fmax((f->trained_length * w / pi2 - f->low) / (f->high - f->low), 0.0), 1.0);
        if (f->kind != GDN_ROTARY_PLAIN && f->kind != GDN_ROTARY_BASE) w = w * (keep + (1.0 - keep) / f->factor);
        inv_freq[i] = (float)w;
    }
    if (scale) *scale = f->kind == GDN_ROTARY_BANDS ? (float)(0.1 * log(f->factor) + 1.0) : 1.0f;
    return GDN_OK;
}
