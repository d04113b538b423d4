// ssm_tc.cu -- the selective state-space scan of prompts on the tcgen05 tensor cores (bf16
// I/O, head_dim a multiple of 8, d_state up to 128).
//
// The recurrence S = a_t S + d_t B_t (x) x_t, y_t = S^T C_t over chunks of L = 64 tokens, with
// g_t = ln a_t, G_i = g_1 + .. + g_i and S0 the state entering the chunk, is
//   y_i = e^{G_i} C_i S0 + sum_{j <= i} M_ij x_j,   M_ij = (C_i . B_j) e^{G_i - G_j} d_j
//   S   = e^{G_L} S0 + sum_j B_j (x) w_j x_j,       w_j = d_j e^{G_L - G_j}
// Every exponent is a difference that is never positive, so nothing overflows.
//
// A CTA takes two units -- a unit is 64 columns of one head's state -- of one B / C group and
// walks the chunks of a sequence (or of one time segment of it).  Two, because the group's
// scores C B^T then serve both and every MMA is 128 x 128 but the scores' 128 x 64: C stands
// twice in shared memory, so that accumulator rows 0-63 are unit 0's tokens and rows 64-127
// unit 1's, and every lane quarter of tensor memory has work.  Per chunk:
//   scores C B^T -> M (fp32 weights, rounded to bf16) -> [M0; M1] [x0 | x1]     \ y, by the y warps
//   C [S0 | S1]                                                                  /
//   w x split into three bf16 terms -> the sum of B^T [term] -> S = e^{G_L} S + ..     by the S warps
// The warps' roles run side by side, a chunk apart where the data allows it.
//
// Bound by the chain from one chunk's y to the next (the state's product, C S, M x, readout) and by issue: a pair
// of units takes 2.4 us a chunk along a long sequence (3.1 with z over 32 chunks, what comes before the first and
// behind the last included), of which the tensor pipe works a third, the issue slots about half and shared
// memory more than half.  8,192 tokens of 64 heads of 64 x 128 with z: 102 us on 128 CTAs, behind 45 us of
// state-only pass and 6 us for the segments' states.
// Precision: the state is fp32 and its update's operands are exact (B) or a three-term bf16 split (w x, to
// fp32's own 2^-24), because the state is returned in fp32 and carried on: it is 1.1e-7 off, as 32-bit
// arithmetic is, where two terms left it 2.4e-6 off (in 3 to 8% less time).  M and the S that C reads are
// rounded once to bf16, half a step (2^-9 of each term's size at random signs), under the one rounding that
// y meets itself.  f16 stays on the FP32 cores: w x and M leave its range.
//
// Where sequences x units leave most SMs idle, each sequence is cut along time: a state-only
// pass of every segment but the last from zero, a short pass that turns the segments' ends into
// the states entering them, and then all segments at once.  (Uncut, the 8,192 tokens above would
// stand on 32 SMs for 128 chunks, 370 us.)  Packed sequences are taken by length.
#include <cudaTypedefs.h>
#include <stddef.h>
#include <string.h>

#include <type_traits>

#include "ssm_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kL = 64;                       // tokens per chunk
constexpr long long kBudget = 4000000000LL;  // cycles (~2 s) before a wait gives up

// Shared memory (1024-byte aligned): stages of what TMA brings, then the operands the threads
// make.  All tiles are stacks of 128-byte-swizzled rows of 64 bf16.  y, on its way to a TMA store, stands
// in z's place, or, where z comes by TMA itself, in B's, which the chunk's last MMAs are done with.  The
// state-only pass has no C, no S and twice the stages, and takes w x in two buffers.
constexpr int ST_B = 0;                      // 2 regions of 64 state columns x 64 rows
constexpr int ST_X = 16384;                  // 2 units x 64 rows
constexpr int ST_C = 32768;                  // 2 regions x 128 rows: C twice
template <bool kState> constexpr int kStageBytes = kState ? 32768 : 65536;
template <bool kState> constexpr int kStages = kState ? 4 : 2;
constexpr int O_Z = 131072;                  // z or y: 2 units x 64 rows
template <bool kState> constexpr int kWx = kState ? O_Z : O_Z + 16384;    // w x: 3 terms of 2 units x 64 rows
constexpr int WX_TERM = 16384, WX_BYTES = 3 * WX_TERM;
constexpr int O_S = kWx<false> + WX_BYTES;   // bf16(S): 2 units x 128 state rows
constexpr int O_CTL = O_S + 32768;           // Ctl

// Tensor memory columns; M is the A operand of the last MMA, bf16 pairs.
constexpr uint32_t T_CB = 0, T_CS = 64, T_DS = 192, T_MX = 320, T_M = 448, kCols = 512;

struct TcParams {
    CUtensorMap tm_x, tm_b, tm_c, tm_z, tm_y;
    const __nv_bfloat16 *dt, *z;
    __nv_bfloat16 *y;
    int64_t ld_dt, ld_z;
    const float *A_log, *dt_bias, *D;
    float dt_min, dt_max;
    const float *state_in;
    float *state_out;
    const int32_t *cu_seqlens;
    int64_t seqlen, rows;
    int32_t num_seqs, heads, groups, P, N;
    int32_t ptiles, units, pairs_per_group;      // units of one group
    int32_t z_tma;                               // z comes by TMA (its rows are on 16-byte boundaries)
    int32_t seg_chunks;                          // chunks per time segment (0: no segments)
    int32_t cut_over;                            // ssm_order cuts if a sequence has more chunks than this
    int4 *items;                                 // [slot] its sequence, segment and seg_chunks, or null: not ordered
    float *seg_state, *seg_total;                // [slot][unit][N][64], [slot][unit]: a segment's own end state, its Gates::total's sum
    int *status;
    long long budget;
};

// Of the chunk's tokens, in log2: s_i = log2 e^{G_L - G_i}, what the state loses behind token i,
// and lw_j = s_j + log2 d_j.  All that is needed follows: w_j = 2^{lw_j}, the scores' weights
// 2^{lw_j - s_i}, and e^{G_i} = 2^{total - s_i}.
struct alignas(16) Gates {       // read in float2 and float4
    float lw[kL];
    float total, decay;          // log2 e^{G_L}, e^{G_L}
    float s[kL];
};
struct alignas(16) StateGates {  // the part of them that the state needs
    float lw[kL];
    float total, decay;
};

struct Ctl {
    // Barriers: pairs by chunk parity where a waiter can be a chunk behind (`full` and s_ready
    // by stage).
    uint64_t full[4], gates[4], y_read[2], s_ready[4], wx_ready[2], ds[2], full_x[2];
    uint64_t y_done[2], full_z, s_read, cb, cs, mx, m_ready, s_first, drain;
    uint32_t tmem;
    int32_t abort;   // a wait ran out
    Gates g[2][2];   // [stage][unit] (the state-only pass: StateGates of four stages)
};
static_assert(sizeof(Gates) % 16 == 0 && sizeof(StateGates) % 16 == 0 && offsetof(Ctl, g) % 16 == 0 && O_CTL % 16 == 0,
              "vector accesses of the gates");
static_assert(kWx<true> + 2 * WX_BYTES <= O_CTL, "w x of the state-only pass");
constexpr int kCtlBytes = offsetof(Ctl, g) + 8 * sizeof(StateGates);       // the state-only pass's
constexpr int kSmem = O_CTL + ((int)sizeof(Ctl) > kCtlBytes ? (int)sizeof(Ctl) : kCtlBytes);
static_assert(kSmem <= 232448, "shared memory of a CTA");

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ F2 words(uint32_t a, uint32_t b) { return {__uint_as_float(a), __uint_as_float(b)}; }
__device__ __forceinline__ F2 widen(uint32_t v) { return {lo_f(v), hi_f(v)}; }
__device__ __forceinline__ uint32_t pack2(F2 a) { return pack2(a.x, a.y); }
// a silu(z) for two values.  Below z = -87.3 the reciprocal is subnormal and flushed: the gate is 0 where
// silu is within 1.1e-36 of it.  (One reciprocal for both, 1 / d0 = d1 / (d0 d1), needs the exponents held
// down: with z held at -41 the gates below it were wrong by orders, and by way of e^-|z| 8,192 tokens took 1% longer.)
__device__ __forceinline__ F2 gated(F2 a, F2 z) {
    const F2 t = mul2(z, both(-kLog2e)), d = add2({ex2(t.x), ex2(t.y)}, both(1.f));
    return mul2(a, mul2(z, {rcp(d.x), rcp(d.y)}));
}

// Tensor-memory loads have landed.  The values pass through it, so that no arithmetic on them
// can be scheduled ahead of the wait (which does not name them itself).
template <int N> __device__ __forceinline__ void landed(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A bounded wait that gives up when another thread has.  Under a short budget
// (gdn_set_wait_budget) a wait that took longer has run out even where a blocking try saw it end.
// (Out of line: with it inlined at every wait the roles' loops together outgrew the instruction
// cache, whose hits went from 90% to 54%.)
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int32_t *abort, long long budget) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > budget) {
            *abort = 1;
            return false;
        }
    }
    if (budget < 100000 && clock64() - t0 > budget) {
        *abort = 1;
        return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int32_t *abort, long long budget) {
    if (budget >= 100000 && mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity, abort, budget);
}

// Eight z values off 16 bytes (which TMA cannot take).
__device__ __noinline__ uint4 load_unaligned(const __nv_bfloat16 *src) {
    const unsigned short *h = reinterpret_cast<const unsigned short *>(src);
    return make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                      h[6] | (uint32_t)h[7] << 16);
}

// ssm_step of a bf16 value, out of line as well (90 instructions).
__device__ __noinline__ float step_of(uint32_t bits, float bias, float lo, float hi) {
    return ssm_step(__uint_as_float(bits << 16), bias, lo, hi);
}

// The decay 2^total of a chunk or a segment, and the carry for the next one (the first has 0).  A state
// that forgets slowly is multiplied by many of them, and ex2.approx is off to one side (65,536
// tokens, 1,024 chunks: the state 6e-6 off, 3e-5 where all steps are alike).  So slow ones are 1 + x + .. +
// x^5 / 5! (x = total ln 2; the rest is below 6e-9), and what 1 + .. rounds away goes into the next one.
// (Out of line, as the waits are: inlined, 65,536 rows took 3% longer.)
__device__ __noinline__ float2 next_decay(float total, float carry) {
    const float x = total * 0.69314718f;
    if (x < -0.125f) return make_float2(ex2(total), 0.f);
    const float em = fmaf(x * x, fmaf(x, fmaf(x, fmaf(x, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f), x) + carry;
    const float d = 1.f + em;
    return make_float2(d, em - (d - 1.f));
}

// One work item: the chunks [t0, t1) of segment k of sequence n.
struct Item {
    int64_t n, slot, t0, t1;
    int k, nseg;
    bool valid;
};

__device__ __forceinline__ int64_t slot_base(const TcParams &p, int64_t n, int64_t ls, int64_t per) {
    return p.cu_seqlens ? p.cu_seqlens[n] / ls + n : n * per;
}

// Item `place` of a call: of an ordered one as ssm_order put it, else every sequence has equally
// many (or there is one sequence).
__device__ __forceinline__ Item item_at(const TcParams &p, int64_t place) {
    Item it;
    int64_t t0, t1, ls = (int64_t)p.seg_chunks * kL;
    if (p.items != nullptr) {
        const int4 v = p.items[place];
        it.n = v.x;
        it.k = v.y;
        ls = (int64_t)v.z * kL;
        it.valid = v.x >= 0;
    } else {
        const int64_t per = ls == 0 ? 1 : (p.seqlen + ls - 1) / ls;
        it.n = per <= 1 ? place : place / per;
        it.k = per <= 1 ? 0 : (int)(place % per);
        it.valid = it.n < p.num_seqs;
    }
    it.valid = it.valid && seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, it.n, t0, t1);
    if (!it.valid) return it;
    it.nseg = ls == 0 || t1 == t0 ? 1 : (int)((t1 - t0 + ls - 1) / ls);
    it.slot = ls == 0 ? it.n : slot_base(p, it.n, ls, (p.seqlen + ls - 1) / ls) + it.k;
    it.t0 = t0 + it.k * ls;
    it.t1 = ls == 0 || it.t0 + ls > t1 ? t1 : it.t0 + ls;
    return it;
}

// The items of packed sequences in order, the long ones first: more of them than SMs are then
// done soonest.  Six sequences of 4,096 to 20,480 tokens on 32 unit pairs took 1,180 us in their
// own order and cut at a fair share, 892 us like this (and 773 by now).  Sequences are cut along time
// only where one is long enough to be worth the state-only pass.  By one block: the
// segments but each sequence's last in the first bin, which are all that the state-only pass needs,
// the others in bins of a quarter of an octave of their chunks.  Atomics place the items of a bin,
// in any order (which no result depends on); places without an item hold sequence -1.  Bound by latency and the launch.
constexpr int kOrderThreads = 512, kBins = 128;
__device__ __forceinline__ int bin_of(int chunks) {            // 1 for the longest
    return chunks <= 0 ? kBins - 1 : kBins - 2 - min(kBins - 3, (int)(__float_as_uint((float)chunks) >> 21) - (127 << 2));
}
__global__ void __launch_bounds__(kOrderThreads) ssm_order(const __grid_constant__ TcParams p, int64_t places) {
    __shared__ int at[kBins], longest, bad, items;
    const int tid = threadIdx.x;
    if (tid < kBins) at[tid] = 0;
    if (tid == 0) longest = bad = 0;
    __syncthreads();
    auto chunks_of = [&](int64_t n) {                          // -1: bad offsets
        int64_t t0, t1;
        return seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, n, t0, t1) ? (int)((t1 - t0 + kL - 1) / kL) : -1;
    };
    int most = 0;
    for (int64_t n = tid; n < p.num_seqs; n += kOrderThreads) {
        const int chunks = chunks_of(n);
        most = max(most, chunks);
        if (chunks < 0) bad = 1;
    }
    if (most > 0) atomicMax(&longest, most);
    __syncthreads();
    // (Beside bad offsets sequences that are fine by themselves may overlap, and have more segments than
    // the rows: they are not cut.)
    const int seg = longest > p.cut_over && bad == 0 ? p.seg_chunks : 0;
    // Of sequence n: `lead` segments of seg chunks ahead of its last, and the last's chunks (-1: no items).
    auto parts = [&](int64_t n, int &lead, int &last) {
        const int chunks = chunks_of(n);
        lead = seg == 0 || chunks <= 0 ? 0 : (chunks - 1) / seg;
        last = chunks - lead * seg;
    };
    int lead, last;
    for (int64_t n = tid; n < p.num_seqs; n += kOrderThreads) {
        parts(n, lead, last);
        if (lead > 0) atomicAdd(&at[0], lead);
        if (last >= 0) atomicAdd(&at[bin_of(last)], 1);
    }
    __syncthreads();
    if (tid < 32) {                                            // counts to first places
        int c[kBins / 32], sum = 0;
        for (int i = 0; i < kBins / 32; ++i) sum += c[i] = at[kBins / 32 * tid + i];
        int upto = sum;
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (tid >= d) upto += v;
        }
        if (tid == 31) items = upto;
        upto -= sum;
        for (int i = 0; i < kBins / 32; ++i) {
            at[kBins / 32 * tid + i] = upto;
            upto += c[i];
        }
    }
    __syncthreads();
    auto put = [&](int place, int64_t n, int k) {
        if (place < places) p.items[place] = make_int4((int)n, k, seg, 0);
    };
    for (int64_t n = tid; n < p.num_seqs; n += kOrderThreads) {
        parts(n, lead, last);
        const int first = lead > 0 ? atomicAdd(&at[0], lead) : 0;
        for (int k = 0; k < lead; ++k) put(first + k, n, k);
        if (last >= 0) put(atomicAdd(&at[bin_of(last)], 1), n, lead);
    }
    for (int64_t i = items + (int64_t)tid; i < places; i += kOrderThreads) p.items[i] = make_int4(-1, 0, seg, 0);
}

// The roles of a CTA's warps, each with its own pace; mbarriers carry the order.
//   0-7    y: M from the scores, and the readout (row 32 (warp % 4) + lane, 32 columns of it)
//   8-15   S: the state (its row n, the 64 columns of one unit, in registers)
//   16     issues the MMAs     17  issues the TMA copies     18, 19  the gates of unit 0, 1; the
//          state-only pass, which two of them bound (46 us, then 41), has 20, 21 for its odd chunks
//   20-23  w x (the state-only pass leaves it to warps 0-7).  With the S warps making it, behind the
//          state's update, they held the others up: 3.09 us a chunk, then 2.87.
constexpr int kSWarp = 8, kIssueWarp = 16, kLoadWarp = 17, kGateWarp = 18, kWxWarp = 20;
constexpr int kZNone = 0, kZTma = 1, kZRows = 2;   // no z, z by TMA, z off 16 bytes
template <bool kState> constexpr int kThreads = 32 * (kState ? kGateWarp + 4 : kWxWarp + 4);

// kState: the state-only pass of a segment (no scores, no y; warps 0-7 make w x there).  kZ: where z
// comes from, known to the compiler because the loops that do not ask are 4% faster.
template <bool kState, int kZ>
__global__ void __launch_bounds__(kThreads<kState>, 1) ssm_chunk_scan(const __grid_constant__ TcParams p) {
    // (Nothing static stands before it, so dynamic shared memory begins on a 1024-byte boundary, as
    // the swizzled tiles need; there is no room to align it here.)
    extern __shared__ __align__(1024) uint8_t sm[];
    Ctl &ctl = *reinterpret_cast<Ctl *>(sm + O_CTL);
    using GateSet = std::conditional_t<kState, StateGates, Gates>;
    GateSet(*const gate)[2] = reinterpret_cast<GateSet(*)[2]>(reinterpret_cast<uint8_t *>(&ctl) + offsetof(Ctl, g));
    const Gates(*const ygate)[2] = ctl.g;            // (the y warps', which the state-only pass has not)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = p.groups * p.pairs_per_group;
    const int pair = blockIdx.x % pairs;
    const Item it = item_at(p, blockIdx.x / pairs);
    if (!it.valid || (kState && it.k + 1 >= it.nseg)) return;
    if (smem_u32(sm) % 1024 != 0) {
        if (tid == 0) atomicOr(p.status, kDevTimeout);
        return;
    }

    // The two units.  An odd last unit is computed twice and stored once.
    const int g = pair / p.pairs_per_group, u0 = 2 * (pair % p.pairs_per_group);
    const int hpg = p.heads / p.groups;
    const bool two = u0 + 1 < p.units;
    auto unit_head = [&](int u) { return g * hpg + (u0 + (two ? u : 0)) / p.ptiles; };
    auto unit_tile = [&](int u) { return (u0 + (two ? u : 0)) % p.ptiles; };

    const long long budget = p.budget > 0 ? p.budget : kBudget;
    if (warp == kIssueWarp) {
        tmem_alloc(&ctl.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.s_ready[i], 8);
            mbar_init(&ctl.gates[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.y_read[i], 8);
            mbar_init(&ctl.wx_ready[i], kState ? 8 : 4);
            mbar_init(&ctl.ds[i], 1);
            mbar_init(&ctl.full_x[i], 1);
            mbar_init(&ctl.y_done[i], 8);
        }
        mbar_init(&ctl.full_z, 1);
        mbar_init(&ctl.s_read, 8);
        mbar_init(&ctl.cb, 1);
        mbar_init(&ctl.cs, 1);
        mbar_init(&ctl.mx, 1);
        mbar_init(&ctl.m_ready, 8);
        mbar_init(&ctl.s_first, 8);
        mbar_init(&ctl.drain, 1);
        fence_mbar_init();
        ctl.abort = 0;
    }
    volatile int32_t *abort = &ctl.abort;
    constexpr int NS = kStages<kState>;
    const int nchunks = (int)((it.t1 - it.t0 + kL - 1) / kL);
    auto chunk_len = [&](int c) {
        const int64_t left = it.t1 - it.t0 - (int64_t)c * kL;
        return left < kL ? (int)left : kL;
    };
    // A phase of a barrier that completes once per chunk, and of one of a pair by chunk parity.
    auto wait = [&](uint64_t *bar, int c) { return wait_for(bar, c & 1, abort, budget); };
    auto wait2 = [&](uint64_t *bar, int c) { return wait_for(bar + (c & 1), (c >> 1) & 1, abort, budget); };
    auto wait_st = [&](uint64_t *bar, int c) { return wait_for(bar + (c & (NS - 1)), (c / NS) & 1, abort, budget); };
    auto stage = [&](int c) { return sm + (c & (NS - 1)) * kStageBytes<kState>; };
    auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    // This warp's tensor-memory accesses are done (and, with `smem`, its shared-memory writes, for
    // the tensor cores and TMA too): one arrival.
    auto arrive = [&](uint64_t *bar, bool smem) {
        if (smem) fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // Rows behind the sequence are another's: as operands they have to be zero.
    auto clear_rows = [&](int c, int who) {
        uint8_t *st = stage(c);
        const int len = chunk_len(c);
        for (int e = who; e < (kL - len) * 32; e += kState ? 256 : 128) {
            const int r = len + (e >> 5), k = e & 31;       // B regions 0, 1, units 0, 1
            *reinterpret_cast<uint4 *>(st + (k >> 3) * 8192 + sw128_offset(r, k & 7)) = make_uint4(0, 0, 0, 0);
        }
    };
    // w x of chunk c by 128 threads (256 in the state-only pass), split into three bf16 terms, at buffer `to`.
    auto make_wx = [&](int c, int who, uint8_t *to) {
        const uint8_t *xt = stage(c) + ST_X;
        const int len = chunk_len(c);
        if (len < kL) clear_rows(c, who);
        constexpr int kStep = kState ? 32 : 16;      // tokens that the threads take at once
        const int j0 = who >> 3;
        const uint32_t at0 = sw128_offset(j0, who & 7);
        const float *lw = &gate[c & (NS - 1)][0].lw[j0];
#pragma unroll 2
        for (int v = 0; v < 128 / kStep; ++v) {
            const int j = j0 + kStep * (v % (64 / kStep));
            const uint32_t at = at0 + 128 * kStep * v;
            const float w = ex2(lw[kStep * (v % (64 / kStep)) + (v < 64 / kStep ? 0 : sizeof(GateSet) / 4)]);   // unit 0's, 1's
            const uint4 xv = j < len ? *reinterpret_cast<const uint4 *>(xt + at) : make_uint4(0, 0, 0, 0);
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
            uint32_t t[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                F2 rest = mul2(both(w), widen(xw[i]));
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    t[k][i] = pack2(rest);
                    if (k < 2) rest = fma2(both(-1.f), widen(t[k][i]), rest);
                }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(to + k * WX_TERM + at) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
        }
    };

    const int q = warp & 3, half = (warp >> 2) & 1;   // TMEM lane quarter, column half
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    bool ok = true;

    if (warp == kIssueWarp) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            const uint32_t base = smem_u32(sm);
            constexpr uint32_t kIdCB = idesc_f16(true, 128, 64, false, false), kIdCS = idesc_f16(true, 128, 128, false, true),
                               kIdDS = idesc_f16(true, 128, 128, true, true);
            const int ksteps = (p.N + 15) / 16;
            // Descriptors; their low field counts 16 bytes, so a K step adds 2 (K-major) or 128.
            // The products over d_state are unrolled whole for 128, else by four K steps: a rolled loop
            // does not feed the tensor cores (C S took 1,070 cycles where the state's unrolled eight took 550).
            // (Unrolled with each MMA under its own condition, nvcc 13.0 gave one of them another's
            // operand.)
            const uint64_t dC = sw128_desc(base + ST_C, 16, 1024), dBk = sw128_desc(base + ST_B, 16, 1024),
                           dS = sw128_desc(base + O_S, 16384, 1024), dBm = sw128_desc(base + ST_B, 8192, 1024),
                           dWX = sw128_desc(base + kWx<kState>, 8192, 1024), dX = sw128_desc(base + ST_X, 8192, 1024);
            auto issue_cb = [&](int c) {
                const uint64_t st = (uint64_t)(c & (NS - 1)) * (kStageBytes<kState> >> 4);
                if (ksteps == 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16(tmem + T_CB, dC + st + (k >> 2) * 1024 + (k & 3) * 2, dBk + st + (k >> 2) * 512 + (k & 3) * 2, kIdCB, k > 0);
                } else {
#pragma unroll 1
                    for (int q4 = 0; q4 < ksteps / 4; ++q4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f16(tmem + T_CB, dC + st + q4 * 1024 + k * 2, dBk + st + q4 * 512 + k * 2, kIdCB, q4 + k > 0);
                    }
#pragma unroll 1
                    for (int k = ksteps & ~3; k < ksteps; ++k)
                        mma_f16(tmem + T_CB, dC + st + (k >> 2) * 1024 + (k & 3) * 2, dBk + st + (k >> 2) * 512 + (k & 3) * 2, kIdCB, k > 0);
                }
                mma_commit(&ctl.cb);
            };
            if (!kState && nchunks > 0 && (ok = wait_st(ctl.full, 0))) issue_cb(0);
            for (int c = 0; ok && c < nchunks; ++c) {
                const uint64_t st = (uint64_t)(c & (NS - 1)) * (kStageBytes<kState> >> 4);
                // The state's.  (B has landed: the scores waited for it.)
                if (!(ok = wait2(ctl.wx_ready, c) && (kState ? wait_st(ctl.full, c) && (c < 2 || wait_st(ctl.s_ready, c - 2))
                                                             : wait2(ctl.full_x, c) && (c == 0 || wait(&ctl.s_read, c - 1)))))
                    break;
                tc_fence_after();
                const uint64_t wx = dWX + (kState && (c & 1) ? WX_BYTES >> 4 : 0);
                const uint32_t dst = tmem + (kState && (c & 1) ? T_CS : T_DS);
#pragma unroll
                for (int k = 0; k < 12; ++k)
                    mma_f16(dst, dBm + st + (k & 3) * 128, wx + (2 - (k >> 2)) * (WX_TERM >> 4) + (k & 3) * 128, kIdDS, k > 0);      // the smallest term first
                mma_commit(&ctl.ds[kState ? c & 1 : 0]);
                if (kState) continue;
                // C S, once S is in place and the accumulators of the chunk before are read.
                if (!(ok = c == 0 ? wait(&ctl.s_first, 0) : wait_st(ctl.s_ready, c - 1) && wait2(ctl.y_read, c - 1))) break;
                tc_fence_after();
                if (ksteps == 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16(tmem + T_CS, dC + st + (k >> 2) * 1024 + (k & 3) * 2, dS + k * 128, kIdCS, k > 0);
                } else {
#pragma unroll 1
                    for (int q4 = 0; q4 < ksteps / 4; ++q4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f16(tmem + T_CS, dC + st + q4 * 1024 + k * 2, dS + (4 * q4 + k) * 128, kIdCS, q4 + k > 0);
                    }
#pragma unroll 1
                    for (int k = ksteps & ~3; k < ksteps; ++k)
                        mma_f16(tmem + T_CS, dC + st + (k >> 2) * 1024 + (k & 3) * 2, dS + k * 128, kIdCS, k > 0);
                }
                mma_commit(&ctl.cs);
                if (!(ok = wait(&ctl.m_ready, c))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_f16_ts(tmem + T_MX, tmem + T_M + 8 * k, dX + st + k * 128, kIdCS, k > 0);
                mma_commit(&ctl.mx);
                if (c + 1 < nchunks) {
                    if (!(ok = wait_st(ctl.full, c + 1))) break;
                    issue_cb(c + 1);
                }
            }
            if (!ok) *abort = 1;
            // What is in flight finishes before the CTA leaves (bounded).
            mma_commit(&ctl.drain);
            mbar_wait(&ctl.drain, 0, kBudget);
        }
        __syncwarp();
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ TMA loads
        if (lane == 0) {
            const int regions = p.N > 64 ? 2 : 1;
            int loaded = 0, loaded_x = 0, loaded_z = 0;
            const int tile_u[2] = {64 * unit_tile(0), 64 * unit_tile(1)}, head_u[2] = {unit_head(0), unit_head(1)};
            auto row_of = [&](int c) { return (int)(it.t0 + (int64_t)c * kL); };
            // z, or (where it does not come by TMA) word that its place is free for y.
            auto load_z = [&](int c) {
                if (c >= nchunks) return;
                loaded_z = c + 1;
                if (kZ != kZTma) {
                    mbar_arrive(&ctl.full_z);
                    return;
                }
                mbar_arrive_expect_tx(&ctl.full_z, 16384);
                for (int u = 0; u < 2; ++u) tma_load_3d(sm + O_Z + u * 8192, &p.tm_z, tile_u[u], head_u[u], row_of(c), &ctl.full_z);
            };
            for (int c = 0; ok && c < nchunks + (kState ? 0 : 2); ++c) {
                uint8_t *st = stage(c);
                // A stage is free when the last MMA of the chunk in it is done: its S has been taken,
                // or its y read out (x with it).  x first: w x waits for it.
                if (c >= NS && !(ok = kState ? wait_st(ctl.s_ready, c - NS) : wait2(ctl.y_read, c - NS))) break;
                uint64_t *bar = &ctl.full[c & (NS - 1)], *bar_x = kState ? bar : &ctl.full_x[c & 1];
                const int t = row_of(c);
                auto load_bc = [&]() {
                    if (!kState) mbar_arrive_expect_tx(bar, 8192u * 3 * regions);
#pragma unroll 1
                    for (int r = 0; r < regions; ++r) {
                        tma_load_3d(st + ST_B + r * 8192, &p.tm_b, 64 * r, g, t, bar);
                        if (!kState) {
                            tma_load_3d(st + ST_C + r * 16384, &p.tm_c, 64 * r, g, t, bar);
                            tma_load_3d(st + ST_C + r * 16384 + 8192, &p.tm_c, 64 * r, g, t, bar);
                        }
                    }
                    loaded = c + 1;
                };
                if (c < nchunks) {
                    if (kState) mbar_arrive_expect_tx(bar, 8192u * (regions + 2));
                    else mbar_arrive_expect_tx(bar_x, 16384);
                    for (int u = 0; u < 2; ++u) tma_load_3d(st + ST_X + u * 8192, &p.tm_x, tile_u[u], head_u[u], t, bar_x);
                    loaded_x = c + 1;
                    if (kZ != kZTma) load_bc();
                }
                if (kState) continue;
                // y of chunk c - 2 goes out, and then what takes its place comes in: the next B, or the next y.  (A
                // sequence's last rows, where they do not fill the chunk, are stored by their threads.)
                if (c >= 2) {
                    if (!(ok = wait2(ctl.y_done, c - 2))) break;
                    if (kZ == kZTma) load_z(c - 1);
                    if (chunk_len(c - 2) == kL) {
                        uint8_t *yt = kZ == kZTma ? st + ST_B : sm + O_Z;
                        for (int u = 0; u < 1 + two; ++u) tma_store_3d(&p.tm_y, yt + u * 8192, tile_u[u], head_u[u], row_of(c - 2));
                        bulk_commit();
                    }
                    bulk_wait_read();
                }
                if (kZ == kZTma) {
                    if (c == 1) load_z(0);
                    if (c < nchunks) load_bc();
                } else if (c > 0) {
                    load_z(c - 1);
                }
            }
            // Copies still in flight finish before the CTA leaves (bounded).
            for (int c = loaded - NS < 0 ? 0 : loaded - NS; c < loaded; ++c) mbar_wait(&ctl.full[c & (NS - 1)], (c / NS) & 1, kBudget);
            if (!kState) {
                for (int c = loaded_x - 2 < 0 ? 0 : loaded_x - 2; c < loaded_x; ++c) mbar_wait(&ctl.full_x[c & 1], (c >> 1) & 1, kBudget);
                if (loaded_z > 0) mbar_wait(&ctl.full_z, (loaded_z - 1) & 1, kBudget);
            }
            bulk_wait_all();
            if (!ok) *abort = 1;
        }
        __syncwarp();
    } else if (!kState && warp >= kWxWarp) {
        // ------------------------------------------------------------ w x (the state's MMA of the chunk before has left its buffer)
        for (int c = 0; c < nchunks; ++c) {
            if (!(ok = all((c == 0 || wait(&ctl.ds[0], c - 1)) && wait2(ctl.full_x, c) && (chunk_len(c) == kL || wait_st(ctl.full, c)) &&
                           wait_st(ctl.gates, c))))
                break;
            make_wx(c, tid - 32 * kWxWarp, sm + kWx<kState>);
            arrive(&ctl.wx_ready[c & 1], true);
        }
        if (!ok) *abort = 1;
    } else if (warp >= kGateWarp) {
        // ------------------------------------------------------------ gates: two tokens to a lane
        // A decay of e^-111 is already nothing in fp32, so g is held above that: a reset then leaves
        // the sums over it small enough to keep the differences of the tokens before it.
        const int u = (warp - kGateWarp) & 1, head = unit_head(u), first = (warp - kGateWarp) >> 1, step = kState ? 2 : 1;
        const float A = ssm_rate(p.A_log[head]) * kLog2e, bias = p.dt_bias ? p.dt_bias[head] : 0.f;
        unsigned short n0 = 0, n1 = 0;      // bits, widened a chunk later: nothing waits for the load here
        float carry = 0.f;
        auto load_dt = [&](int c) {
            const int64_t t = it.t0 + (int64_t)c * kL + 2 * lane;
            const unsigned short *at = reinterpret_cast<const unsigned short *>(p.dt + t * p.ld_dt + head);
            if (t < it.t1) n0 = at[0];
            if (t + 1 < it.t1) n1 = at[p.ld_dt];
        };
        if (first < nchunks) load_dt(first);
        for (int c = first; c < nchunks; c += step) {
            const int len = chunk_len(c);
            const float d0 = 2 * lane < len ? step_of(n0, bias, p.dt_min, p.dt_max) : 0.f;
            const float d1 = 2 * lane + 1 < len ? step_of(n1, bias, p.dt_min, p.dt_max) : 0.f;
            if (c + step < nchunks) load_dt(c + step);      // (behind the calls, which would wait for it)
            float g0 = A * d0, g1 = A * d1;
            g0 = g0 < -160.f ? -160.f : g0;
            g1 = g1 < -160.f ? -160.f : g1;
            float suf = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane + o < 32) suf += v;
            }
            float after = __shfl_down_sync(0xffffffffu, suf, 1);
            if (lane == 31) after = 0.f;
            const float l0 = __log2f(d0), l1 = __log2f(d1);   // -inf where the step is zero: no weight
            const float2 decay = next_decay(suf, carry);      // (lane 0's is the whole chunk's)
            carry = decay.y;
            if (c >= NS && !(ok = all(wait_st(ctl.s_ready, c - NS) && (kState || wait2(ctl.y_read, c - NS))))) break;
            GateSet &G = gate[c & (NS - 1)][u];
            if constexpr (!kState) *reinterpret_cast<float2 *>(&G.s[2 * lane]) = make_float2(after + g1, after);
            *reinterpret_cast<float2 *>(&G.lw[2 * lane]) = make_float2(after + g1 + l0, after + l1);
            if (lane == 0) {
                G.total = suf;
                G.decay = decay.x;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.gates[c & (NS - 1)]);
        }
        if (!ok) *abort = 1;
    } else if (warp >= kSWarp) {
        // ------------------------------------------------------------ S: state row sn, the 64 columns of unit su
        const int sn = 32 * q + lane, su = (warp >> 2) & 1;
        const int ucols = p.P - unit_tile(su) * 64;       // columns of this unit that exist
        const int64_t nunits = (int64_t)p.groups * p.units;
        const int64_t sunit = (int64_t)g * p.units + u0 + (two ? su : 0);
        const size_t sglob = (((size_t)it.n * p.heads + unit_head(su)) * p.N + sn) * p.P + unit_tile(su) * 64;
        const size_t sseg = ((size_t)it.slot * nunits + sunit) * p.N * 64 + (size_t)sn * 64;
        const float *from = nullptr;
        if (!kState && sn < p.N) from = it.nseg > 1 ? p.seg_state + sseg : p.state_in ? p.state_in + sglob : nullptr;
        const int have = from == nullptr ? 0 : it.nseg > 1 ? 64 : ucols;
        float S[64];
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < have) v = *reinterpret_cast<const float4 *>(from + i);
            S[i] = v.x; S[i + 1] = v.y; S[i + 2] = v.z; S[i + 3] = v.w;
        }
        auto put_S = [&]() {     // bf16(S) as the next readout's operand
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(sm + O_S + su * 16384 + sw128_offset(sn, c)) =
                    make_uint4(pack2(S[8 * c], S[8 * c + 1]), pack2(S[8 * c + 2], S[8 * c + 3]), pack2(S[8 * c + 4], S[8 * c + 5]),
                               pack2(S[8 * c + 6], S[8 * c + 7]));
        };
        if (!kState) {
            put_S();
            arrive(&ctl.s_first, true);
        }
        float seg_total = 0.f;
        for (int c = 0; ok && c < nchunks; ++c) {
            if (!(ok = all((kState ? wait2(ctl.ds, c) : wait(&ctl.ds[0], c)) && wait_st(ctl.gates, c)))) break;
            tc_fence_after();
            const float dec = gate[c & (NS - 1)][su].decay;
            seg_total += gate[c & (NS - 1)][su].total;
            const uint32_t src = tmem + lanes + (kState && (c & 1) ? T_CS : T_DS) + 64 * su;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                uint32_t r[8];
                tmem_ld8(src + 8 * b, r);
                tmem_ld_wait();
                landed(r);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const F2 v = fma2(both(dec), {S[8 * b + i], S[8 * b + i + 1]}, words(r[i], r[i + 1]));
                    S[8 * b + i] = v.x;
                    S[8 * b + i + 1] = v.y;
                }
            }
            if (!kState) {
                arrive(&ctl.s_read, false);
                if (!(ok = all(wait(&ctl.cs, c)))) break;      // the readout has read the old S
                put_S();
            }
            arrive(&ctl.s_ready[c & (NS - 1)], !kState);
        }
        if (!ok) {
            *abort = 1;
        } else if (sn < p.N && (su == 0 || two)) {
            if (kState) {
#pragma unroll
                for (int i = 0; i < 64; i += 4)
                    *reinterpret_cast<float4 *>(p.seg_state + sseg + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
                if (sn == 0) p.seg_total[it.slot * nunits + sunit] = seg_total;
            } else if (it.k + 1 == it.nseg) {
#pragma unroll
                for (int i = 0; i < 64; i += 4)
                    if (i < ucols) *reinterpret_cast<float4 *>(p.state_out + sglob + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
            }
        }
    } else if (kState) {
        // ------------------------------------------------------------ w x of the state-only pass, two buffers
        for (int c = 0; c < nchunks; ++c) {
            if (!(ok = all(wait_st(ctl.full, c) && wait_st(ctl.gates, c) && (c < 2 || wait2(ctl.ds, c - 2))))) break;
            make_wx(c, tid, sm + kWx<kState> + (c & 1) * WX_BYTES);
            arrive(&ctl.wx_ready[c & 1], true);
        }
        if (!ok) *abort = 1;
    } else {
        // ------------------------------------------------------------ M and y
        // Token ri of unit ru; columns 32 half .. of the scores and of the unit.
        const int row = 32 * q + lane, ru = q >> 1, ri = row & 63;
        const int head = unit_head(ru), col = unit_tile(ru) * 64 + 32 * half;
        const bool live = (ru == 0 || two) && col < p.P;
        const float D = p.D ? p.D[head] : 0.f;
        // Scores of chunk c, weighted: 0 above the diagonal (all of this warp's where its
        // columns are behind its rows).
        auto make_m = [&](int c) {
            const Gates &G = ygate[c & 1][ru];
            const float si = G.s[ri];
            tc_fence_after();
#pragma unroll 1
            for (int j0 = 32 * half; j0 < 32 * half + 32; j0 += 8) {
                uint32_t m[4] = {0, 0, 0, 0};
                if (j0 <= 32 * (q & 1) + 31) {
                    uint32_t r[8];
                    tmem_ld8(tmem + T_CB + lanes + j0, r);
                    tmem_ld_wait();
                    landed(r);
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 lw = *reinterpret_cast<const float4 *>(&G.lw[j0 + i]);
                        const F2 e0 = add2({lw.x, lw.y}, both(-si)), e1 = add2({lw.z, lw.w}, both(-si));
                        F2 v0 = mul2(words(r[i], r[i + 1]), {ex2(e0.x), ex2(e0.y)});
                        F2 v1 = mul2(words(r[i + 2], r[i + 3]), {ex2(e1.x), ex2(e1.y)});
                        const int past = j0 + i - ri;
                        v0 = {past <= 0 ? v0.x : 0.f, past + 1 <= 0 ? v0.y : 0.f};
                        v1 = {past + 2 <= 0 ? v1.x : 0.f, past + 3 <= 0 ? v1.y : 0.f};
                        m[i / 2] = pack2(v0);
                        m[i / 2 + 1] = pack2(v1);
                    }
                }
                tmem_st4(tmem + T_M + lanes + j0 / 2, m);
            }
            tmem_st_wait();
        };
        auto next_m = [&](int c) {
            if (!(ok = all(wait_st(ctl.gates, c) && wait(&ctl.cb, c)))) return;
            make_m(c);
            arrive(&ctl.m_ready, false);
        };
        if (nchunks > 0) next_m(0);
        for (int c = 0; ok && c < nchunks; ++c) {
            // (The last MMA of the chunk: what was issued before it, C S among it, is done too.)
            if (!(ok = all(wait(&ctl.mx, c) && wait2(ctl.full_x, c) && wait(&ctl.full_z, c)))) break;
            tc_fence_after();
            const uint8_t *xt = stage(c) + ST_X + ru * 8192, *zt = sm + O_Z + ru * 8192;
            uint8_t *yt = (kZ == kZTma ? stage(c) + ST_B : sm + O_Z) + ru * 8192;
            const float e = ex2(ygate[c & 1][ru].total - ygate[c & 1][ru].s[ri]);
            const int len = chunk_len(c);
            __nv_bfloat16 *dst = p.y + ((it.t0 + (int64_t)c * kL + ri) * p.heads + head) * (int64_t)p.P + col;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t m[8], cs[8];
                const uint32_t at = lanes + 64 * ru + 32 * half + 8 * b;
                tmem_ld8(tmem + T_MX + at, m);
                tmem_ld8(tmem + T_CS + at, cs);
                const uint32_t piece = sw128_offset(ri, 4 * half + b);
                const uint4 xv = *reinterpret_cast<const uint4 *>(xt + piece);
                const int pc = 8 * b;
                uint4 zv = make_uint4(0, 0, 0, 0);
                if (kZ != kZNone) {
                    if (kZ == kZTma) zv = *reinterpret_cast<const uint4 *>(zt + piece);
                    else if (live && ri < len && col + pc < p.P)
                        zv = load_unaligned(p.z + (it.t0 + (int64_t)c * kL + ri) * p.ld_z + (int64_t)head * p.P + col + pc);
                }
                tmem_ld_wait();
                landed(m);
                landed(cs);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, zw[4] = {zv.x, zv.y, zv.z, zv.w};
                uint32_t out[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    F2 a = fma2(both(D), widen(xw[i]), fma2(both(e), words(cs[2 * i], cs[2 * i + 1]), words(m[2 * i], m[2 * i + 1])));
                    if (kZ != kZNone) a = gated(a, widen(zw[i]));
                    out[i] = pack2(a);
                }
                const uint4 o = make_uint4(out[0], out[1], out[2], out[3]);
                // A whole chunk's y goes out by TMA.
                if (len == kL) *reinterpret_cast<uint4 *>(yt + piece) = o;
                else if (live && ri < len && col + pc < p.P) *reinterpret_cast<uint4 *>(dst + pc) = o;
            }
            arrive(&ctl.y_read[c & 1], false);
            arrive(&ctl.y_done[c & 1], true);
            if (c + 1 < nchunks) next_m(c + 1);
        }
        if (!ok) *abort = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && ctl.abort) atomicOr(p.status, kDevTimeout);
    if (warp == kIssueWarp) tmem_dealloc(tmem, kCols);
}

// The state entering each segment, in the place of the segment's own end state: of sequence
// blockIdx.x, or of an ordered call's item there, where it is its sequence's first of several.
__global__ void __launch_bounds__(256) ssm_segment_states(const __grid_constant__ TcParams p) {
    const int64_t unit = blockIdx.y, nunits = (int64_t)p.groups * p.units;
    int64_t n = blockIdx.x;
    if (p.items != nullptr) {
        const int4 v = p.items[n];
        if (v.x < 0 || v.y != 0 || v.z == 0) return;
        n = v.x;
    }
    const int64_t ls = (int64_t)p.seg_chunks * kL, per = (p.seqlen + ls - 1) / ls;
    int64_t t0, t1;
    if (!seq_range(p.cu_seqlens, p.seqlen, p.num_seqs, p.status, n, t0, t1)) return;
    const int nseg = (int)((t1 - t0 + ls - 1) / ls);
    if (nseg <= 1) return;
    const int64_t first = slot_base(p, n, ls, per);
    const int head = (int)(unit / p.units) * (p.heads / p.groups) + (int)(unit % p.units) / p.ptiles;
    const int tile = (int)(unit % p.units) % p.ptiles;
    const int e = blockIdx.z * 256 + threadIdx.x, r = e >> 4, col = 4 * (e & 15);
    if (e >= p.N * 16) return;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.state_in && tile * 64 + col < p.P)
        S = *reinterpret_cast<const float4 *>(p.state_in + (((size_t)n * p.heads + head) * p.N + r) * p.P + tile * 64 + col);
    const size_t step = (size_t)nunits * p.N * 64;
    float4 *place = reinterpret_cast<float4 *>(p.seg_state + (size_t)(first * nunits + unit) * p.N * 64 + 4 * (size_t)e);
    const float *total = p.seg_total + first * nunits + unit;
    float carry = 0.f;
    constexpr int kAhead = 8;         // segments loaded at once: the chain itself is a decay and an FMA each
    for (int k0 = 0; k0 < nseg; k0 += kAhead) {
        float4 own[kAhead];
        float t[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k0 + i + 1 < nseg) {
                own[i] = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(place) + (size_t)(k0 + i) * step);
                t[i] = total[(int64_t)(k0 + i) * nunits];
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k0 + i >= nseg) break;
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(place) + (size_t)(k0 + i) * step) = S;
            if (k0 + i + 1 == nseg) break;
            const float2 d = next_decay(t[i], carry);
            carry = d.y;
            S.x = fmaf(d.x, S.x, own[i].x); S.y = fmaf(d.x, S.y, own[i].y);
            S.z = fmaf(d.x, S.z, own[i].z); S.w = fmaf(d.x, S.w, own[i].w);
        }
    }
}

int unit_pairs(int heads, int groups, int head_dim) {
    const int units = heads / groups * ((head_dim + 63) / 64);
    return groups * ((units + 1) / 2);
}

// A state-only chunk takes 0.45 (with z) to 0.57 of a whole one, so cutting into the SMs' fair shares costs
// 1.5 of one at least, and up to 2 with rests: uncut sequences of up to kCutOver shares are as good.
constexpr int kSms = 152, kMinSegChunks = 8;
constexpr double kCutOver = 1.6;

// Chunks per segment (0: no segments).  Sequences are cut where sequences x pairs of units
// fill less than half of the SMs; the segments then fill them once.
int segment_chunks(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int pairs) {
    if (num_seqs <= 0 || pairs <= 0) return 0;
    const int64_t chunks = varlen ? (rows + kL - 1) / kL : (seqlen + kL - 1) / kL;
    const int64_t wanted = kSms / (varlen ? pairs : pairs * num_seqs);   // packed: of the whole row
    if (wanted < 2) return 0;
    int64_t seg = (chunks + wanted - 1) / wanted;
    if (seg < kMinSegChunks) seg = kMinSegChunks;
    return seg >= chunks ? 0 : (int)seg;
}

int64_t segment_slots(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int seg) {
    if (seg == 0) return num_seqs;
    const int64_t ls = (int64_t)seg * kL;
    return varlen ? rows / ls + num_seqs : num_seqs * ((seqlen + ls - 1) / ls);
}

struct SegBytes {
    int seg;
    int64_t slots;
    bool ordered;
    size_t state, items, total;
};
SegBytes segment_bytes(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int heads, int groups, int head_dim,
                       int d_state) {
    SegBytes b{};
    b.seg = segment_chunks(varlen, seqlen, rows, num_seqs, unit_pairs(heads, groups, head_dim));
    b.slots = segment_slots(varlen, seqlen, rows, num_seqs, b.seg);
    b.ordered = varlen && num_seqs > 1 && (b.seg > 0 || b.slots * unit_pairs(heads, groups, head_dim) > kSms);
    if (b.seg > 0) {
        const size_t units = (size_t)heads * ((head_dim + 63) / 64);
        b.state = (size_t)b.slots * units * d_state * 64 * 4;
        b.items = b.state + ((size_t)b.slots * units * 4 + 255) / 256 * 256;
    }
    b.total = b.items + (b.ordered ? (size_t)b.slots * 16 : 0);
    return b;
}

}  // namespace

bool ssm_tc_shape_ok(gdn_dtype io, int head_dim, int d_state) {
    return io == GDN_BF16 && head_dim % 8 == 0 && d_state <= 128;
}

bool ssm_tc_rows_ok(const SsmParams &p) {
    return reinterpret_cast<uintptr_t>(p.xs) % 16 == 0 && p.ldx % 8 == 0 && p.x_head % 8 == 0 && p.off_b % 8 == 0 &&
           p.off_c % 8 == 0 && p.bc_group % 8 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
}

int ssm_tc_launches(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int heads, int groups, int head_dim, bool *segments) {
    const SegBytes b = segment_bytes(varlen, seqlen, rows, num_seqs, heads, groups, head_dim, 1);
    *segments = b.seg > 0;
    return (b.ordered ? 1 : 0) + (b.seg > 0 ? 3 : 1);
}

size_t ssm_tc_workspace(bool varlen, int64_t seqlen, int64_t rows, int64_t num_seqs, int heads, int groups, int head_dim,
                        int d_state) {
    return segment_bytes(varlen, seqlen, rows, num_seqs, heads, groups, head_dim, d_state).total;
}

cudaError_t launch_ssm_tc(const SsmParams &s, void *workspace, cudaStream_t stream) {
    TcParams p;
    memset(&p, 0, sizeof(p));
    const bool varlen = s.cu_seqlens != nullptr;
    const uint64_t row = (uint64_t)s.ldx * 2;
    const __nv_bfloat16 *xs = static_cast<const __nv_bfloat16 *>(s.xs);
    const uint32_t box[3] = {64, 1, kL};
    const uint64_t dx[3] = {(uint64_t)s.head_dim, (uint64_t)s.heads, (uint64_t)s.rows}, sx[2] = {(uint64_t)s.x_head * 2, row};
    const uint64_t db[3] = {(uint64_t)s.d_state, (uint64_t)s.groups, (uint64_t)s.rows}, sb[2] = {(uint64_t)s.bc_group * 2, row};
    if (!encode_map_3d(&p.tm_x, xs, GDN_BF16, dx, sx, box, true) || !encode_map_3d(&p.tm_b, xs + s.off_b, GDN_BF16, db, sb, box, true) ||
        !encode_map_3d(&p.tm_c, xs + s.off_c, GDN_BF16, db, sb, box, true))
        return cudaErrorInvalidValue;
    p.dt = static_cast<const __nv_bfloat16 *>(s.dt);
    p.z = static_cast<const __nv_bfloat16 *>(s.z);
    p.y = static_cast<__nv_bfloat16 *>(s.y);
    p.ld_dt = s.ld_dt; p.ld_z = s.ld_z; p.A_log = s.A_log; p.dt_bias = s.dt_bias; p.D = s.D;
    p.dt_min = s.dt_min; p.dt_max = s.dt_max; p.state_in = s.state_in; p.state_out = s.state_out;
    p.cu_seqlens = s.cu_seqlens; p.seqlen = s.seqlen; p.rows = s.rows; p.num_seqs = s.num_seqs;
    p.heads = s.heads; p.groups = s.groups; p.P = s.head_dim; p.N = s.d_state;
    p.ptiles = (s.head_dim + 63) / 64;
    p.units = s.heads / s.groups * p.ptiles;
    p.pairs_per_group = (p.units + 1) / 2;
    p.z_tma = s.z != nullptr && reinterpret_cast<uintptr_t>(s.z) % 16 == 0 && s.ld_z % 8 == 0;
    const uint64_t sy[2] = {(uint64_t)s.head_dim * 2, (uint64_t)s.head_dim * s.heads * 2}, sz[2] = {sy[0], (uint64_t)s.ld_z * 2};
    if (!encode_map_3d(&p.tm_y, s.y, GDN_BF16, dx, sy, box, true) ||
        (p.z_tma && !encode_map_3d(&p.tm_z, s.z, GDN_BF16, dx, sz, box, true)))
        return cudaErrorInvalidValue;
    p.status = s.status;
    p.budget = __atomic_load_n(&g_wait_budget, __ATOMIC_RELAXED);
    const SegBytes b = segment_bytes(varlen, s.seqlen, s.rows, s.num_seqs, s.heads, s.groups, s.head_dim, s.d_state);
    p.seg_chunks = b.seg;
    const int pairs = s.groups * p.pairs_per_group;
    if (b.seg > 0) p.cut_over = (int32_t)(kCutOver * ((s.rows + kL - 1) / kL) * pairs / kSms);
    p.seg_state = static_cast<float *>(workspace);
    p.seg_total = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + b.state);
    p.items = b.ordered ? reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + b.items) : nullptr;

    const int64_t grid = b.slots * pairs;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    void (*const main)(TcParams) = s.z == nullptr ? ssm_chunk_scan<false, kZNone> : p.z_tma ? ssm_chunk_scan<false, kZTma> : ssm_chunk_scan<false, kZRows>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_chunk_scan<true, kZNone>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (b.ordered) {
        ssm_order<<<1, kOrderThreads, 0, stream>>>(p, b.slots);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (b.seg > 0) {
        // Of an ordered call only the first bin's items, each whole segments of its own rows.
        const int64_t lead = s.rows / ((int64_t)b.seg * kL);
        ssm_chunk_scan<true, kZNone><<<(unsigned)((b.ordered ? lead : b.slots) * pairs), kThreads<true>, kSmem, stream>>>(p);
        ssm_segment_states<<<dim3((unsigned)(b.ordered ? lead : s.num_seqs), (unsigned)(s.groups * p.units), (unsigned)((s.d_state + 15) / 16)), 256, 0, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    main<<<(unsigned)grid, kThreads<false>, kSmem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
