// The norm after a block, its gate, the residual add and the norm before the next block, in one pass over the rows, and
// the backward pass of that.
//
//   b = x rx w'              rx = rsqrt(mean(x^2) + eps), w' = offset + post_weight     (b = x without post_norm)
//   s = bf16(residual + scale f(gate) b)
//   y = s rs w               rs = rsqrt(mean(s^2) + eps), w = offset + pre_weight
//
// Backward, with s^ = s rs, x^ = x rx and mean over the row:
//   D = dsum + rs (dy w - s^ mean(dy w s^))              dresidual = D
//   dgate = scale D b f'(gate)   summed over what shares the gate
//   e = scale f(gate) D,  dx = rx (e w' - x^ mean(e w' x^))       (dx = e without post_norm)
//   dpre_weight = sum_t dy s^,  dpost_weight = sum_t e x^
//
// Bound: bytes, then instructions.  Forward, a thread keeps CH segments of 8 elements of a row in registers from the one read to
// the write; sums over the row go through shuffles and shared memory.  Backward, a block walks over every gridDim-th
// row: its next rows are on their way (by the copy engine, into rings) under this one's sums.  A row needs two rounds of sums:
// of what needs only the inputs, then of what needs D; the first of the next row go with the second of this one, one
// barrier a row.  The sums over rows of a thread's columns lie in shared memory, are
// written as one row of the workspace, and a second launch adds those up in a fixed order.
// Measured: forward of 16384 x 2048 with a gate per element 59 us (336 MB, 5.7 TB/s; one row a block of 256 threads 86), one row 1.8 us behind
// another launch; backward of the same 95 us (537 MB, 5.7 TB/s; 205 with a barrier for each sum and values one by
// one, 123 with rows through registers), of 8192 x 5120 112 us (6.0 TB/s; 147 with two barriers a row and every thread reading every
// warp's sums), of 777 x 5120 with a gate per channel 20 us, of which the sums over blocks are 4.
#include "bf16.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

__device__ __forceinline__ uint4 load8(const uint16_t *p, size_t seg) { return reinterpret_cast<const uint4 *>(p)[seg]; }
__device__ __forceinline__ uint4 load8_once(const uint16_t *p, size_t seg) { return __ldcs(reinterpret_cast<const uint4 *>(p) + seg); }
constexpr long long kWaitPolls = 1 << 20;                 // bound of a wait, about a second

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// offset + weight, or ones, of a segment.
__device__ __forceinline__ void weights(const uint16_t *w, uint4 raw, F2 offset, F2 (&v)[4])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2(1.f, 1.f);
        return;
    }
    unpack8(raw, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], offset);
}
__device__ __forceinline__ float sum2(F2 v)
{
    const float2 p = unf2(v);
    return p.x + p.y;
}
// f of a segment's gate values.
__device__ __forceinline__ void gate_values(int act, uint4 raw, F2 (&f)[4])
{
    unpack8(raw, f);
    if (act == MOE_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 g = unf2(f[i]);
        const float s0 = sigmoid(g.x), s1 = sigmoid(g.y);
        f[i] = act == MOE_ACT_SILU ? f2(g.x * s0, g.y * s1) : f2(s0, s1);
    }
}

// Sums of N values over the TPR threads of a row, and with `more` (N > 1, rows of more than four warps) of one more; buf, more_buf: a float4 a warp that no thread
// still reads.  Every thread of the block takes part.  Four values share their first two exchanges (each lane goes on with
// one of them): 6 shuffles in place of 20.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float4 *buf, float *more = nullptr, float4 *more_buf = nullptr)
{
    static_assert(N <= 4, "a float4 a warp");
    constexpr bool kWide = N > 1 && TPR / 32 > 4;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, w0 = w / (TPR / 32) * (TPR / 32);
    if (N > 1) {
        const float v2 = N > 2 ? v[N > 2 ? 2 : 0] : 0.f, v3 = N > 3 ? v[N > 3 ? 3 : 0] : 0.f;
        const bool odd = lane & 1, high = lane & 2;
        float p = odd ? v[1] : v[0], q = odd ? v3 : v2;                          // values 0 and 2, or 1 and 3
        p += __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[1], 1);
        if (N > 2) q += __shfl_xor_sync(0xFFFFFFFFu, odd ? v2 : v3, 1);
        float r = N > 2 && high ? q : p;
        r += __shfl_xor_sync(0xFFFFFFFFu, N > 2 ? (high ? p : q) : p, 2);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
        if (TPR == 32) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, r, i);
            return;
        }
        if (lane < 4) reinterpret_cast<float *>(buf + w)[lane] = r;
    } else {
#pragma unroll
        for (int o = 16; o; o >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        if (TPR == 32) return;
        if (lane == 0) buf[w].x = v[0];
    }
    if (kWide && more) {
#pragma unroll
        for (int o = 16; o; o >>= 1) *more += __shfl_xor_sync(0xFFFFFFFFu, *more, o);
        if (lane == 0) more_buf[w].x = *more;
    }
    __syncthreads();
    if constexpr (kWide) {
        // a lane adds up one value of every eighth warp (a float4 read by all lanes costs four of one word, for each warp)
        float r = 0.f;
#pragma unroll
        for (int j = 0; j < TPR / 32; j += 8)
            if (j + (lane >> 2) < TPR / 32) r += reinterpret_cast<const float *>(buf + w0 + j)[lane];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, r, i);
        if (more) {
            float q = lane < TPR / 32 ? more_buf[w0 + lane].x : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
            *more = q;
        }
        return;
    }
    F2 lo = f2(0.f, 0.f), hi = lo;
    float one = 0.f;
#pragma unroll 8
    for (int j = 0; j < TPR / 32; ++j) {
        if (N == 1) {
            one += buf[w0 + j].x;
        } else if (N == 2) {
            const float2 p = *reinterpret_cast<const float2 *>(buf + w0 + j);
            lo = add2(lo, f2(p.x, p.y));
        } else {
            const float4 p = buf[w0 + j];
            lo = add2(lo, f2(p.x, p.y));
            hi = add2(hi, f2(p.z, p.w));
        }
    }
    const float2 l = unf2(lo), h = unf2(hi);
    v[0] = N == 1 ? one : l.x;
    if (N > 1) v[N > 1 ? 1 : 0] = l.y;
    if (N > 2) v[N > 2 ? 2 : 0] = h.x;
    if (N > 3) v[N > 3 ? 3 : 0] = h.y;
}

constexpr int block_of(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR, int CH>
__global__ void __launch_bounds__(block_of(TPR)) gated_norm_kernel(const __grid_constant__ GatedNormArgs a)
{
    constexpr int kRows = block_of(TPR) / TPR;
    __shared__ float4 buf[2][block_of(TPR) / 32];
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, tr = threadIdx.x % TPR, t = blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = t < a.T;
    const size_t row = (size_t)t * nseg;
    uint4 rx[CH], rr[CH], rg[CH], w0[CH], w1[CH];
    const float row_gate = live && a.gate_shape == MOE_GATE_ROW ? bf16_bits_to_float(a.gate[t]) : 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int seg = c * TPR + tr;
        const bool on = live && seg < nseg;
        rx[c] = on ? load8_once(a.x, row + seg) : zero4();
        rr[c] = on && a.residual ? load8_once(a.residual, row + seg) : zero4();
        rg[c] = on && a.gate_shape == MOE_GATE_FULL      ? load8_once(a.gate, row + seg)
                : on && a.gate_shape == MOE_GATE_CHANNEL ? load8(a.gate, seg)
                                                         : zero4();
        w0[c] = on && a.post_weight ? load8(a.post_weight, seg) : zero4();
        w1[c] = on && a.y && a.pre_weight ? load8(a.pre_weight, seg) : zero4();
    }
    F2 x[CH][4];
#pragma unroll
    for (int c = 0; c < CH; ++c) unpack8(rx[c], x[c]);
    float rstd = 1.f;
    if (a.post_norm) {
        F2 ss = f2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fma2(x[c][i], x[c][i], ss);
        float v[1] = {sum2(ss)};
        row_sums<TPR>(v, buf[0]);
        rstd = rsqrtf(v[0] / (float)a.n + a.eps);
    }
    float each = a.scale * rstd;
    if (a.gate_shape == MOE_GATE_ROW) each *= act_value(a.act, row_gate);
    const F2 each2 = f2(each, each), off2 = f2(a.weight_offset, a.weight_offset);
    F2 ss = f2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int seg = c * TPR + tr;
        F2 r[4], w[4], g[4];
        unpack8(rr[c], r);
        weights(a.post_weight, w0[c], off2, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][i] = mul2(mul2(x[c][i], each2), w[i]);
        if (a.gate_shape >= MOE_GATE_CHANNEL) {
            gate_values(a.act, rg[c], g);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[c][i] = fma2(g[i], x[c][i], r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[c][i] = add2(x[c][i], r[i]);
        }
        const uint4 s = pack8(x[c]);
        if (live && seg < nseg && a.sum) reinterpret_cast<uint4 *>(a.sum)[row + seg] = s;
        unpack8(s, x[c]);
        if (seg < nseg) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fma2(x[c][i], x[c][i], ss);
        }
    }
    if (!a.y) return;
    float v[1] = {sum2(ss)};
    row_sums<TPR>(v, buf[1]);
    rstd = rsqrtf(v[0] / (float)a.n + a.eps);
    const F2 r2 = f2(rstd, rstd);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int seg = c * TPR + tr;
        F2 w[4];
        weights(a.pre_weight, w1[c], off2, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][i] = mul2(mul2(x[c][i], r2), w[i]);
        if (live && seg < nseg) reinterpret_cast<uint4 *>(a.y)[row + seg] = pack8(x[c]);
    }
}

// A row's inputs as they were read.
struct RawRow {
    uint4 x, s, dy, ds, gate;
    float row_gate;
};
__device__ __forceinline__ RawRow load_row(const GatedNormArgs &a, int t, int nseg, int seg, bool on)
{
    RawRow r{zero4(), zero4(), zero4(), zero4(), zero4(), 0.f};
    if (t >= a.T) return r;
    if (a.gate_shape == MOE_GATE_ROW) r.row_gate = bf16_bits_to_float(a.gate[t]);
    if (!on) return r;
    const size_t at = (size_t)t * nseg + seg;
    r.x = load8_once(a.x, at);
    r.s = load8_once(a.sum, at);
    if (a.dy) r.dy = load8_once(a.dy, at);
    if (a.dsum) r.ds = load8_once(a.dsum, at);
    if (a.gate_shape == MOE_GATE_FULL) r.gate = load8_once(a.gate, at);
    if (a.gate_shape == MOE_GATE_CHANNEL) r.gate = load8(a.gate, seg);
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4 &u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }
__device__ __forceinline__ F2 pair_of(const uint4 &u, int i) { return f2(bf16_lo(word(u, i)), bf16_hi(word(u, i))); }
// A segment of weights with their offset: in fp32 (KEEP, where registers last) or as they were read; ones without weights.
template <bool KEEP>
struct Weights {
    F2 v[KEEP ? 4 : 1], off;
    uint4 raw;
    __device__ __forceinline__ Weights(const uint16_t *w, int seg, bool on, float offset)
    {
        raw = w && on ? load8(w, seg) : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        off = w ? f2(offset, offset) : f2(0.f, 0.f);
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < (KEEP ? 4 : 1); ++i) v[i] = add2(pair_of(raw, i), off);
        }
    }
    __device__ __forceinline__ F2 operator[](int i) const { return KEEP ? v[KEEP ? i : 0] : add2(pair_of(raw, i), off); }
};
__device__ __forceinline__ uint32_t pack_pair(F2 v)
{
    const float2 p = unf2(v);
    return pack_bf16(p.x, p.y);
}
template <int ACT>
__device__ __forceinline__ void gate_pair(F2 raw, F2 &f, F2 &slope)
{
    f = raw;
    slope = f2(1.f, 1.f);
    if (ACT == MOE_ACT_NONE) return;
    const float2 g = unf2(raw);
    if (ACT == MOE_ACT_SILU) {
        const F2 s = f2(sigmoid(g.x), sigmoid(g.y)), minus = f2(-1.f, -1.f);
        f = mul2(raw, s);
        slope = fma2(f, fma2(s, minus, f2(1.f, 1.f)), s);       // s + g s (1 - s)
    } else {
        // (one by one: in pairs 2 to 5% slower)
        const float2 lo = sigmoid_slope(g.x), hi = sigmoid_slope(g.y);
        f = f2(lo.x, hi.x);
        slope = f2(lo.y, hi.y);
    }
}

// A place of a ring: its rows one behind the other (of x's one, of the other's s, dy, dsum and a gate per element).
__device__ __forceinline__ uint4 ring8(const uint8_t *row, int which, int nseg, int seg) { return reinterpret_cast<const uint4 *>(row)[which * nseg + seg]; }

// STAGES: rows come through rings in shared memory, filled by the copy engine STAGES rows ahead of this one, x's a place longer
// than the others' (x is read once more behind the row's last sums, when the others' places are free).  ARRAYS of a place
// besides x: all 4, or s and dy alone, where dsum and a gate per element come through registers a row ahead.  No stages: all of
// it through registers, the next row's elements on their way under this row's sums, where the rings pay nothing.
// Rows are kept as they were read and widened in each round; the sums over rows lie in shared memory, each thread's own.
template <int TPR, int BLOCKS, int STAGES, int ARRAYS, bool BY_ELEMENT, int ACT>
__global__ void __launch_bounds__(TPR, BLOCKS) gated_norm_grad_kernel(const __grid_constant__ GatedNormArgs a)
{
    extern __shared__ float4 sums[];                           // [post, pre, gate][half of a segment][thread]
    __shared__ float4 buf[2][2][TPR / 32];                     // [row's parity][round]
    __shared__ uint64_t landed[STAGES ? STAGES : 1];
    __shared__ int failed[2];                                  // by the row's parity: whether a wait for the row after it ran out
    constexpr bool kJoint = STAGES > 0;
    constexpr bool kLate = kJoint && ARRAYS < 4;
    const int nseg = a.n / 8, seg = threadIdx.x;
    const bool on = seg < nseg;
    pdl_trigger();
    if (STAGES && threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(tc::smem_u32(&landed[i]), 1);
        failed[0] = failed[1] = 0;
        tc::fence_mbar_init();
    }
    if (STAGES) __syncthreads();
    pdl_wait();
    const uint32_t row_bytes = 2 * a.n;
    uint8_t *const ring_x = reinterpret_cast<uint8_t *>(sums + 6 * TPR), *const ring = ring_x + (STAGES + 1) * row_bytes;
    const bool gate_rows = BY_ELEMENT && a.gate_shape == MOE_GATE_FULL;
    // row t into the rings' places `st` and `sx` (one thread)
    auto fetch = [&](int t, int st, int sx) {
        if (t >= a.T) return;
        const uint32_t bar = tc::smem_u32(&landed[st]), to = tc::smem_u32(ring) + st * ARRAYS * row_bytes;
        const uint16_t *const src[4] = {a.sum, a.dy, a.dsum, gate_rows ? a.gate : nullptr};
        uint32_t arrays = 1;
        for (int i = 0; i < ARRAYS; ++i) arrays += src[i] != nullptr;
        tc::mbar_arrive_expect_tx(bar, arrays * row_bytes);
        tc::bulk_load(tc::smem_u32(ring_x) + sx * row_bytes, a.x + (size_t)t * a.n, row_bytes, bar);
        for (int i = 0; i < ARRAYS; ++i)
            if (src[i]) tc::bulk_load(to + i * row_bytes, src[i] + (size_t)t * a.n, row_bytes, bar);
    };
    if (STAGES && threadIdx.x == 0)
        for (int i = 0; i < STAGES; ++i) fetch(blockIdx.x + i * gridDim.x, i, i);
    const bool want_post = a.dpost_weight != nullptr, want_pre = a.dpre_weight != nullptr;
    const bool want_gate = BY_ELEMENT && a.dgate && a.gate_shape == MOE_GATE_CHANNEL;
    const bool full = BY_ELEMENT && a.dgate && a.gate_shape == MOE_GATE_FULL;
    const F2 scale2 = f2(a.scale, a.scale);
    const float inv_n = 1.0f / (float)a.n;
    constexpr bool kKeep = TPR * BLOCKS <= 512;
    const Weights<kKeep> post(a.post_weight, seg, on, a.weight_offset), pre(a.pre_weight, seg, on, a.weight_offset);
    float4 *const mine = sums + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 6; ++i) mine[i * TPR] = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint4 channel_gate = BY_ELEMENT && !gate_rows && on ? load8(a.gate, seg) : zero4();
    RawRow next;
    if (!kJoint) next = load_row(a, blockIdx.x, nseg, seg, on);
    int parity = 0, st = 0, sx = 0, t = blockIdx.x;
    uint32_t ph = 0;
    // A wait that runs out is met by all threads behind the next barrier; until then they compute with what is there.  A thread ahead of
    // the others may give up on a later row before they have looked: that is the other flag, so that all leave behind the same barrier.
    auto await = [&](int at, uint32_t phase, int which) {
        if (!tc::mbar_wait(tc::smem_u32(&landed[at]), phase, kWaitPolls, nullptr)) failed[which] = 1;
    };
    auto given_up = [&](int which) { return *static_cast<volatile int *>(&failed[which]) != 0; };
    auto from_ring = [&](RawRow &r, int at, int at_x) {
        const uint8_t *const row = ring + at * ARRAYS * row_bytes;
        r.x = on ? ring8(ring_x, at_x, nseg, seg) : zero4();
        r.s = on ? ring8(row, 0, nseg, seg) : zero4();
        r.dy = on && a.dy ? ring8(row, 1, nseg, seg) : zero4();
    };
    auto row_gate_of = [&](int row) { return !BY_ELEMENT && a.gate_shape == MOE_GATE_ROW && row < a.T ? bf16_bits_to_float(a.gate[row]) : 0.f; };
    // a thread's part of what needs only the inputs: sums of s^2, dy w s and x^2
    auto first_sums = [&](const RawRow &r, float &ss_of, float &m_of, float &xx_of) {
        F2 ss = f2(0.f, 0.f), m = ss, xx = ss;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 s = pair_of(r.s, i), x = pair_of(r.x, i);
            ss = fma2(s, s, ss);
            m = fma2(mul2(pair_of(r.dy, i), pre[i]), s, m);
            xx = fma2(x, x, xx);
        }
        ss_of = sum2(ss);
        m_of = sum2(m);
        xx_of = sum2(xx);
    };
    uint4 late_ds = zero4(), late_gate = zero4();
    auto load_late = [&](int row) {
        if (!kLate || !on) return;
        if (a.dsum) late_ds = load8(a.dsum + (size_t)row * a.n, seg);
        if (gate_rows) late_gate = load8(a.gate + (size_t)row * a.n, seg);
    };
    float v[3] = {0.f, 0.f, 0.f}, gate_ahead = 0.f;
    bool broken = false;
    if constexpr (kJoint) {
        RawRow raw;
        gate_ahead = row_gate_of(t);
        load_late(t);
        await(0, 0, 1);                                        // (there are no more blocks than rows)
        from_ring(raw, 0, 0);
        first_sums(raw, v[0], v[1], v[2]);
        row_sums<TPR>(v, buf[1][0]);
        broken = given_up(1);
    }
    for (; !broken && t < a.T; t += gridDim.x, parity ^= 1) {
        RawRow raw;
        if constexpr (kJoint) {
            const uint8_t *const row = ring + st * ARRAYS * row_bytes;
            raw.row_gate = gate_ahead;
            from_ring(raw, st, sx);
            if (kLate) {
                raw.ds = late_ds;
                raw.gate = gate_rows ? late_gate : channel_gate;
            } else {
                raw.ds = on && a.dsum ? ring8(row, 2, nseg, seg) : zero4();
                raw.gate = gate_rows ? (on ? ring8(row, 3, nseg, seg) : zero4()) : channel_gate;
            }
        } else {
            raw = next;
            next = load_row(a, t + gridDim.x, nseg, seg, on);
            first_sums(raw, v[0], v[1], v[2]);
            row_sums<TPR>(v, buf[parity][0]);
        }
        const size_t at = (size_t)t * nseg + seg;
        const float rx = a.post_norm ? rsqrtf(v[2] * inv_n + a.eps) : 1.0f;
        const float rs = a.dy ? rsqrtf(v[0] * inv_n + a.eps) : 0.0f, ms = -v[1] * inv_n * rs * rs * rs;
        float2 row_f = make_float2(1.f, 0.f);
        if (!BY_ELEMENT && a.gate_shape == MOE_GATE_ROW) row_f = act_slope(a.act, raw.row_gate);
        const F2 rs2 = f2(rs, rs), ms2 = f2(ms, ms);            // -rs^3 mean(dy w s): what s is multiplied by
        const F2 rx2 = f2(rx, rx), row2 = f2(row_f.x, row_f.x);
        F2 e[4], m = f2(0.f, 0.f), db = m;
        uint32_t wd[4], wg[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            F2 add[3][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = 2 * h + j;
                const F2 s = pair_of(raw.s, i), dr = mul2(pair_of(raw.dy, i), rs2);
                F2 d = pair_of(raw.ds, i);
                if (a.dy) d = fma2(s, ms2, fma2(dr, pre[i], d));
                add[1][j] = mul2(dr, s);
                wd[i] = pack_pair(d);
                const F2 x = mul2(pair_of(raw.x, i), rx2), b = mul2(x, post[i]), ds = mul2(d, scale2);
                if (BY_ELEMENT) {
                    F2 f, slope;
                    gate_pair<ACT>(pair_of(raw.gate, i), f, slope);
                    add[2][j] = mul2(mul2(ds, b), slope);
                    wg[i] = pack_pair(add[2][j]);
                    e[i] = mul2(ds, f);
                } else {
                    db = fma2(ds, b, db);
                    e[i] = mul2(ds, row2);
                    add[2][j] = f2(0.f, 0.f);
                    wg[i] = 0;
                }
                add[0][j] = mul2(e[i], x);
                m = fma2(e[i], b, m);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k == 0 ? !want_post : k == 1 ? !want_pre : !want_gate) continue;
                float4 *const p = mine + (2 * k + h) * TPR;
                const float4 o = *p;
                const float2 lo = unf2(add2(f2(o.x, o.y), add[k][0])), hi = unf2(add2(f2(o.z, o.w), add[k][1]));
                *p = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        if (on && a.dresidual) reinterpret_cast<uint4 *>(a.dresidual)[at] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
        if (on && full) reinterpret_cast<uint4 *>(a.dgate)[at] = make_uint4(wg[0], wg[1], wg[2], wg[3]);
        float mean = 0.f;
        if constexpr (kJoint) {
            float u[4] = {0.f, 0.f, 0.f, sum2(m)}, sum_db = sum2(db);
            if (t + (int)gridDim.x < a.T) {
                const int after = st + 1 == STAGES ? 0 : st + 1, after_x = sx == STAGES ? 0 : sx + 1;
                RawRow r;
                gate_ahead = row_gate_of(t + gridDim.x);
                load_late(t + gridDim.x);
                await(after, after ? ph : ph ^ 1, parity);
                from_ring(r, after, after_x);
                first_sums(r, u[0], u[1], u[2]);
            }
            row_sums<TPR>(u, buf[parity][0], BY_ELEMENT ? nullptr : &sum_db, buf[parity][1]);
            broken = given_up(parity);
            if (broken) break;
            // every thread is past the row before, whose x is free, and needs nothing but x of this row
            if (threadIdx.x == 0) fetch(t + STAGES * gridDim.x, st, sx ? sx - 1 : STAGES);
            v[0] = u[0];
            v[1] = u[1];
            v[2] = u[2];
            mean = -u[3] * inv_n;
            if (!BY_ELEMENT && a.gate_shape == MOE_GATE_ROW && a.dgate && threadIdx.x == 0) static_cast<float *>(a.dgate)[t] = sum_db * row_f.y;
        } else if (BY_ELEMENT) {
            float u[1] = {sum2(m)};
            if (a.post_norm) row_sums<TPR>(u, buf[parity][1]);
            mean = -u[0] * inv_n;
        } else if (a.post_norm || a.gate_shape == MOE_GATE_ROW) {
            float u[2] = {sum2(m), sum2(db)};
            row_sums<TPR>(u, buf[parity][1]);
            if (a.gate_shape == MOE_GATE_ROW && a.dgate && threadIdx.x == 0) static_cast<float *>(a.dgate)[t] = u[1] * row_f.y;
            mean = -u[0] * inv_n;
        }
        if (a.post_norm) {
            if (kJoint) raw.x = on ? ring8(ring_x, sx, nseg, seg) : zero4();
            const F2 mean2 = f2(mean * rx, mean * rx);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = mul2(fma2(pair_of(raw.x, i), mean2, mul2(e[i], post[i])), rx2);
        }
        if (on) reinterpret_cast<uint4 *>(a.dx)[at] = make_uint4(pack_pair(e[0]), pack_pair(e[1]), pack_pair(e[2]), pack_pair(e[3]));
        if (kJoint) {
            if (++st == STAGES) {
                st = 0;
                ph ^= 1;
            }
            if (++sx > STAGES) sx = 0;
        }
    }
    if (STAGES && broken) {
        // nothing is left on its way into this block's shared memory: the rows that were asked for, this one first
        if (threadIdx.x == 0) {
            record_status(a.status, MOE_ERR_TIMEOUT);
            for (int i = 0; i < STAGES && t + i * gridDim.x < a.T; ++i) {
                tc::mbar_wait(tc::smem_u32(&landed[st]), ph, kWaitPolls, nullptr);
                if (++st == STAGES) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        return;
    }
    if (!on) return;
    float *const out = a.partial + (size_t)blockIdx.x * 3 * a.n + 8 * seg;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (k == 0 ? want_post : k == 1 ? want_pre : want_gate) *reinterpret_cast<float4 *>(out + k * a.n + 4 * h) = mine[(2 * k + h) * TPR];
}

// Adds up the blocks' sums: a block has 32 columns of one of the three gradients, a warp every kWarps-th block,
// kFlight loads on their way at once.
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) gated_norm_sum_kernel(const __grid_constant__ GatedNormArgs a, int blocks)
{
    constexpr int kFlight = 10;                                // the 152 blocks of a wide row over 16 warps
    __shared__ float part[kWarps][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *const out = which == 0 ? a.dpost_weight : which == 1 ? a.dpre_weight
                       : a.gate_shape == MOE_GATE_CHANNEL ? static_cast<float *>(a.dgate) : nullptr;
    if (!out) return;
    float v = 0.f;
    if (col < a.n) {
        const float *p = a.partial + (size_t)which * a.n + col;
        for (int b = warp; b < blocks; b += kFlight * kWarps) {
            float x[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) x[i] = b + i * kWarps < blocks ? p[(size_t)(b + i * kWarps) * 3 * a.n] : 0.f;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) v += x[i];
        }
    }
    part[warp][lane] = v;
    __syncthreads();
    if (warp) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += part[i][lane];
    if (col < a.n) out[col] = v;
}

// Threads of a block of the backward pass, blocks an SM, stages of its rings and arrays of a place.  Narrow rows (threads, blocks): 16384 x 1024 in 4 blocks
// through registers 60 us, 3 or 5 70 and 63, 6 with rings 57, but a gate per channel 44 in 4 and 50 in 6.  2560 columns in two blocks
// of 320 61 us for 8192 rows, in one of 512 106; 3192 in two of 416 44 us for 3469 rows, in one of 512 51.
// With two arrays a place more blocks fit: 4096 columns in two blocks of 512 and 64 registers 87 us for 8192 rows with a gate per
// token (one block 99), but 62 for 4096 rows with a gate per element (54), 16384 x 2048 in four blocks 107 (95); 6144 columns, three stages of two
// arrays 76.5, two of four 80; 8192 columns 122, with everything through registers and no rings 154.
constexpr int kGradPlans[][4] = {{32, 16, 0, 0}, {64, 8, 0, 0}, {128, 4, 0, 0}, {256, 3, 2, 4}, {320, 2, 3, 4},
                                 {416, 2, 2, 4}, {512, 1, 4, 4}, {640, 1, 3, 4}, {768, 1, 3, 2}, {1024, 1, 2, 2}};
int grad_plan(int n)
{
    int i = 0;
    while (kGradPlans[i][0] * 8 < n) ++i;
    return i;
}
// Blocks of the backward pass, the same on any device: all that fit on 152 SMs, of at least two rows each once there are three
// blocks an SM, since each block's sums are written and read again (1500 x 256 11.6 -> 7.8 us, 3000 x 64 11.2 -> 9.3; 333 x 64 in
// blocks of two rows 4.6 -> 5.6).
int grad_blocks(int T, int n)
{
    const int most = 152 * kGradPlans[grad_plan(n)][1], some = T < 3 * 152 ? T : 3 * 152, each = T / 2 > some ? T / 2 : some;
    return each < most ? each : most;
}
template <int I, bool BY_ELEMENT, int ACT>
cudaError_t launch_plan(const GatedNormArgs &a, int blocks, cudaStream_t st)
{
    constexpr int kThreads = kGradPlans[I][0], kStages = kGradPlans[I][2], kArrays = kGradPlans[I][3], kRing = kStages ? (1 + kArrays) * kStages + 1 : 0, kMost = (6 + kRing) * 16 * kThreads;
    static_assert((kMost + 2 * kThreads + 1024 + 64) * kGradPlans[I][1] <= 228 * 1024, "shared memory");
    auto k = gated_norm_grad_kernel<kThreads, kGradPlans[I][1], kStages, kArrays, BY_ELEMENT, ACT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = set_shared(k, kMost, ready);
    return e != cudaSuccess ? e : launch_dependent(k, blocks, kThreads, 6 * 16 * kThreads + kRing * 2 * a.n, st, a);
}
template <int I>
cudaError_t launch_backward(const GatedNormArgs &a, int blocks, cudaStream_t st)
{
    if (a.gate_shape < MOE_GATE_CHANNEL) return launch_plan<I, false, MOE_ACT_NONE>(a, blocks, st);
    if (a.act == MOE_ACT_SILU) return launch_plan<I, true, MOE_ACT_SILU>(a, blocks, st);
    if (a.act == MOE_ACT_SIGMOID) return launch_plan<I, true, MOE_ACT_SIGMOID>(a, blocks, st);
    return launch_plan<I, true, MOE_ACT_NONE>(a, blocks, st);
}

template <int TPR, int CH>
cudaError_t launch_forward(const GatedNormArgs &a, cudaStream_t st)
{
    const int rows = block_of(TPR) / TPR;
    return launch_dependent(gated_norm_kernel<TPR, CH>, (unsigned)((a.T + rows - 1) / rows), block_of(TPR), 0, st, a);
}

}  // namespace

size_t gated_norm_partials(int T, int n) { return (size_t)grad_blocks(T, n) * 3 * n; }

cudaError_t launch_gated_norm(const GatedNormArgs &a, cudaStream_t st)
{
    const int nseg = a.n / 8;
    if (nseg <= 32) return launch_forward<32, 1>(a, st);
    if (nseg <= 128) return launch_forward<128, 1>(a, st);
    if (nseg <= 256 && a.T >= 512) return launch_forward<128, 2>(a, st);
    if (nseg <= 256) return launch_forward<256, 1>(a, st);
    if (nseg <= 512) return launch_forward<256, 2>(a, st);
    return launch_forward<512, 2>(a, st);
}

cudaError_t launch_gated_norm_grad(const GatedNormArgs &a, cudaStream_t st)
{
    const int blocks = grad_blocks(a.T, a.n);
    cudaError_t e = cudaErrorInvalidValue;
    switch (grad_plan(a.n)) {
    case 0: e = launch_backward<0>(a, blocks, st); break;
    case 1: e = launch_backward<1>(a, blocks, st); break;
    case 2: e = launch_backward<2>(a, blocks, st); break;
    case 3: e = launch_backward<3>(a, blocks, st); break;
    case 4: e = launch_backward<4>(a, blocks, st); break;
    case 5: e = launch_backward<5>(a, blocks, st); break;
    case 6: e = launch_backward<6>(a, blocks, st); break;
    case 7: e = launch_backward<7>(a, blocks, st); break;
    case 8: e = launch_backward<8>(a, blocks, st); break;
    case 9: e = launch_backward<9>(a, blocks, st); break;
    }
    if (e != cudaSuccess || !(a.dpost_weight || a.dpre_weight || (a.dgate && a.gate_shape == MOE_GATE_CHANNEL))) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((a.n + 31) / 32, 3);
    const bool few = blocks <= 160;
    cfg.blockDim = dim3(few ? 512 : 1024);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t s = cudaLaunchKernelEx(&cfg, few ? gated_norm_sum_kernel<16> : gated_norm_sum_kernel<32>, a, blocks);
    return s == cudaSuccess ? s : cudaGetLastError();
}

}  // namespace qmoe
