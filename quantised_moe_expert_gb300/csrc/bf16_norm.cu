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
// A thread keeps 8 consecutive elements of a row in registers from the one read to the write; sums over the row go through
// shuffles and shared memory.  Backward, a block walks over every gridDim-th row with the sums over rows of its threads'
// columns in registers, writes them as one row of the workspace, and a second launch adds those up in a fixed order.
#include "bf16.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

constexpr int kMaxThreads = kNormMaxN / 8;

__device__ __forceinline__ void unpack(uint4 u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack(const float (&v)[8])
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ uint4 load8(const uint16_t *p, size_t seg) { return reinterpret_cast<const uint4 *>(p)[seg]; }

// Sum of v over the block (blockDim a multiple of 32); buf: 32 floats that no thread still reads.
__device__ __forceinline__ float block_sum(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += buf[i];
    return s;
}

// offset + weight of this thread's elements, or ones.
__device__ __forceinline__ void weights(const uint16_t *w, float offset, int seg, bool on, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
    if (!w || !on) return;
    unpack(load8(w, seg), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += offset;
}

__global__ void __launch_bounds__(kMaxThreads) gated_norm_kernel(const __grid_constant__ GatedNormArgs a)
{
    __shared__ float buf[2][32];
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, seg = threadIdx.x, t = blockIdx.x;
    const bool on = seg < nseg;
    const size_t at = (size_t)t * nseg + seg;
    float x[8] = {}, r[8] = {}, g[8], w[8];
    if (on) unpack(load8(a.x, at), x);
    if (on && a.residual) unpack(load8(a.residual, at), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = a.scale;
    if (on && a.gate_shape != MOE_GATE_NONE) {
        if (a.gate_shape == MOE_GATE_ROW) {
            const float f = act_value(a.act, bf16_bits_to_float(a.gate[t]));
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = f * a.scale;
        } else {
            unpack(load8(a.gate, a.gate_shape == MOE_GATE_FULL ? at : seg), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = act_value(a.act, g[e]) * a.scale;
        }
    }
    if (a.post_norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float rx = rsqrtf(block_sum(ss, buf[0]) / (float)a.n + a.eps);
        weights(a.post_weight, a.weight_offset, seg, on, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * rx * w[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = fmaf(g[e], x[e], r[e]);
    const uint4 s = pack(r);
    if (on && a.sum) reinterpret_cast<uint4 *>(a.sum)[at] = s;
    if (!a.y) return;
    unpack(s, r);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[e], r[e], ss);
    const float rs = rsqrtf(block_sum(on ? ss : 0.f, buf[1]) / (float)a.n + a.eps);
    weights(a.pre_weight, a.weight_offset, seg, on, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = r[e] * rs * w[e];
    if (on) reinterpret_cast<uint4 *>(a.y)[at] = pack(r);
}

__global__ void __launch_bounds__(kMaxThreads) gated_norm_grad_kernel(const __grid_constant__ GatedNormArgs a)
{
    __shared__ float buf[5][32];
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, seg = threadIdx.x;
    const bool on = seg < nseg;
    float post[8], pre[8], gate[8], slope[8];
    weights(a.post_weight, a.weight_offset, seg, on, post);
    weights(a.pre_weight, a.weight_offset, seg, on, pre);
#pragma unroll
    for (int e = 0; e < 8; ++e) gate[e] = 1.f, slope[e] = 0.f;
    if (on && a.gate_shape == MOE_GATE_CHANNEL) {
        unpack(load8(a.gate, seg), gate);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = act_slope(a.act, gate[e]);
            gate[e] = f.x;
            slope[e] = f.y;
        }
    }
    float sum_pre[8] = {}, sum_post[8] = {}, sum_gate[8] = {};
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t at = (size_t)t * nseg + seg;
        float x[8] = {}, s[8] = {}, dy[8] = {}, d[8] = {};
        if (on) unpack(load8(a.x, at), x);
        if (on) unpack(load8(a.sum, at), s);
        if (on && a.dy) unpack(load8(a.dy, at), dy);
        if (on && a.dsum) unpack(load8(a.dsum, at), d);
        if (a.gate_shape == MOE_GATE_FULL && on) {
            unpack(load8(a.gate, at), gate);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = act_slope(a.act, gate[e]);
                gate[e] = f.x;
                slope[e] = f.y;
            }
        }
        float row_slope = 0.f;
        if (a.gate_shape == MOE_GATE_ROW) {
            const float2 f = act_slope(a.act, bf16_bits_to_float(a.gate[t]));
            row_slope = f.y;
#pragma unroll
            for (int e = 0; e < 8; ++e) gate[e] = f.x;
        }
        if (a.dy) {
            float ss = 0.f, m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(s[e], s[e], ss);
                m = fmaf(dy[e] * pre[e], s[e], m);
            }
            const float rs = rsqrtf(block_sum(ss, buf[0]) / (float)a.n + a.eps);
            m = block_sum(m, buf[1]) / (float)a.n * rs * rs;            // mean(dy w s^) rs
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum_pre[e] = fmaf(dy[e], s[e] * rs, sum_pre[e]);
                d[e] += rs * dy[e] * pre[e] - s[e] * rs * m;
            }
        }
        if (on && a.dresidual) reinterpret_cast<uint4 *>(a.dresidual)[at] = pack(d);
        float rx = 1.f;
        if (a.post_norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            rx = rsqrtf(block_sum(ss, buf[2]) / (float)a.n + a.eps);
        }
        float dg[8], row = 0.f, m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= rx;
            const float ds = a.scale * d[e], db = ds * x[e] * post[e];
            row += db;
            dg[e] = db * slope[e];
            sum_gate[e] += dg[e];
            d[e] = ds * gate[e];
            sum_post[e] = fmaf(d[e], x[e], sum_post[e]);
            d[e] *= post[e];
            m = fmaf(d[e], x[e], m);
        }
        if (a.dgate && a.gate_shape == MOE_GATE_FULL && on) reinterpret_cast<uint4 *>(a.dgate)[at] = pack(dg);
        if (a.dgate && a.gate_shape == MOE_GATE_ROW) {
            row = block_sum(row, buf[3]);
            if (threadIdx.x == 0) static_cast<float *>(a.dgate)[t] = row * row_slope;
        }
        if (a.post_norm) {
            m = block_sum(m, buf[4]) / (float)a.n;
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = rx * (d[e] - x[e] * m);
        }
        if (on) reinterpret_cast<uint4 *>(a.dx)[at] = pack(d);
        __syncthreads();                               // the sums' buffers are the next row's
    }
    float *const out = a.partial + (size_t)blockIdx.x * 3 * a.n + 8 * seg;
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        if (a.dpost_weight) *reinterpret_cast<float4 *>(out + e) = make_float4(sum_post[e], sum_post[e + 1], sum_post[e + 2], sum_post[e + 3]);
        if (a.dpre_weight) *reinterpret_cast<float4 *>(out + a.n + e) = make_float4(sum_pre[e], sum_pre[e + 1], sum_pre[e + 2], sum_pre[e + 3]);
        if (a.dgate && a.gate_shape == MOE_GATE_CHANNEL)
            *reinterpret_cast<float4 *>(out + 2 * a.n + e) = make_float4(sum_gate[e], sum_gate[e + 1], sum_gate[e + 2], sum_gate[e + 3]);
    }
}

// Adds up the blocks' sums: a block has 32 columns of one of the three gradients, a warp every 32nd block.
__global__ void __launch_bounds__(1024) gated_norm_sum_kernel(const __grid_constant__ GatedNormArgs a, int blocks)
{
    __shared__ float part[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *const out = which == 0 ? a.dpost_weight : which == 1 ? a.dpre_weight
                       : a.gate_shape == MOE_GATE_CHANNEL ? static_cast<float *>(a.dgate) : nullptr;
    if (!out) return;
    float v = 0.f;
    if (col < a.n)
        for (int b = warp; b < blocks; b += 32) v += a.partial[(size_t)b * 3 * a.n + (size_t)which * a.n + col];
    part[warp][lane] = v;
    __syncthreads();
    if (warp) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][lane];
    if (col < a.n) out[col] = v;
}

int threads_of(int n) { return (n / 8 + 31) / 32 * 32; }
// Blocks of the backward pass: 1024 threads an SM of 152.
int grad_blocks(int T, int n)
{
    const int most = 152 * (1024 / threads_of(n) < 8 ? 1024 / threads_of(n) : 8);
    return T < most ? T : most;
}

}  // namespace

size_t gated_norm_partials(int T, int n) { return (size_t)grad_blocks(T, n) * 3 * n; }

cudaError_t launch_gated_norm(const GatedNormArgs &a, cudaStream_t st)
{
    return launch_dependent(gated_norm_kernel, (unsigned)a.T, threads_of(a.n), 0, st, a);
}

cudaError_t launch_gated_norm_grad(const GatedNormArgs &a, cudaStream_t st)
{
    const int blocks = grad_blocks(a.T, a.n);
    const cudaError_t e = launch_dependent(gated_norm_grad_kernel, blocks, threads_of(a.n), 0, st, a);
    if (e != cudaSuccess || !(a.dpost_weight || a.dpre_weight || (a.dgate && a.gate_shape == MOE_GATE_CHANNEL))) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((a.n + 31) / 32, 3);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t s = cudaLaunchKernelEx(&cfg, gated_norm_sum_kernel, a, blocks);
    return s == cudaSuccess ? s : cudaGetLastError();
}

}  // namespace qmoe
