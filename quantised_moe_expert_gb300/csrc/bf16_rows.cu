// Rows of the 16-bit operators that no product touches: token rows into expert-sorted rows, the weighted sum of a
// token's picks and its gradient, and the gradient through an activation.
//
// Bound: bytes.  A thread moves 16 bytes (8 elements) of a row at a time, so that a warp's accesses are whole lines.  Measured,
// 4096 tokens, hidden 2048, 8 picks and a shared expert: weighted sum 35 us (168 MB, 4.8 TB/s), its gradient 50 us (319 MB, 6.4 TB/s),
// gradient of a gated pair of 36864 x 512 29 us (189 MB, 6.6 TB/s); dispatch of 512 tokens 5.5 us, of one 2.4.
#include "bf16.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

constexpr int kThreads = 256;

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

// Row of slot j of token t among the expert-sorted rows (j == k: the shared expert's), -1 and a report where the
// arguments place it outside.
__device__ __forceinline__ long long slot_row(const RoutedArgs &a, int t, int j)
{
    if (j == a.k) return (long long)a.T * a.k + t;
    const int r = a.inv_perm[t * a.k + j];
    if (r >= 0 && r < a.T * a.k) return r;
    record_status(a.status, MOE_ERR_DEVICE);
    return -1;
}

constexpr int kBatch = 4;                          // slots whose rows are looked up, and read, together

__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ RoutedArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, slots = a.k + a.has_shared;
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    const int t = (int)(i / nseg), seg = (int)(i - (size_t)t * nseg);
    if (t >= a.T) return;
    const uint4 v = reinterpret_cast<const uint4 *>(a.x)[i];
    for (int j0 = 0; j0 < slots; j0 += kBatch) {
        long long row[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) row[j] = j0 + j < slots ? slot_row(a, t, j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (row[j] >= 0) reinterpret_cast<uint4 *>(a.y)[row[j] * nseg + seg] = v;
    }
}

template <int kBatch>
__global__ void __launch_bounds__(kThreads) weighted_sum_kernel(const __grid_constant__ RoutedArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, slots = a.k + a.has_shared;
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    const int t = (int)(i / nseg), seg = (int)(i - (size_t)t * nseg);
    if (t >= a.T) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < slots; j0 += kBatch) {
        long long row[kBatch];
        uint4 v[kBatch];
        float w[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            row[j] = j0 + j < slots ? slot_row(a, t, j0 + j) : -1;
            w[j] = 1.0f;
            if (a.p && row[j] >= 0) w[j] = bf16_bits_to_float(j0 + j < a.k ? a.p[t * a.k + j0 + j] : a.w_shared[t]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (row[j] >= 0) v[j] = reinterpret_cast<const uint4 *>(a.x)[row[j] * nseg + seg];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (row[j] < 0) continue;
            float f[8];
            unpack(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], f[e], acc[e]);
        }
    }
    reinterpret_cast<uint4 *>(a.y)[i] = pack(acc);
}

constexpr int kSegs = 4;                           // segments of both rows that a lane reads together

// A block a token, a warp a slot: dy's row comes from L1 for all warps but the first.
__global__ void __launch_bounds__(32 * (kMaxTopK + 1)) weighted_sum_grad_kernel(const __grid_constant__ RoutedArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int nseg = a.n / 8, t = blockIdx.x, j = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long row = lane == 0 ? slot_row(a, t, j) : 0;
    row = __shfl_sync(0xFFFFFFFFu, row, 0);
    const bool shared = j == a.k;
    float *const out = shared ? a.dw_shared : a.dp;
    float dot = 0.f;
    if (row >= 0) {
        const float w = bf16_bits_to_float(shared ? a.w_shared[t] : a.p[t * a.k + j]);
        const uint4 *dy = reinterpret_cast<const uint4 *>(a.dy) + (size_t)t * nseg;
        const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * nseg;
        uint4 *y = reinterpret_cast<uint4 *>(a.y) + row * nseg;
        for (int s0 = lane; s0 < nseg; s0 += 32 * kSegs) {
            uint4 d[kSegs], v[kSegs];
#pragma unroll
            for (int b = 0; b < kSegs; ++b) {
                const int s = s0 + 32 * b;
                d[b] = v[b] = make_uint4(0, 0, 0, 0);
                if (s < nseg) d[b] = dy[s];
                if (s < nseg && out) v[b] = x[s];
            }
#pragma unroll
            for (int b = 0; b < kSegs; ++b) {
                const int s = s0 + 32 * b;
                float f[8], r[8];
                unpack(d[b], f);
                unpack(v[b], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot = fmaf(f[e], r[e], dot);
                    f[e] *= w;
                }
                if (s < nseg) y[s] = pack(f);
            }
        }
    }
    if (!out) return;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    if (lane == 0) out[shared ? t : t * a.k + j] = dot;
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const __grid_constant__ ActGradArgs a)
{
    pdl_trigger();
    pdl_wait();
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.n / 8) return;
    float dy[8], pre[8], up[8], d[8];
    const uint4 rdy = reinterpret_cast<const uint4 *>(a.dy)[i], rpre = reinterpret_cast<const uint4 *>(a.pre)[i];
    const uint4 rup = GATED ? reinterpret_cast<const uint4 *>(a.up)[i] : make_uint4(0, 0, 0, 0);
    unpack(rdy, dy);
    unpack(rpre, pre);
    unpack(rup, up);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 f = act_slope(a.act, pre[e]);
        d[e] = GATED ? dy[e] * up[e] * f.y : dy[e] * f.y;
        up[e] = dy[e] * f.x;
    }
    reinterpret_cast<uint4 *>(a.dpre)[i] = pack(d);
    if (GATED) reinterpret_cast<uint4 *>(a.dup)[i] = pack(up);
}

unsigned blocks_of(size_t segments) { return (unsigned)((segments + kThreads - 1) / kThreads); }

}  // namespace

cudaError_t launch_dispatch(const RoutedArgs &a, cudaStream_t st)
{
    return launch_dependent(dispatch_kernel, blocks_of((size_t)a.T * (a.n / 8)), kThreads, 0, st, a);
}
cudaError_t launch_weighted_sum(const RoutedArgs &a, cudaStream_t st)
{
    // Few rows: all of a token's at once, for the shortest way (one token of 2048, 9 rows: 3.5 -> 3.1 us); many: more threads
    // with fewer (4096 tokens 35 us, 41 with 9 at once).
    const unsigned grid = blocks_of((size_t)a.T * (a.n / 8));
    return grid <= 152 ? launch_dependent(weighted_sum_kernel<9>, grid, kThreads, 0, st, a)
                       : launch_dependent(weighted_sum_kernel<kBatch>, grid, kThreads, 0, st, a);
}
cudaError_t launch_weighted_sum_grad(const RoutedArgs &a, cudaStream_t st)
{
    return launch_dependent(weighted_sum_grad_kernel, (unsigned)a.T, 32 * (a.k + a.has_shared), 0, st, a);
}
cudaError_t launch_act_grad(const ActGradArgs &a, cudaStream_t st)
{
    const unsigned grid = blocks_of(a.n / 8);
    return a.up ? launch_dependent(act_grad_kernel<true>, grid, kThreads, 0, st, a)
                : launch_dependent(act_grad_kernel<false>, grid, kThreads, 0, st, a);
}

}  // namespace qmoe
