// Grouped products of few block-scaled rows, a row at a time.
//
//   acc[r, n] = sum_b sa[r, b] sw[g, n, b] sum_{j in block b} a[r, j] w[g, n, j]
//   y[r, n]   = row_scale[r] alpha[g] acc[r, n]
//   h[r, n]   = silu(gate) up of two such products, quantised
//
// A tensor-core tile (scaled_gemm.cu) takes 0.2 to 0.3 us a K step for one row as for 128, one step behind the other.
// Here a call asks for all of its weights at once, by as many warps as there are outputs and K slices to share out, and
// costs its launch, a latency of memory, the conversions and one exchange of sums.
//
// The products are m16n8k16 of fp16 (both operands' codes are exact in it, and so are the products in fp32): 16
// weight rows against one row of activations, each lane's 32 elements in a column of their own and zeros in the others',
// so that a column ends as the sum over one block, which its scales multiply in fp32.  The conversion of the codes (a
// byte's two codes an instruction, 64 lanes a cycle) is most of the work: a warp has two tiles of weights for each
// conversion of its activations.
//
// 1 x 4096 x 2048: 2.8 us in either format (1.7 TB/s from L2), against 4.5 (NVFP4) and 5.9 of a tile; 1 x 4096 x 8192 NVFP4 6.7
// against 8.5; 1 x 4096 x 8192 MXFP8 5.3 (4.9 with the blocks' scales multiplied with each other first, which leaves fp32's
// range where the sum does not).  One token of 9 experts, hidden 2048, inter 512, NVFP4: 4.5 and 3.7 us against 7.4 and 4.4.  1.9 us are
// launch to launch, 0.4 the search for a row's group.  Ways that were slower, where this took 3.0 us: packed fp16 FMAs
// (4.0), byte dot products of looked-up codes (4.3), m16n8k32 of E4M3 (4.7), the activations converted once into
// shared memory (3.8); the scales fetched by column tiles into shared memory cost 0.5 us at K = 512.
#include "scaled.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

constexpr int kOutputs = 32;                       // outputs of a CTA: whole blocks of h
constexpr int kChunk = 128;                        // elements of a warp's step along K: 32 of each of four lanes

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

// Eight E2M1 codes to four pairs.
__device__ __forceinline__ void from_e2m1x8(uint32_t q, uint32_t (&h)[4])
{
    asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\ncvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
}
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return h;
}
// c += a b: 16 x 16 by 16 x 8; a's rows i, i + 8 and b's column i in lane 4 i + q, places 2 q, 2 q + 1, 2 q + 8, 2 q + 9.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The scales of a lane's 32 elements: two E4M3 bytes, or one E8M0 byte (s[0]).
template <bool NV>
__device__ __forceinline__ void from_scales(uint32_t b, float (&s)[2])
{
    uint32_t h;
    if (NV) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        s[0] = v.x;
        s[1] = v.y;
    } else {
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
        s[0] = __uint_as_float(h << 16);
    }
}
// acc + d fx fw.  Two E4M3 scales have an exact product; that of two powers of two can leave fp32's range where the sum
// does not (and make a NaN of a sum of zero), so the smaller one comes first: d is a multiple of 2^-10, which 2^-127
// takes to a subnormal exactly, and what then overflows or is rounded does so in the sum too.  A NaN scale stays.
template <bool NV>
__device__ __forceinline__ float scaled_add(float d, float fx, float fw, float acc)
{
    if (NV) return fmaf(d, fx * fw, acc);
    float lo, hi;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(fx), "f"(fw));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(fx), "f"(fw));
    return fmaf(d * lo, hi, acc);
}
template <bool NV>
__device__ __forceinline__ uint32_t load_scales(const uint8_t *p)
{
    return NV ? *reinterpret_cast<const uint16_t *>(p) : *p;
}

// A CTA has 32 outputs of one row.  A warp has two tiles of 16 weight rows, the CTA's or a gate tile and its up tile; S
// warps share them, taking their steps in turn.
template <int FMT, bool DUAL, int S, int kAhead>
__global__ void __launch_bounds__(32 * (DUAL ? 2 : 1) * S, DUAL && S == 4 && kAhead == 2 ? 2 : 1)
scaled_vec_kernel(const __grid_constant__ ScaledGemmArgs a, int blocks)
{
    constexpr bool kNv = FMT == MOE_SCALED_NVFP4;
    constexpr int kMats = DUAL ? 2 : 1, kWarps = kMats * S, kThreads = 32 * kWarps, kX = kNv ? 1 : 2;
    __shared__ uint32_t count[kWarps], begin[kWarps];
    __shared__ float part[S][kMats][kOutputs];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x / blocks, block = blockIdx.x - row * blocks, n0 = block * kOutputs;
    pdl_wait();

    // the row's group: as many groups start at or before it, less one, the last of them at `start`; malformed offsets
    // counted in the upper half
    int g = 0, start = 0;
    if (a.offsets) {
        uint32_t c = 0, m = 0;
        constexpr int kPer = kThreads < 512 ? 512 / kThreads : 1;       // loads on their way together
        for (int i0 = threadIdx.x; i0 < a.G; i0 += kThreads * kPer) {
            int o[kPer], next[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = i0 + j * kThreads;
                o[j] = i < a.G ? a.offsets[i] : a.R;
                next[j] = i + 1 < a.G ? a.offsets[i + 1] : a.R;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                m = o[j] <= row ? max(m, (uint32_t)o[j]) : m;
                c += (o[j] <= row) + ((o[j] < 0 || o[j] > a.R || next[j] < o[j]) ? 1u << 16 : 0u);
            }
        }
        c = __reduce_add_sync(0xFFFFFFFFu, c);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) {
            count[warp] = c;
            begin[warp] = m;
        }
        __syncthreads();
        c = m = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            c += count[i];
            m = max(m, begin[i]);
        }
        if (c >> 16) {
            if (blockIdx.x == 0 && threadIdx.x == 0) record_status(a.status, MOE_ERR_DEVICE);
            return;
        }
        if (c == 0) return;                                                       // before the first group
        g = (int)c - 1;
        start = (int)m;
    }

    const int slice = warp / kMats, first = DUAL ? (warp & 1) * 16 : 0;
    const int i = lane >> 2, q = lane & 3;                 // the lane's weight rows i and i + 8, its 32 elements of a step
    const int steps = (a.K + kChunk - 1) / kChunk, ct = scaled_col_tiles(FMT, a.K);
    const size_t wbytes = (size_t)a.K / 2, wrt = (a.N + kScaleRows - 1) / kScaleRows;
    const long long srow = (long long)group_row_tile(start, g) * kScaleRows + (row - start);
    const int first_block = kNv ? 2 * q : q;               // of a step
    const uint8_t *w[2][2], *ws[2][2];                     // [tile][row i, i + 8]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            // rows past the last are read as the last and not written
            const int m = DUAL ? t : 0, r = min(n0 + first + (DUAL ? 0 : 16 * t) + 8 * o + i, a.N - 1);
            w[t][o] = a.w_codes[m] + ((size_t)g * a.N + r) * wbytes + 16 * q;
            ws[t][o] = a.w_scales[m] + (size_t)g * wrt * ct * kScaleTile + scale_at(r, first_block, ct);
        }
    const uint8_t *const xc = a.a_codes + (kNv ? (size_t)row * wbytes + 16 * q : (size_t)row * a.K + 32 * q);
    const uint8_t *const xs = a.a_scales + scale_at(srow, first_block, ct);
    // column 2 q is for the lanes q's elements: the lane of it that has them fills it in
    const bool fills = i == 2 * q;
    // what the outputs are multiplied by, on its way under the products
    const float rs = a.a_row_scale ? a.a_row_scale[row] : 1.0f;
    const float alpha0 = a.alpha[0] ? a.alpha[0][g] : 1.0f, alpha1 = DUAL && a.alpha[1] ? a.alpha[1][g] : 1.0f;
    const float hg = DUAL && kNv ? a.h_gscale[g] : 1.0f;

    float acc[2][2] = {};
    for (int c0 = slice; c0 < steps; c0 += S * kAhead) {
        uint4 u[kAhead][2][2], x[kAhead][kX];
        uint32_t e[kAhead][2][2], ex[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c = c0 + k * S;
            const bool live = c * kChunk + 32 * q < a.K;
            const size_t wb = (size_t)c * (kChunk / 2), sb = (size_t)c * (kNv ? 2 : 1) * kScaleTile;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    u[k][t][o] = live ? *reinterpret_cast<const uint4 *>(w[t][o] + wb) : zero;
                    e[k][t][o] = live ? load_scales<kNv>(ws[t][o] + sb) : 0;
                }
            ex[k] = live ? load_scales<kNv>(xs + sb) : 0;
#pragma unroll
            for (int j = 0; j < kX; ++j)
                x[k][j] = live && fills ? reinterpret_cast<const uint4 *>(xc + wb * kX)[j] : zero;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (c0 + k * S >= steps) break;
            float d[2][2][4] = {};                         // [tile][first and second half of the lanes' elements]
            const uint32_t y[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][kX - 1].x, x[k][kX - 1].y, x[k][kX - 1].z, x[k][kX - 1].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t b[4];
                if (kNv) {
                    from_e2m1x8(y[j], b);
                } else {
#pragma unroll
                    for (int o = 0; o < 4; ++o) b[o] = from_e4m3x2(y[2 * j + o / 2] >> (16 * (o & 1)) & 0xFFFFu);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t h0[4], h1[4];
                    from_e2m1x8((&u[k][t][0].x)[j], h0);
                    from_e2m1x8((&u[k][t][1].x)[j], h1);
                    mma_f16(d[t][kNv ? j >> 1 : 0], h0[0], h1[0], h0[1], h1[1], b[0], b[1]);
                    mma_f16(d[t][kNv ? j >> 1 : 0], h0[2], h1[2], h0[3], h1[3], b[2], b[3]);
                }
            }
            float fx[2];
            from_scales<kNv>(ex[k], fx);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    float f[2];
                    from_scales<kNv>(e[k][t][o], f);
#pragma unroll
                    for (int j = 0; j < (kNv ? 2 : 1); ++j) acc[t][o] = scaled_add<kNv>(d[t][j][2 * o], fx[j], f[j], acc[t][o]);
                }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
#pragma unroll
            for (int m = 1; m < 4; m <<= 1) acc[t][o] += __shfl_xor_sync(0xFFFFFFFFu, acc[t][o], m);
            if (q == 0) part[slice][DUAL ? t : 0][first + (DUAL ? 0 : 16 * t) + 8 * o + i] = acc[t][o];
        }
    __syncthreads();
    if (warp) return;
    float sum[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
        sum[m] = 0.f;
#pragma unroll
        for (int j = 0; j < S; ++j) sum[m] += part[j][m][lane];
    }
    if constexpr (!DUAL) {
        const float y = sum[0] * (rs * alpha0);
        const size_t at = (size_t)row * a.N + n0 + lane;
        if (n0 + lane < a.N) {
            if (a.y_f32) static_cast<float *>(a.y)[at] = y;
            else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(y);
        }
    } else {
        // a lane an output: the block's largest magnitude, its scale, and the codes
        constexpr int kBlk = scaled_block(FMT);
        const float h = silu(sum[0] * (rs * alpha0)) * (sum[kMats - 1] * (rs * alpha1));
        uint32_t m = __float_as_uint(h) & 0x7FFFFFFFu;
#pragma unroll
        for (int d = kBlk / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        float inv;
        uint32_t sc;
        if (kNv) {
            sc = nvfp4_scale(m, __fdiv_rn(1.0f, hg), inv);
        } else {
            sc = pow2_scale<MOE_SCALED_MXFP8>(m);
            inv = pow2_inverse(sc);
        }
        const float e = h * inv;
        if (kNv) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, e, (8 * lane + k) & 31);
            if (lane < 4) reinterpret_cast<uint32_t *>(a.h_codes + ((size_t)row * a.N + n0) / 2)[lane] = to_e2m1x8(v);
        } else {
            a.h_codes[(size_t)row * a.N + n0 + lane] = (uint8_t)to_e4m3x2(0.f, e);
        }
        if (lane % kBlk == 0) a.h_scales[scale_at(srow, (n0 + lane) / kBlk, scaled_col_tiles(FMT, a.N))] = (uint8_t)sc;
    }
}

template <int FMT, bool DUAL, int S, int A>
cudaError_t launch_vec(const ScaledGemmArgs &a, cudaStream_t st)
{
    const int blocks = (a.N + kOutputs - 1) / kOutputs;
    const unsigned grid = (unsigned)(a.R * blocks);
    // Where there is an SM for every CTA, shared memory that keeps a second one off: two would land on some SMs
    // all the same (1 x 4096 x 2048 NVFP4 3.5 us without, 3.0 with; the SwiGLU of one token 6.3 and 5.0).
    constexpr int kWholeSm = 116 * 1024;
    const size_t smem = grid <= (unsigned)device_sm_count() ? kWholeSm : 0;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = set_shared(scaled_vec_kernel<FMT, DUAL, S, A>, kWholeSm, ready);
    if (e != cudaSuccess) return e;
    return launch_dependent(scaled_vec_kernel<FMT, DUAL, S, A>, grid, 32 * (DUAL ? 2 : 1) * S, smem, st, a, blocks);
}
template <int FMT, bool DUAL>
cudaError_t launch_fmt(const ScaledGemmArgs &a, cudaStream_t st)
{
    // Warps that share a tile's steps, and steps that each loads together.  Short sums: more warps while all CTAs
    // run at once (9 rows of experts' down products behind their SwiGLU 8.4 us with (4, 1), 9.0 with (2, 2); 18 rows 5.5 and 4.2 by
    // themselves).  The SwiGLU with an SM for every CTA, few warps that load far ahead, else two CTAs an SM: one token's 4.7
    // us with (4, 4), 5.0 with (8, 2), 5.2 with (4, 2); two tokens' 8.8 with (8, 2), 6.7 with (4, 2).
    const int steps = (a.K + kChunk - 1) / kChunk, sms = device_sm_count();
    const long long ctas = (long long)a.R * ((a.N + kOutputs - 1) / kOutputs);
    if (steps <= 4) return ctas <= 4 * sms ? launch_vec<FMT, DUAL, 4, 1>(a, st) : launch_vec<FMT, DUAL, 2, 2>(a, st);
    if (steps <= 8 || (DUAL && ctas > sms)) return launch_vec<FMT, DUAL, 4, 2>(a, st);
    if constexpr (DUAL) return launch_vec<FMT, DUAL, 4, 4>(a, st);
    else return launch_vec<FMT, DUAL, 8, 2>(a, st);
}

}  // namespace

cudaError_t launch_scaled_vec(const ScaledGemmArgs &a, int fmt, bool swiglu, cudaStream_t st)
{
    if (fmt == MOE_SCALED_NVFP4)
        return swiglu ? launch_fmt<MOE_SCALED_NVFP4, true>(a, st) : launch_fmt<MOE_SCALED_NVFP4, false>(a, st);
    return swiglu ? launch_fmt<MOE_SCALED_MXFP8, true>(a, st) : launch_fmt<MOE_SCALED_MXFP8, false>(a, st);
}

}  // namespace qmoe
