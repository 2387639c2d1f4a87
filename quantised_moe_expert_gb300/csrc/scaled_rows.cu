// Rows to block-scaled rows: the residual add with RMSNorm, plain quantisation (activations and weights)
// and quantisation into expert-sorted rows; and the re-ordering of stored scales into scale tiles.
//
//   s = bf16(x + residual)                        (norm; what the next residual add sees)
//   v = s * rsqrt(mean(s^2) + eps) * (offset + w) (fp32; rounded once, to bf16 and to codes)
//   codes and scales of v: see scaled.cuh
//
// Bound: bytes.  TPR threads share a row and keep it in registers between the one read and the writes:
// each thread holds CH segments of 8 elements (one 16-byte load of bf16), neighbouring threads
// neighbouring segments, so loads, code stores and bf16 stores are coalesced and a block's maximum is
// one or two shuffles; the four scale bytes of a column tile are ORed over their lanes and written as
// one word.  Measured: norm of 32768 x 2048 with residual to bf16 and MXFP8 (604 MB) 89.4 us, 6.76 TB/s, the rate
// of a plain copy; 777 x 5120 7.8 us; one row 1.9 us behind another launch; 512 rows of 2048 into 9 expert-sorted
// copies each 4.0 us, 16 rows 2.6.
#include "f32x2.cuh"
#include "scaled.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kEarlyBlocks = 152;                  // one block an SM

// Sum or maximum over the TPR threads of a row; `buf` holds one value per warp.  Every thread of the
// block takes part.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (TPR == 32) return v;
    const int w = threadIdx.x >> 5, w0 = w / (TPR / 32) * (TPR / 32);
    if ((threadIdx.x & 31) == 0) buf[w] = v;
    __syncthreads();
    float s = buf[w0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) s += buf[w0 + i];
    return s;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *buf)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (TPR == 32) return v;
    const int w = threadIdx.x >> 5, w0 = w / (TPR / 32) * (TPR / 32);
    if ((threadIdx.x & 31) == 0) buf[w] = v;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) s = max(s, buf[w0 + i]);
    return s;
}

// max(m, |a|, |b|); a NaN stays.
__device__ __forceinline__ float max_abs(float m, F2 v)
{
    const float2 x = unf2(v);
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return r;
}

// bf16(a + b), rounded once.  The same as the fp32 sum rounded to bf16: where that sum is not exact, one
// value is below 2^-16 of the other and both ways give the other.
__device__ __forceinline__ uint4 add_bf16(uint4 a, uint4 b)
{
    uint4 r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(a.x), "r"(b.x));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(a.y), "r"(b.y));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.z) : "r"(a.z), "r"(b.z));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.w) : "r"(a.w), "r"(b.w));
    return r;
}

// Where a row goes: its code row and its row in the tiled scales.  A pick that the arguments do not place
// among the rows is reported and skipped.
struct Dest {
    long long row, srow;                                // row < 0: skip
};
__device__ __forceinline__ Dest routed_dest(const RowArgs &a, int t, int j)
{
    const int Tk = a.T * a.k;
    if (j == a.k)                                       // the shared expert's group: token order
        return Dest{(long long)Tk + t, (long long)group_row_tile(Tk, a.E) * kScaleRows + t};
    const int f = t * a.k + j, g = a.ids[f], r = a.inv_perm[f];
    const int off = g >= 0 && g < a.E ? a.offsets[g] : -1;
    if (off < 0 || off > r || r >= Tk) {
        record_status(a.status, MOE_ERR_DEVICE);
        return Dest{-1, 0};
    }
    return Dest{r, (long long)group_row_tile(off, g) * kScaleRows + (r - off)};
}

// FMT 0: no block-scaled output (norm only).  PANELS: rows longer than TPR * CH segments, a panel at a time: where nothing is
// needed of the rest of the row (no norm, no factor of its own).
template <int FMT, bool NORM, bool F32, int TPR, int CH, bool PANELS>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a)
{
    constexpr int kBlk = FMT == MOE_SCALED_NVFP4 ? 16 : 32;   // elements per scale
    constexpr int kLanes = kBlk / 8;                          // lanes of a block
    __shared__ float sbuf[kThreads / 32];
    __shared__ uint32_t mbuf[kThreads / 32];
    // The successor may come in at once; beside a full grid that writes many copies a row only when the rows
    // are read, since its waiting blocks slow that one (512 rows into 9 copies each: 5.2 us against 4.0; the
    // norm of 777 x 5120 is faster with it, 7.9 us against 8.4).
    const bool early = NORM || !a.ids || gridDim.x <= kEarlyBlocks;
    if (early) tc::pdl_trigger();
    tc::pdl_wait();
    const int tr = threadIdx.x % TPR;
    const int t = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    const bool live = t < a.T;
    __shared__ Dest dest[kThreads / TPR][kMaxTopK + 1];
    const int copies = a.ids ? a.k + a.has_shared : 1;
    const int nseg = a.n / 8, ct = scaled_col_tiles(FMT ? FMT : MOE_SCALED_NVFP4, a.n);
    const int group = a.rows_per_group ? t / a.rows_per_group : 0;
    for (int seg0 = 0; seg0 < (PANELS ? nseg : 1); seg0 += TPR * CH) {
        F2 v[CH][4];
        float amax[CH];
        uint4 raw[CH], wv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int seg = seg0 + c * TPR + tr;
            const bool on = live && seg < nseg;
            if (F32) {
                float4 u0 = make_float4(0.f, 0.f, 0.f, 0.f), u1 = u0;
                if (on) {
                    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.x) + (size_t)t * a.n);
                    u0 = __ldcs(p + 2 * seg);
                    u1 = __ldcs(p + 2 * seg + 1);
                }
                v[c][0] = f2(u0.x, u0.y);
                v[c][1] = f2(u0.z, u0.w);
                v[c][2] = f2(u1.x, u1.y);
                v[c][3] = f2(u1.z, u1.w);
            } else {
                raw[c] = make_uint4(0u, 0u, 0u, 0u);
                if (on) raw[c] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + (size_t)t * a.n) + seg);
            }
            if (NORM) {
                wv[c] = make_uint4(0u, 0u, 0u, 0u);
                if (on && a.residual)
                    raw[c] = add_bf16(raw[c], __ldcs(reinterpret_cast<const uint4 *>(a.residual + (size_t)t * a.n) + seg));
                if (on) wv[c] = a.weight ? reinterpret_cast<const uint4 *>(a.weight)[seg]
                                         : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            }
        }
        if (a.ids && seg0 == 0) {
            // one thread a destination, while the row's elements are on their way
            for (int i = threadIdx.x; i < kThreads / TPR * copies; i += kThreads) {
                const int r = i / copies, tt = blockIdx.x * (kThreads / TPR) + r;
                if (tt < a.T) dest[r][i - r * copies] = routed_dest(a, tt, i - r * copies);
            }
            __syncthreads();
        }
        if (!F32) {
#pragma unroll
            for (int c = 0; c < CH; ++c) unpack8(raw[c], v[c]);
        }
        if (NORM) {
            F2 ss2 = f2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) ss2 = fma2(v[c][i], v[c][i], ss2);
                // the sum as the next layer's residual: rounded, and what is normalised here
                const int seg = c * TPR + tr;
                if (a.sum_out && live && seg < nseg) reinterpret_cast<uint4 *>(a.sum_out + (size_t)t * a.n)[seg] = raw[c];
            }
            const float2 sp = unf2(ss2);
            const float rstd = rsqrtf(row_sum<TPR>(sp.x + sp.y, sbuf) / (float)a.n + a.eps);
            const float off = a.weight ? a.weight_offset : 0.f;
            const F2 r2 = f2(rstd, rstd), off2 = f2(off, off);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                F2 w[4];
                unpack8(wv[c], w);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[c][i] = mul2(mul2(v[c][i], r2), add2(w[i], off2));
                const int seg = c * TPR + tr;
                if (a.y_out && live && seg < nseg) reinterpret_cast<uint4 *>(a.y_out + (size_t)t * a.n)[seg] = pack8(v[c]);
            }
        }
        if (FMT == 0) return;
        float row_amax = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_abs(m, v[c][i]);
            if (FMT == MOE_SCALED_NVFP4) row_amax = max_abs(row_amax, f2(m, 0.f));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) m = max_abs(m, f2(__shfl_xor_sync(0xFFFFFFFFu, m, o), 0.f));
            amax[c] = m;
        }
        float g = 1.f, ginv = 1.f;
        if (FMT == MOE_SCALED_NVFP4) {
            if (PANELS || a.gscale) g = live ? a.gscale[group] : 1.f;
            else g = nvfp4_row_factor(row_max<TPR>(__float_as_uint(row_amax) & 0x7FFFFFFFu, mbuf));
            ginv = __fdiv_rn(1.0f, g);
        }
        uint32_t lo[CH], hi[CH], word[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint32_t s;
            float inv;
            if (FMT == MOE_SCALED_NVFP4) {
                s = nvfp4_scale(__float_as_uint(amax[c]) & 0x7FFFFFFFu, ginv, inv);
            } else {
                s = pow2_scale<FMT ? FMT : MOE_SCALED_MXFP8>(__float_as_uint(amax[c]) & 0x7FFFFFFFu);
                inv = pow2_inverse(s);
            }
            float q[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = unf2(mul2(v[c][i], f2(inv, inv)));
                q[2 * i] = p.x;
                q[2 * i + 1] = p.y;
            }
            if (FMT == MOE_SCALED_MXFP8) {
                lo[c] = to_e4m3x2(q[1], q[0]) | ((uint32_t)to_e4m3x2(q[3], q[2]) << 16);
                hi[c] = to_e4m3x2(q[5], q[4]) | ((uint32_t)to_e4m3x2(q[7], q[6]) << 16);
            } else {
                lo[c] = to_e2m1x8(q);
                hi[c] = 0;
            }
            const int seg = seg0 + c * TPR + tr;
            word[c] = seg < nseg ? s << (8 * ((seg / kLanes) & 3)) : 0u;
#pragma unroll
            for (int o = kLanes; o < 4 * kLanes; o <<= 1) word[c] |= __shfl_xor_sync(0xFFFFFFFFu, word[c], o);
        }
        if (!early) tc::pdl_trigger();
        if (!live) return;
        for (int j = 0; j < copies; ++j) {
            Dest d;
            if (a.ids) {
                d = dest[threadIdx.x / TPR][j];
                if (d.row < 0) continue;
            } else {
                d.row = t;
                const int rpg = a.rows_per_group;
                d.srow = rpg ? (long long)group * ((rpg + kScaleRows - 1) / kScaleRows) * kScaleRows + t % rpg : t;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int seg = seg0 + c * TPR + tr;
                if (seg >= nseg) continue;
                if (FMT == MOE_SCALED_MXFP8)
                    reinterpret_cast<uint2 *>(a.codes + (size_t)d.row * a.n)[seg] = make_uint2(lo[c], hi[c]);
                else
                    reinterpret_cast<uint32_t *>(a.codes + (size_t)d.row * (a.n / 2))[seg] = lo[c];
                if (seg % (4 * kLanes) == 0)
                    *reinterpret_cast<uint32_t *>(a.scales + scale_at(d.srow, seg / kLanes, ct)) = word[c];
            }
            if (FMT == MOE_SCALED_NVFP4 && !a.gscale && a.row_scale && tr == 0) a.row_scale[d.row] = g;
        }
    }
}

template <int FMT, bool NORM, bool F32, int TPR, int CH, bool PANELS = false>
cudaError_t launch_one(const RowArgs &a, cudaStream_t st)
{
    const int rows = kThreads / TPR;
    return launch_dependent(rows_kernel<FMT, NORM, F32, TPR, CH, PANELS>, (unsigned)((a.T + rows - 1) / rows), kThreads, 0, st, a);
}

// Threads a row and segments a thread.  Few rows: a segment a thread, for the shortest way through (T = 1,
// n = 2048: 1.9 us from launch to launch).  Many rows of 1025 to 2048 elements: two segments a thread
// share its fixed work (reduction, root, addresses): norm of 32768 x 2048 to MXFP8 96 us -> 90.5 us, and
// 512 rows are the first to gain (3.5 -> 3.3 us; 128 threads of 4 segments: 92 us, a warp a row: 147 us).
template <int FMT, bool NORM, bool F32>
cudaError_t launch_fmt(const RowArgs &a, cudaStream_t st)
{
    const int nseg = a.n / 8;
    if (nseg <= 128) return launch_one<FMT, NORM, F32, 128, 1>(a, st);
    if (nseg <= 256 && a.T >= 512) return launch_one<FMT, NORM, F32, 128, 2>(a, st);
    const int ch = (nseg + kThreads - 1) / kThreads;
    if (ch <= 1) return launch_one<FMT, NORM, F32, 256, 1>(a, st);
    if (ch <= 2) return launch_one<FMT, NORM, F32, 256, 2>(a, st);
    if (ch <= 4) return launch_one<FMT, NORM, F32, 256, 4>(a, st);
    if constexpr (!NORM)
        if (FMT != MOE_SCALED_NVFP4 || a.gscale) return launch_one<FMT, NORM, F32, 256, 4, true>(a, st);
    return launch_one<FMT, NORM, F32, 256, 8>(a, st);
}

// One thread per word of four scales of a row.
__global__ void tile_scales_kernel(const uint8_t *src, uint8_t *dst, int nb, int ct, int N, int row_tiles,
                                   size_t words)
{
    tc::pdl_trigger();
    tc::pdl_wait();
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (size_t)gridDim.x * blockDim.x) {
        // word i of the tiles: tile i / 128, row (i % 128) % 4 * 32 + (i % 128) / 4 of it
        const size_t tile = i >> 7;
        const int in = (int)(i & 127), q = (in & 3) * 32 + (in >> 2);
        const int c = (int)(tile % ct);
        const size_t rt = tile / ct, g = rt / row_tiles;
        const int r = (int)(rt % row_tiles) * kScaleRows + q;
        uint32_t w = 0;
        if (r < N) {
            const uint8_t *p = src + (g * N + r) * nb + 4 * c;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (4 * c + b < nb) w |= (uint32_t)p[b] << (8 * b);
        }
        reinterpret_cast<uint32_t *>(dst)[i] = w;
    }
}

}  // namespace

cudaError_t launch_rows(const RowArgs &a, int fmt, bool norm, cudaStream_t st)
{
    if (norm) {
        if (fmt == MOE_SCALED_NVFP4) return launch_fmt<MOE_SCALED_NVFP4, true, false>(a, st);
        if (fmt == MOE_SCALED_MXFP8) return launch_fmt<MOE_SCALED_MXFP8, true, false>(a, st);
        return launch_fmt<0, true, false>(a, st);
    }
    if (fmt == MOE_SCALED_NVFP4)
        return a.x_f32 ? launch_fmt<MOE_SCALED_NVFP4, false, true>(a, st) : launch_fmt<MOE_SCALED_NVFP4, false, false>(a, st);
    if (fmt == MOE_SCALED_MXFP8)
        return a.x_f32 ? launch_fmt<MOE_SCALED_MXFP8, false, true>(a, st) : launch_fmt<MOE_SCALED_MXFP8, false, false>(a, st);
    return a.x_f32 ? launch_fmt<MOE_SCALED_MXFP4, false, true>(a, st) : launch_fmt<MOE_SCALED_MXFP4, false, false>(a, st);
}

cudaError_t launch_tile_scales(const uint8_t *src, uint8_t *dst, int fmt, int G, int N, int n, cudaStream_t st)
{
    const int nb = n / scaled_block(fmt), ct = scaled_col_tiles(fmt, n), row_tiles = (N + kScaleRows - 1) / kScaleRows;
    const size_t words = (size_t)G * row_tiles * ct * 128;
    const size_t blocks = (words + 255) / 256;
    return launch_dependent(tile_scales_kernel, (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16), 256, 0, st, src, dst, nb, ct,
                            N, row_tiles, words);
}

}  // namespace qmoe
