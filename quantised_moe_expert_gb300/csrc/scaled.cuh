// Block-scaled rows (narrow codes, one scale per block of consecutive elements): formats, the scale tile
// order, conversions, and the argument blocks of the kernels that make and multiply them.
#pragma once

#include "moe_common.cuh"

#include <atomic>

namespace qmoe {

// Elements per block, codes per byte and columns of a K step of each format.
__host__ __device__ constexpr int scaled_block(int fmt) { return fmt == MOE_SCALED_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr bool scaled_is4(int fmt) { return fmt != MOE_SCALED_MXFP8; }

// Scale tiles: 128 rows x 4 consecutive block scales of each row, 512 bytes, in the order in which tensor
// memory holds them (32 lanes x four 32-bit columns): byte (r % 32) * 16 + (r / 32) * 4 + b.
constexpr int kScaleTile = 512;
constexpr int kScaleRows = 128;
__host__ __device__ constexpr int scaled_col_tiles(int fmt, int n) { return (n / scaled_block(fmt) + 3) / 4; }
// Byte of block b of row r (a row of the whole tiled array), ct column tiles a row.
__host__ __device__ inline size_t scale_at(long long r, int b, int ct)
{
    const int q = (int)(r & 127);
    return ((size_t)(r >> 7) * ct + (b >> 2)) * kScaleTile + (q & 31) * 16 + (q >> 5) * 4 + (b & 3);
}
// First row tile of a group whose rows start at row `off` of the grouped rows: disjoint for any counts
// (off / 128 grows by at least ceil(count / 128) - 1 from one group to the next), without a prefix sum.
__host__ __device__ inline int group_row_tile(int off, int g) { return off / kScaleRows + g; }

// ---------------------------------------------------------------- conversions

// Two values to E4M3, ties to even, at most +-448; lo in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float hi, float lo)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight values to E2M1, ties to even, at most +-6; value i in bits 4i.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The value of an E4M3 byte.
__device__ __forceinline__ float from_e4m3(uint32_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

constexpr uint32_t kInfBits = 0x7F800000u;

// The power-of-two scale of a block from the bits of its largest magnitude (as an fp32): the smallest
// 2^e with amax <= top 2^e, e in [-127, 127]; returns e + 127.  top = 1.75 * 2^8 (E4M3) or 1.5 * 2^2
// (E2M1), so one comparison of the fraction decides between e = E - top_exp and the next; no element
// of the block saturates.  fp32 subnormals (E = -126 or below) end in the clamp.  Non-finite: 255 (NaN).
template <int FMT>
__device__ __forceinline__ uint32_t pow2_scale(uint32_t amax_bits)
{
    constexpr uint32_t kFrac = FMT == MOE_SCALED_MXFP8 ? 0x600000u : 0x400000u;
    constexpr int kTop = FMT == MOE_SCALED_MXFP8 ? 8 : 2;
    if (amax_bits >= kInfBits) return 255u;
    const int e = (int)(amax_bits >> 23) - kTop + ((amax_bits & 0x7FFFFFu) > kFrac ? 1 : 0);
    return (uint32_t)max(e, 0);
}
// 2^(127 - b): the factor that divides by the scale byte b (exact; 2^-127 is subnormal).
__device__ __forceinline__ float pow2_inverse(uint32_t b) { return pow2f(127 - (int)b); }

// NVFP4: the E4M3 scale of a block for a row factor g (ginv = 1 / g), and the factor that maps the
// block's elements to codes.  Non-finite amax: the NaN scale.
__device__ __forceinline__ uint32_t nvfp4_scale(uint32_t amax_bits, float ginv, float &inv)
{
    if (amax_bits >= kInfBits) {
        inv = 0.f;
        return 0x7Fu;
    }
    const uint32_t s = to_e4m3x2(0.f, __uint_as_float(amax_bits) * ginv * (1.0f / 6.0f)) & 0xFFu;
    inv = s ? __fdiv_rn(ginv, from_e4m3(s)) : 0.f;
    return s;
}
// Factor of a row from its largest magnitude: 448 * 6 = 2688 times the smallest unit; kept away from
// zero so that 1 / g stays finite.
__device__ __forceinline__ float nvfp4_row_factor(uint32_t amax_bits)
{
    return amax_bits >= kInfBits ? __uint_as_float(0x7FC00000u)
                                 : fmaxf(__uint_as_float(amax_bits) * (1.0f / 2688.0f), 7.70371977754894e-34f);
}

// ---------------------------------------------------------------- launches

// Every kernel of this family lets its successor in the stream start early (griddepcontrol.launch_dependents)
// and reads or writes memory only after griddepcontrol.wait, in every block: a successor's set-up (barriers,
// tensor memory, tensor maps) runs under its predecessor's tail.  So a kernel is there while its predecessor still
// writes: whatever an earlier launch may have written (offsets, picks, factors, weights) is read by plain loads, never
// through the read-only path (__ldg, const __restrict__), which is for memory that nobody writes while the kernel
// runs and whose loads the compiler may move above the wait.  A norm of one row behind another: 2.6 us from
// launch to launch without, 1.9 us with.
template <class... P, class... A>
cudaError_t launch_dependent_clusters(void (*kernel)(P...), unsigned grid, unsigned cluster, unsigned block, size_t smem,
                                      cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e == cudaSuccess ? e : cudaGetLastError();    // the error is returned, not left for a later launch to find
}
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    return launch_dependent_clusters(kernel, grid, 1, block, smem, st, args...);
}

// Once per kernel and device: its dynamic shared memory (`ready`: the devices on which that is done).
template <class K>
cudaError_t set_shared(K kernel, int bytes, std::atomic<uint64_t> &ready)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (ready.load(std::memory_order_relaxed) >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// ---------------------------------------------------------------- kernel arguments

// Rows to block-scaled rows (scaled_rows.cu).
struct RowArgs {
    const void *x;              // [T, n] bf16 or fp32 (x_f32)
    const uint16_t *residual;   // norm: bf16 [T, n] or null
    const uint16_t *weight;     // norm: bf16 [n] or null (ones)
    uint16_t *sum_out;          // norm: bf16 [T, n] or null
    uint16_t *y_out;            // norm: bf16 [T, n] or null
    uint8_t *codes, *scales;    // destination rows, scale tiles
    float *row_scale;           // NVFP4 without gscale: [rows]
    const float *gscale;        // NVFP4: factor per group, or null
    const int32_t *ids, *inv_perm, *offsets;   // routed destination, or null
    int *status;
    float eps, weight_offset;
    int T, n, x_f32;
    int rows_per_group;         // plain destination: rows of a group (scale tiles start anew with each)
    int k, E, has_shared;       // routed destination
};
cudaError_t launch_rows(const RowArgs &a, int fmt, bool norm, cudaStream_t st);
cudaError_t launch_tile_scales(const uint8_t *src, uint8_t *dst, int fmt, int G, int N, int n, cudaStream_t st);

// Grouped product of block-scaled rows (scaled_gemm.cu).
struct ScaledGemmArgs {
    const uint8_t *a_codes, *a_scales;
    const float *a_row_scale;            // [R] or null
    const uint8_t *w_codes[2], *w_scales[2];
    const float *alpha[2];               // [G] or null; [1]: the up matrices of a SwiGLU pair
    const int32_t *offsets;              // [G] first row of each group (the last group ends at R), or null (G == 1)
    void *y;                             // [R, N] bf16 or fp32 (y_f32)
    uint8_t *h_codes, *h_scales;         // SwiGLU: [R, N] block-scaled
    const float *h_gscale;               // SwiGLU, NVFP4: [G]
    int *status;
    int R, N, K, G, y_f32;
    long long wait_limit;
};
cudaError_t launch_scaled_gemm(const ScaledGemmArgs &a, int fmt, bool swiglu, cudaStream_t st);
cudaError_t launch_scaled_vec(const ScaledGemmArgs &a, int fmt, bool swiglu, cudaStream_t st);   // few rows (scaled_vec.cu)

}  // namespace qmoe
