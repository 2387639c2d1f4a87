// Grouped products of bf16 rows with bf16 matrices, 32-bit sums, with their epilogue, and their weight gradients.
//
//   y[r] = act(sum over the pairs of a[r] w_g^T + bias_g) + residual[r]     (GLU: act(a gate_g^T + ..) (a up_g^T + ..))
//   dw_g = sum over the group's rows of dy[r]^T x[r],  db_g = sum of dy[r]
//
// Tiles of 64 x 64 outputs on the fp32 units, operands through shared memory 16 elements deep.
#include "bf16.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

constexpr int kThreads = 256, kTile = 64, kDeep = 16, kMaxGroups = 1024;

// Checks the offsets; every thread takes part.  False (and a report): nothing is computed.
__device__ __forceinline__ bool offsets_ok(const int32_t *offsets, int G, int R, int *status)
{
    int bad = 0;
    for (int i = threadIdx.x; i < G; i += kThreads) {
        const int o = offsets[i], next = i + 1 < G ? offsets[i + 1] : R;
        bad |= o < 0 || o > R || next < o;
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0 && blockIdx.x == 0) record_status(status, MOE_ERR_DEVICE);
    return !bad;
}

__device__ __forceinline__ float load16(const uint16_t *p, size_t row, size_t pitch, int col)
{
    return bf16_bits_to_float(p[row * pitch + col]);
}

__global__ void __launch_bounds__(kThreads) gemm_kernel(const __grid_constant__ GemmArgs a)
{
    __shared__ float sa[kDeep][kTile + 1], sw[2][kDeep][kTile + 1];
    __shared__ int sh[3];
    pdl_trigger();
    pdl_wait();
    const int n_tiles = (a.N + kTile - 1) / kTile, mt = blockIdx.x / n_tiles, n0 = (blockIdx.x - mt * n_tiles) * kTile;
    int g = 0, row0 = mt * kTile, end = a.R;
    if (a.offsets) {
        if (!offsets_ok(a.offsets, a.G, a.R, a.status)) return;
        if (threadIdx.x == 0) {
            int left = mt;
            sh[0] = -1;
            for (int i = 0; i < a.G; ++i) {
                const int o = a.offsets[i], e = i + 1 < a.G ? a.offsets[i + 1] : a.R, tiles = (e - o + kTile - 1) / kTile;
                if (left < tiles) {
                    sh[0] = i;
                    sh[1] = o + left * kTile;
                    sh[2] = e;
                    break;
                }
                left -= tiles;
            }
        }
        __syncthreads();
        g = sh[0];
        if (g < 0) return;
        row0 = sh[1];
        end = sh[2];
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[2][4][4] = {};
    for (int pair = 0; pair < a.pairs; ++pair) {
        for (int k0 = 0; k0 < a.K; k0 += kDeep) {
            for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
                const int r = i / kDeep, k = i % kDeep;
                sa[k][r] = row0 + r < end && k0 + k < a.K ? load16(a.a[pair], row0 + r, a.K, k0 + k) : 0.f;
            }
            for (int m = 0; m < (a.glu ? 2 : 1); ++m) {
                const uint16_t *w = a.w[a.glu ? m : pair] + (size_t)g * a.N * a.K;
                for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
                    const int n = a.w_kn ? i % kTile : i / kDeep, k = a.w_kn ? i / kTile : i % kDeep;
                    const bool in = n0 + n < a.N && k0 + k < a.K;
                    sw[m][k][n] = !in ? 0.f : a.w_kn ? load16(w, k0 + k, a.N, n0 + n) : load16(w, n0 + n, a.K, k0 + k);
                }
            }
            __syncthreads();
            for (int k = 0; k < kDeep; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) {
                        acc[0][i][j] = fmaf(sa[k][ty + 16 * i], sw[0][k][tx + 16 * j], acc[0][i][j]);
                        if (a.glu) acc[1][i][j] = fmaf(sa[k][ty + 16 * i], sw[1][k][tx + 16 * j], acc[1][i][j]);
                    }
            __syncthreads();
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = row0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (r >= end || n >= a.N) continue;
            const size_t at = (size_t)r * a.N + n;
            float v[2];
            for (int m = 0; m < 2; ++m) {
                v[m] = acc[m][i][j] + (a.bias[m] ? load16(a.bias[m], g, a.N, n) : 0.f);
                if (a.pre[m]) a.pre[m][at] = float_to_bf16_bits(v[m]);
            }
            float y = act_value(a.act, v[0]);
            if (a.glu) y *= v[1];
            if (a.residual) y += bf16_bits_to_float(a.residual[at]);
            if (a.y_f32) static_cast<float *>(a.y)[at] = y;
            else static_cast<uint16_t *>(a.y)[at] = float_to_bf16_bits(y);
        }
}

__device__ __forceinline__ void put(void *p, size_t at, int f32, int accumulate, float v)
{
    if (f32) static_cast<float *>(p)[at] = accumulate ? static_cast<float *>(p)[at] + v : v;
    else static_cast<uint16_t *>(p)[at] = float_to_bf16_bits(v);
}

__global__ void __launch_bounds__(kThreads) wgrad_kernel(const __grid_constant__ WgradArgs a)
{
    __shared__ float sd[kDeep][kTile + 1], sx[kDeep][kTile + 1];
    pdl_trigger();
    pdl_wait();
    const int nt = (a.N + kTile - 1) / kTile, kt = (a.K + kTile - 1) / kTile;
    const int g = blockIdx.x / (nt * kt), n0 = blockIdx.x / kt % nt * kTile, k0 = blockIdx.x % kt * kTile;
    if (a.offsets && !offsets_ok(a.offsets, a.G, a.R, a.status)) return;
    const int start = a.offsets ? a.offsets[g] : 0, end = a.offsets && g + 1 < a.G ? a.offsets[g + 1] : a.R;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, db = 0.f;
    for (int r0 = start; r0 < end; r0 += kDeep) {
        for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
            const int r = r0 + i / kTile, c = i % kTile;
            sd[i / kTile][c] = r < end && n0 + c < a.N ? load16(a.dy, r, a.N, n0 + c) : 0.f;
            sx[i / kTile][c] = r < end && k0 + c < a.K ? load16(a.x, r, a.K, k0 + c) : 0.f;
        }
        __syncthreads();
        for (int r = 0; r < kDeep; ++r)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sd[r][ty + 16 * i], sx[r][tx + 16 * j], acc[i][j]);
        if (threadIdx.x < kTile)
            for (int r = 0; r < kDeep; ++r) db += sd[r][threadIdx.x];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + ty + 16 * i, k = k0 + tx + 16 * j;
            if (n < a.N && k < a.K) put(a.dw, ((size_t)g * a.N + n) * a.K + k, a.f32, a.accumulate, acc[i][j]);
        }
    if (a.db && k0 == 0 && threadIdx.x < kTile && n0 + (int)threadIdx.x < a.N)
        put(a.db, (size_t)g * a.N + n0 + threadIdx.x, a.f32, a.accumulate, db);
}

}  // namespace

cudaError_t launch_gemm(const GemmArgs &a, cudaStream_t st)
{
    const long long mt = a.offsets ? a.R / kTile + (a.G < a.R ? a.G : a.R) : (a.R + kTile - 1) / kTile;
    const long long tiles = mt * ((a.N + kTile - 1) / kTile);
    return launch_dependent(gemm_kernel, (unsigned)tiles, kThreads, 0, st, a);
}

cudaError_t launch_wgrad(const WgradArgs &a, cudaStream_t st)
{
    const long long tiles = (long long)a.G * ((a.N + kTile - 1) / kTile) * ((a.K + kTile - 1) / kTile);
    return launch_dependent(wgrad_kernel, (unsigned)tiles, kThreads, 0, st, a);
}

}  // namespace qmoe
