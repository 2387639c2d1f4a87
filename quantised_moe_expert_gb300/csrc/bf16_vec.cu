// Grouped products of few bf16 rows a group, without tensor-memory tiles.
//
//   y[r, n] = act(sum over the pairs of a[r] . w_g[n] + bias_g[n]) + residual[r, n]      (w [G, N, K]; or a gated pair)
//
// Bound: the weights' bytes and a few latencies.  A tile of tensor memory (bf16_gemm.cu) copies its weights a ring of stages at
// a time on as many SMs as there are tiles; here the sum is shared out too: a warp has 16 outputs and a slice of their
// terms, asks for 16 loads a lane at once, and the slices' sums meet in shared memory.
//
// The products are m16n8k16: 16 weight rows against up to 8 rows of activations, so that a group's rows share one
// read of its weights.  The order of the terms is free as long as both operands share it: a lane's 16 bytes of a row serve two
// instructions as they are, and nothing is rearranged.
//
// 1 x 4096 x 2048: 3.6 us from L2, 4.9 from HBM (3.4 TB/s), against 10.4 of tiles; one token's gated pair of 9 experts (hidden 2048, inter 512)
// 7.7 us, its down products 3.9, against 11.8 and 6.8.  1.9 us are launch to launch, 0.4 the search for a chunk of rows.  fp32
// multiply-adds in place of the instructions, two weight rows a warp: 4.4 us, and 10.2 and 8.0.
#include "bf16.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace {

using tc::pdl_trigger;
using tc::pdl_wait;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxGroups = 1024;
constexpr int kChunk = 32;                         // terms of a lane quartet's load: 8 of each lane
constexpr int kSegment = 768;                      // terms of an fp32 output that the instructions add up in one go (as in bf16_gemm.cu)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4 &u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

struct Chunk {
    int g, row, rows;                              // a group's rows, at most as many as the instructions take
};

// The chunk `index` of all groups' rows in chunks of ROWS.  Every thread takes part; rows == 0: there is none.
template <int ROWS>
__device__ __forceinline__ Chunk find_chunk(const GemmArgs &a, int index)
{
    constexpr int kPer = kMaxGroups / kThreads;
    __shared__ int sums[kWarps], bad;
    __shared__ Chunk found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g0 = threadIdx.x * kPer;
    if (threadIdx.x == 0) {
        bad = 0;
        found.rows = 0;
    }
    int o[kPer + 1], n = 0, b = 0;
#pragma unroll
    for (int i = 0; i <= kPer; ++i) o[i] = g0 + i < a.G ? a.offsets[g0 + i] : a.R;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        b |= o[i] < 0 || o[i] > a.R || o[i + 1] < o[i];
        n += (max(o[i + 1] - o[i], 0) + ROWS - 1) / ROWS;
    }
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (b) bad = 1;
    int base = incl - n;
    for (int w = 0; w < warp; ++w) base += sums[w];
    if (index >= base && index < base + n) {
        int left = index - base;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = (max(o[i + 1] - o[i], 0) + ROWS - 1) / ROWS;
            if (left >= 0 && left < c) {
                found.g = g0 + i;
                found.row = o[i] + left * ROWS;
                found.rows = min(o[i + 1] - found.row, ROWS);
            }
            left -= c;
        }
    }
    __syncthreads();
    if (bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_status(a.status, MOE_ERR_DEVICE);
        return Chunk{0, 0, 0};
    }
    return found;
}

// A CTA has the outputs of kWarps / S tiles of 16 for one chunk of rows; S warps share a tile's terms.  NB: 8 rows each.
// SEGMENTS: a slice's sums leave the instructions' accumulators every kSegment terms and meet in shared memory, since no registers
// are left.  65536 terms: error in the 2-norm 9.2e-6 -> 7.2e-7 (two pairs 1.9e-5 -> 7.4e-7), 8 x 1024 x 65536 47 us either way, 30 rows of 3
// groups x 72 71 -> 86.  A kernel of its own: as a branch in the others it took 2 to 17% of their time.
template <bool DUAL, int NB, int S, bool SEGMENTS>
__global__ void __launch_bounds__(kThreads, 2) gemm_vec_kernel(const __grid_constant__ GemmArgs a, int blocks)
{
    constexpr int kMats = DUAL ? 2 : 1, kTiles = kWarps / S, kOut = 16 * kTiles, kRows = 8 * NB;
    constexpr int kAhead = 8 / kMats;              // chunks whose weights are on their way together
    __shared__ float part[kMats][S][kRows][kOut + 4];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, q = lane & 3;
    const int index = blockIdx.x / blocks, n0 = (blockIdx.x - index * blocks) * kOut;
    pdl_wait();
    Chunk c{0, index * kRows, min(a.R - index * kRows, kRows)};
    if (a.offsets) c = find_chunk<kRows>(a, index);
    if (c.rows <= 0) return;

    const int tile = warp / S, slice = warp % S, first = n0 + 16 * tile;
    const size_t matrix = (size_t)c.g * a.N;
    const int chunks = (a.K + kChunk - 1) / kChunk, per = (chunks + S - 1) / S, lo = slice * per, hi = min(lo + per, chunks);
    float acc[kMats][NB][4] = {};
    // the thread's own places in the slices' sums
    auto place = [&](int m, int b, int e) -> float & { return part[m][slice][8 * b + 2 * q + (e & 1)][16 * tile + i + 8 * (e >> 1)]; };
    int rounds = 0;                                // of loads since the last segment
    bool more = false;                             // there are sums of earlier segments
    if (first < a.N) {
        for (int pair = 0; pair < a.pairs; ++pair) {
            const uint16_t *w[kMats][2], *x[NB];
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)        // rows past the last are read as the last and not written
                    w[m][h] = a.w[DUAL ? m : pair] + (matrix + min(first + 8 * h + i, a.N - 1)) * a.K + 8 * q;
#pragma unroll
            for (int b = 0; b < NB; ++b) x[b] = a.a[pair] + (size_t)(c.row + min(8 * b + i, c.rows - 1)) * a.K + 8 * q;
            for (int c0 = lo; c0 < hi; c0 += kAhead) {
                if (SEGMENTS && rounds++ == kSegment / (kAhead * kChunk)) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            place(0, b, e) = more ? place(0, b, e) + acc[0][b][e] : acc[0][b][e];
                            acc[0][b][e] = 0.f;
                        }
                    more = true;
                    rounds = 1;
                }
                uint4 u[kAhead][kMats][2], v[kAhead][NB];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int k = (c0 + j) * kChunk;
                    const bool on = c0 + j < hi && k + 8 * q < a.K;
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) u[j][m][h] = on ? *reinterpret_cast<const uint4 *>(w[m][h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        v[j][b] = on && 8 * b + i < c.rows ? *reinterpret_cast<const uint4 *>(x[b] + k) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma_bf16(acc[m][b], word(u[j][m][0], 2 * h), word(u[j][m][1], 2 * h), word(u[j][m][0], 2 * h + 1),
                                         word(u[j][m][1], 2 * h + 1), word(v[j][b], 2 * h), word(v[j][b], 2 * h + 1));
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) place(m, b, e) = SEGMENTS && more ? place(m, b, e) + acc[m][b][e] : acc[m][b][e];
    __syncthreads();
    for (int t = threadIdx.x; t < c.rows * kOut; t += kThreads) {
        const int r = t / kOut, o = t - r * kOut, n = n0 + o;
        if (n >= a.N) continue;
        const size_t at = (size_t)(c.row + r) * a.N + n;
        float v[kMats];
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) v[m] += part[m][s][r][o];
            if (a.bias[m]) v[m] += bf16_bits_to_float(a.bias[m][matrix + n]);
            if (a.pre[m]) a.pre[m][at] = float_to_bf16_bits(v[m]);
        }
        float y = act_value(a.act, v[0]);
        if (DUAL) y *= v[kMats - 1];
        if (!DUAL && a.residual) y += bf16_bits_to_float(a.residual[at]);
        if (!DUAL && a.y_f32) static_cast<float *>(a.y)[at] = y;
        else static_cast<uint16_t *>(a.y)[at] = float_to_bf16_bits(y);
    }
}

template <bool DUAL, int NB, int S, bool SEGMENTS = false>
cudaError_t launch(const GemmArgs &a, cudaStream_t st)
{
    constexpr int kOut = 16 * (kWarps / S), kRows = 8 * NB;
    const int blocks = (a.N + kOut - 1) / kOut, chunks = a.offsets ? a.R / kRows + (a.G < a.R ? a.G : a.R) : (a.R + kRows - 1) / kRows;
    return launch_dependent(gemm_vec_kernel<DUAL, NB, S, SEGMENTS>, (unsigned)chunks * blocks, kThreads, 0, st, a, blocks);
}
template <bool DUAL, int NB>
cudaError_t launch_slices(const GemmArgs &a, cudaStream_t st)
{
    if constexpr (!DUAL)
        if (a.y_f32 && (long long)a.K * a.pairs > kWarps * kSegment) return launch<DUAL, NB, kWarps, true>(a, st);
    // a slice of 256 terms is one round of loads
    if (a.K > 1024) return launch<DUAL, NB, 8>(a, st);
    if (a.K > 512) return launch<DUAL, NB, 4>(a, st);
    if (a.K > 256) return launch<DUAL, NB, 2>(a, st);
    return launch<DUAL, NB, 1>(a, st);
}

}  // namespace

cudaError_t launch_gemm_vec(const GemmArgs &a, cudaStream_t st)
{
    // 16 rows a chunk where groups have more than 8 on average.  Without a second matrix that kernel spills 280 bytes of what it has on its
    // way at 128 registers (24 rows in 2 groups x 1032 x 2048 7.1 us); gated pairs 12.
    if (a.R > 8 && (!a.offsets || a.R > 8 * a.G)) return a.glu ? launch_slices<true, 2>(a, st) : launch_slices<false, 2>(a, st);
    return a.glu ? launch_slices<true, 1>(a, st) : launch_slices<false, 1>(a, st);
}

}  // namespace qmoe
