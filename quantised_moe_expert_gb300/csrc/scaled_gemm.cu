// Grouped products of block-scaled rows on the block-scaled tensor-core kinds.
//
//   acc[r, n] = sum_b sa[r, b] sw[g, n, b] sum_{j in block b} a[r, j] w[g, n, j]      (fp32, in tensor memory)
//   y[r, n]   = row_scale[r] alpha[g] acc[r, n]
//   h[r, n]   = silu(gate) up of two such products, quantised in the epilogue
//
// Rows are sorted by group (expert): group g owns rows [offsets[g], offsets[g + 1]).  Operands:
//   NVFP4 x NVFP4   kind::mxf4nvf4, 64 elements an instruction, an E4M3 scale per 16
//   MXFP8 x MXFP4   kind::mxf8f6f4, 32 elements an instruction, an E8M0 scale per 32; TMA widens the
//                   4-bit codes to the byte containers that kind takes
// Either way a K step of a tile is rows of 128 bytes (256 or 128 elements) in the 128-byte swizzle.  Tokens
// are the M = 128 operand whatever their number (a step's cost is its weight bytes, not its rows: only
// the rows present are copied), weights the N = BN operand, so that a thread of the epilogue holds
// consecutive outputs of one row: whole blocks of h for its scale, whole sectors of y.
//
// One CTA per SM walks over the tiles: warp 0 copies codes (TMA), warp 2 copies scale tiles (bulk), warp 1
// moves a step's scales from shared into tensor memory (tcgen05.cp, in order with the MMAs behind it) and
// issues its MMAs, warps 4-11 read the accumulators and write.  Every stage has its own scale columns, so
// a stage's barriers also guard them.  (Scales through registers, tcgen05.st by four more warps, which
// read every tile four times from shared memory: 8192 x 8192 x 4096 117 us against 112 us.)
//
// Bounds and measurements (hidden 2048, inter 512, 257 groups): 512 tokens, NVFP4, the gate/up pair 51 us (6.1 TB/s
// of weights and rows) and the down products 32 us (5.5 TB/s): HBM.  4096 tokens, MXFP8, 93 and 66 us: the copies
// that widen the 4-bit codes, about 32 bytes of shared memory a cycle, and in the down products (4 steps a tile) the
// change of tile as well.  Small products: 0.28 to 0.30 us a K step (NVFP4, 16 rows; the issue of its 8 scale copies and
// 4 MMAs, some 460 cycles, is most of it) or 0.21 to 0.23 (MXFP8, whose 2 copies and 4 MMAs would take 0.13: what paces
// it has not been found), behind a launch (16 x 4096 x 2048 NVFP4 4.5 us); those of fewest rows go to scaled_vec.cu.
// 8192 x 8192 x 4096 NVFP4 100 us, 5.5 PFLOP/s: of 13,100 cycles a tile 8,000 of products, 2,300 until the last
// tile's accumulators are read and 2,700 for full stages (see the pair below).
#include "scaled.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kMaxGroups = 1024;
constexpr int kStepBytes = 128;                    // bytes of a K step in a row of codes (as in shared memory)

template <int FMT, bool DUAL, int BN, bool SPLIT>
struct Plan {
    static constexpr bool kNv = FMT == MOE_SCALED_NVFP4;
    static constexpr int kStepK = kNv ? 256 : 128;           // elements of a K step
    static constexpr int kTilesK = kNv ? 4 : 1;              // scale column tiles of a K step
    static constexpr int kOutN = DUAL ? BN / 2 : BN;         // output columns of a tile
    static constexpr int kMmaN = DUAL && BN == 128 ? 64 : BN;   // N of one instruction
    static constexpr int kChunks = DUAL || BN > 128 ? 2 : 1; // weight scale row tiles of a tile
    static constexpr int kABytes = 128 * kStepBytes, kBBytes = BN * kStepBytes;
    static constexpr int kBTxBytes = kNv ? kBBytes : kBBytes / 2;   // a widened copy counts the codes, not the padding
    static constexpr int kSfaBytes = kTilesK * kScaleTile, kSfbBytes = kChunks * kTilesK * kScaleTile;
    // shared memory: the stages' codes (whole 1024-byte swizzle atoms), then their scales
    static constexpr int kCodeBytes = kABytes + kBBytes, kSfBytes = kSfaBytes + kSfbBytes;
    static_assert(kCodeBytes % 1024 == 0, "swizzle atoms");
    static constexpr int kStages = BN == 256 ? (DUAL || !kNv ? 4 : 3) : BN == 128 ? (DUAL && SPLIT && kNv ? 4 : 5) : 7;
    static constexpr int kStaged = BN == 256 && !kNv ? 64 : 128;     // bytes of a row that an epilogue warp stages at a time
    static constexpr int kOutBytes = DUAL || BN == 64 ? 0 : 8 * 32 * kStaged;
    static constexpr int kAccs = BN == 256 ? 1 : 2;          // accumulator buffers
    static constexpr int kSfCols = 4 * kTilesK * (1 + kChunks);   // tensor-memory columns of a stage's scales
    static constexpr int kPartCols = (DUAL ? 2 : 1) * kOutN / 2;     // accumulator columns of an epilogue warp
    static constexpr int kPartBytes = SPLIT ? 128 * kPartCols * 4 : 0;   // the other CTA's sums of half of the columns
    static constexpr int kSfAt = kStages * kCodeBytes, kOutAt = kSfAt + kStages * kSfBytes, kPartAt = kOutAt + kOutBytes;
    static constexpr int kSmem = kPartAt + kPartBytes + 1024;
    static_assert(kAccs * BN + kStages * kSfCols <= 512, "tensor memory");
};

struct Maps {
    CUtensorMap a128, a32, w[2];
};

struct Shared {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], part[4], drain;
    uint32_t tmem;
    int abort;
    int bad, groups, row_tiles;                              // malformed offsets; groups with rows; their row tiles
    int gave_up, issued[2][2];                               // a pair's: whether any of its waits ran out; copies [CTA][codes, scales]
    int2 warp_sum[kThreads / 32];
    int2 group[kMaxGroups + 1];                              // those groups: row tiles before it, start << 10 | group
};

struct Tile {
    int g, row0, rows, srow_tile, nt;                        // rows [row0, row0 + rows), their scale row tile
};

constexpr int kGroupBits = 10;
static_assert(kMaxGroups == 1 << kGroupBits, "the table's packing");

// Tile `tile` of tiles of ROWS rows.
template <int ROWS>
__device__ __forceinline__ Tile tile_at(const ScaledGemmArgs &a, const Shared &sh, int tile, int n_tiles)
{
    const int mt = tile / n_tiles;
    Tile t;
    t.nt = tile - mt * n_tiles;
    if (!a.offsets) {                                        // one group
        t.g = 0;
        t.row0 = mt * ROWS;
        t.rows = min(a.R - t.row0, ROWS);
        t.srow_tile = mt * (ROWS / kScaleRows);
        return t;
    }
    int lo = 0, hi = sh.groups;                              // the last entry whose first tile is not past mt
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.group[mid].x <= mt) lo = mid;
        else hi = mid;
    }
    const int2 e = sh.group[lo];
    const int start = (int)((uint32_t)e.y >> kGroupBits), end = (int)((uint32_t)sh.group[lo + 1].y >> kGroupBits), m = mt - e.x;
    t.g = e.y & (kMaxGroups - 1);
    t.row0 = start + m * ROWS;
    t.rows = min(end - t.row0, ROWS);
    t.srow_tile = group_row_tile(start, t.g) + m * (ROWS / kScaleRows);
    return t;
}

// The table of groups with rows: each thread has a few neighbouring groups, whose tiles of ROWS rows and
// whose number it scans with the block.  Every thread takes part.
template <int ROWS>
__device__ __forceinline__ void build_table(const ScaledGemmArgs &a, Shared &sh, int warp, int lane)
{
    constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
    const int g0 = threadIdx.x * kPer;
    int o[kPer + 1];
#pragma unroll
    for (int i = 0; i <= kPer; ++i) o[i] = g0 + i < a.G ? a.offsets[g0 + i] : a.R;
    int2 n = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (o[i] < 0 || o[i] > a.R || o[i + 1] < o[i]) sh.bad = 1;
        n.x += (max(o[i + 1] - o[i], 0) + ROWS - 1) / ROWS;
        n.y += o[i + 1] > o[i];
    }
    int2 incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl.x, d), y = __shfl_up_sync(0xFFFFFFFFu, incl.y, d);
        if (lane >= d) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    int2 base = make_int2(incl.x - n.x, incl.y - n.y);
    for (int w = 0; w < warp; ++w) {
        base.x += sh.warp_sum[w].x;
        base.y += sh.warp_sum[w].y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (o[i + 1] <= o[i]) continue;
        sh.group[base.y] = make_int2(base.x, o[i] << kGroupBits | (g0 + i));
        base.x += (o[i + 1] - o[i] + ROWS - 1) / ROWS;
        base.y += 1;
    }
    if (threadIdx.x == kThreads - 1) {
        sh.groups = base.y;
        sh.row_tiles = sh.bad ? 0 : base.x;
        sh.group[base.y] = make_int2(base.x, (int)((uint32_t)a.R << kGroupBits));
        if (sh.bad) record_status(a.status, MOE_ERR_DEVICE);
    }
}

// Scale tiles in shared memory as tcgen05.cp takes them: 8 rows x 16 bytes cores, 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
// One scale tile from shared memory to four columns of all four quarters of the lanes (CG == 2: in both CTAs
// of the pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc, uint32_t issue)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::%3.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
                 "l"(desc), "r"(issue), "n"(CG)
                 : "memory");
}

// Instruction descriptor of the block-scaled kinds: scale ids [4,6) (B) and [29,31) (A), A format [7,10),
// B format [10,13), N >> 3 [17,23), scale format [23] (0 E4M3, 1 E8M0), M >> 4 [24,29).
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_scaled(uint32_t m, uint32_t n, uint32_t sf_id)
{
    return (sf_id << 4) | ((FMT == MOE_SCALED_NVFP4 ? 1u : 0u) << 7) | ((FMT == MOE_SCALED_NVFP4 ? 1u : 5u) << 10) |
           ((n >> 3) << 17) | ((FMT == MOE_SCALED_NVFP4 ? 0u : 1u) << 23) | ((m >> 4) << 24) | (sf_id << 29);
}
template <int FMT, int CG>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t accumulate, uint32_t issue)
{
    if (FMT == MOE_SCALED_NVFP4)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::%8.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(issue), "n"(CG)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::%8.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(issue), "n"(CG)
            : "memory");
}

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

// Adds the other CTA's sums of 16 columns from `col` on to this row's: part[column / 4][row], or null.
__device__ __forceinline__ void add_part(uint32_t (&u)[16], const float4 *part, int col, int lane)
{
    if (part == nullptr) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 p = part[(col / 4 + i) * 32 + lane];
        u[4 * i] = __float_as_uint(__uint_as_float(u[4 * i]) + p.x);
        u[4 * i + 1] = __float_as_uint(__uint_as_float(u[4 * i + 1]) + p.y);
        u[4 * i + 2] = __float_as_uint(__uint_as_float(u[4 * i + 2]) + p.z);
        u[4 * i + 3] = __float_as_uint(__uint_as_float(u[4 * i + 3]) + p.w);
    }
}

// 32 rows of ROW_BYTES (64 or 128), a lane a row in 16-byte chunks w[], to rows `pitch` bytes apart from `dst` on, the
// first `rows` rows and `chunks` chunks of each, through `stage`: 4 or 8 lanes write a row's bytes together.
template <int ROW_BYTES>
__device__ __forceinline__ void store_staged(uint8_t *dst, size_t pitch, const uint32_t *w, int rows, int chunks, int lane, uint8_t *stage)
{
    // row r's chunk k at k ^ r (rows of 128 bytes) or k ^ r / 2 (of 64) of the row: no bank is met twice in a phase
    constexpr int kChunks = ROW_BYTES / 16, kShift = ROW_BYTES == 64 ? 1 : 0;
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
        *reinterpret_cast<uint4 *>(stage + lane * ROW_BYTES + ((k ^ (lane >> kShift)) % kChunks) * 16) =
            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    __syncwarp();
    const int k = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int r = i * (32 / kChunks) + lane / kChunks;
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * ROW_BYTES + ((k ^ (r >> kShift)) % kChunks) * 16);
        if (r < rows && k < chunks) *reinterpret_cast<uint4 *>(dst + r * pitch + 16 * k) = v;
    }
    __syncwarp();
}

// COLS accumulator columns of the warp's 32 rows (from `row` on, the first `rows` of them exist) to y;
// release() once they are in registers.  Outputs go through `stage`, the warp's part of shared memory, STAGE bytes
// a row at a time (128, or 64 where another stage of operands fits then): a lane of its own row touches 32
// lines in every store, which costs the load/store unit a cycle a line or more (4300 cycles a 128 x 256 tile
// of bf16, more than its products at K = 512; the routed layer of 4096 tokens, whose down products are 302 MB
// of fp32, took 363 us with such stores, against 283).
template <int COLS, int STAGE, class Release>
__device__ __forceinline__ void store_rows(const ScaledGemmArgs &a, uint32_t d, size_t row, int rows, int col0, float s, int lane,
                                           uint8_t *stage, const float4 *part, Release release)
{
    constexpr int kBatch = COLS;
    const size_t pitch = (size_t)a.N * (a.y_f32 ? 4 : 2);
    uint8_t *y = static_cast<uint8_t *>(a.y) + row * pitch + (size_t)col0 * (a.y_f32 ? 4 : 2);
    if (a.y_f32) {
        uint32_t u[COLS / 16][16];
#pragma unroll
        for (int i = 0; i < COLS / 16; ++i) tmem_ld16(d + 16 * i, u[i]);
        tmem_ld_wait();
        release();
#pragma unroll
        for (int i = 0; i < COLS / 16; ++i) {
            add_part(u[i], part, 16 * i, lane);
#pragma unroll
            for (int k = 0; k < 16; ++k) u[i][k] = __float_as_uint(__uint_as_float(u[i][k]) * s);
        }
        if constexpr (COLS < 64) {                         // few tiles: the shortest way (0.15 us of 4.7 at one token)
#pragma unroll
            for (int i = 0; i < COLS; i += 4)
                if (lane < rows && col0 + i < a.N)
                    *reinterpret_cast<uint4 *>(y + lane * pitch + 4 * i) =
                        make_uint4(u[i / 16][i % 16], u[i / 16][i % 16 + 1], u[i / 16][i % 16 + 2], u[i / 16][i % 16 + 3]);
        } else {
#pragma unroll
            for (int c = 0; c < COLS; c += STAGE / 4) {
                uint32_t w[STAGE / 4];
#pragma unroll
                for (int i = 0; i < STAGE / 4; ++i) w[i] = u[(c + i) / 16][i % 16];
                store_staged<STAGE>(y + 4 * c, pitch, w, rows, (a.N - col0 - c) / 4, lane, stage);
            }
        }
        return;
    }
    uint32_t w[COLS / 2];
#pragma unroll
    for (int c = 0; c < COLS; c += kBatch) {
        uint32_t u[kBatch / 16][16];
#pragma unroll
        for (int i = 0; i < kBatch / 16; ++i) tmem_ld16(d + c + 16 * i, u[i]);
        tmem_ld_wait();
        release();
#pragma unroll
        for (int i = 0; i < kBatch / 16; ++i) add_part(u[i], part, c + 16 * i, lane);
#pragma unroll
        for (int i = 0; i < kBatch / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(u[i / 8][2 * i % 16]) * s,
                                                           __uint_as_float(u[i / 8][2 * i % 16 + 1]) * s);
            w[c / 2 + i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    if constexpr (COLS < 64) {
#pragma unroll
        for (int i = 0; i < COLS / 2; i += 4)
            if (lane < rows && col0 + 2 * i < a.N)
                *reinterpret_cast<uint4 *>(y + lane * pitch + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
        for (int c = 0; c < COLS / 2; c += STAGE / 4) {
            uint32_t v[STAGE / 4];
#pragma unroll
            for (int i = 0; i < STAGE / 4; ++i) v[i] = w[c + i];
            store_staged<STAGE>(y + 4 * c, pitch, v, rows, (a.N - col0 - 2 * c) / 8, lane, stage);
        }
    }
}

// SPLIT: no more tiles than half the SMs, where the K steps one after the other are the time: two CTAs (a
// cluster) take half of a tile's steps each, hand each other half of the columns' sums through shared memory and
// finish the other half.
template <int FMT, bool DUAL, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
scaled_gemm_kernel(const __grid_constant__ ScaledGemmArgs a, const __grid_constant__ Maps maps)
{
    using P = Plan<FMT, DUAL, BN, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    uint8_t *smem = align_smem_1024(smem_raw);
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int n_tiles = (a.N + P::kOutN - 1) / P::kOutN, n_steps = (a.K + P::kStepK - 1) / P::kStepK;
    const int ct = scaled_col_tiles(FMT, a.K);
    // this CTA's tiles and its K steps of each
    const int rank = SPLIT ? (int)cluster_ctarank() : 0;
    const int first_tile = SPLIT ? blockIdx.x >> 1 : blockIdx.x, stride = SPLIT ? gridDim.x >> 1 : gridDim.x;
    const int ks0 = SPLIT && rank ? (n_steps + 1) / 2 : 0, ks1 = SPLIT && !rank ? (n_steps + 1) / 2 : n_steps;
    const int w_row_tiles = (a.N + kScaleRows - 1) / kScaleRows;      // scale row tiles of a matrix

    pdl_trigger();
    if (threadIdx.x == 0) {
        prefetch_map(&maps.w[0]);
        if (DUAL) prefetch_map(&maps.w[1]);
        prefetch_map(&maps.a32);
        prefetch_map(&maps.a128);
        for (int i = 0; i < P::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 2);                      // codes and scales
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < P::kAccs; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), 8);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.part[i]), 1);
        sh.abort = 0;
        sh.bad = 0;
        sh.row_tiles = (a.R + kScaleRows - 1) / kScaleRows;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    __syncthreads();
    if (SPLIT) cluster_arrive();
    pdl_wait();
    if (a.offsets) build_table<kScaleRows>(a, sh, warp, lane);
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_wait();                                        // the first CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
    const int total = __shfl_sync(0xFFFFFFFFu, sh.row_tiles * n_tiles, 0);
    volatile int *abort = &sh.abort;
    const uint32_t smem0 = smem_u32(smem);
    auto fail = [&]() {
        record_status(a.status, MOE_ERR_TIMEOUT);
        *abort = 1;
    };

    // A role's warp walks its loop as a whole and only the issuing instructions are one lane's, so that loop
    // counters, addresses and descriptors stay in uniform registers: with the loop itself in one lane's
    // branch a step's issue took 750 cycles, twice its products.
    // registers: 384 x 168 at launch, redistributed by warpgroup to 104 and 2 x 200 (the same total)
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || warp == 2) {
        // ---- copies: warp 0 the codes, warp 2 the scales
        const bool leader = elect_one();
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            const Tile t = tile_at<kScaleRows>(a, sh, tile, n_tiles);
            const int n0 = t.nt * P::kOutN, wrow = t.g * a.N + n0;
            const bool second = P::kChunks == 2 && (DUAL || n0 / kScaleRows + 1 < w_row_tiles);
            const int boxes = t.rows > 96 ? 4 : (t.rows + 31) / 32;
            const size_t row = (size_t)ct * kScaleTile, wt = (size_t)t.g * w_row_tiles + n0 / kScaleRows;
            const uint8_t *pa = a.a_scales + t.srow_tile * row, *pb = a.w_scales[0] + wt * row;
            const uint8_t *pc = a.w_scales[DUAL ? 1 : 0] + (DUAL ? wt : wt + 1) * row;
            for (int ks = ks0; ks < ks1; ++ks) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.empty[st]), ph ^ 1, a.wait_limit, abort));
                if (!ok) {
                    if (leader) fail();
                    break;
                }
                const uint32_t base = smem0 + st * P::kCodeBytes, bar = smem_u32(&sh.full[st]);
                if (warp == 0) {
                    if (leader) {
                        mbar_arrive_expect_tx(bar, boxes * 32 * kStepBytes + P::kBTxBytes);
                        // x in the map's elements: bytes, or 4-bit codes for the widened weights
                        const int xa = ks * kStepBytes, xw = P::kNv ? ks * kStepBytes : ks * P::kStepK;
                        tma_load_2d(base + P::kABytes, &maps.w[0], xw, wrow, bar);
                        if (DUAL) tma_load_2d(base + P::kABytes + P::kBBytes / 2, &maps.w[1], xw, wrow, bar);
                        if (boxes == 4)
                            tma_load_2d(base, &maps.a128, xa, t.row0, bar);
                        else
                            for (int i = 0; i < boxes; ++i)
                                tma_load_2d(base + i * 32 * kStepBytes, &maps.a32, xa, t.row0 + 32 * i, bar);
                    }
                } else if (leader) {
                    const int bytes = min(P::kTilesK, ct - ks * P::kTilesK) * kScaleTile;
                    const uint32_t sfa = smem0 + P::kSfAt + st * P::kSfBytes, sfb = sfa + P::kSfaBytes;
                    const size_t k0 = (size_t)ks * P::kTilesK * kScaleTile;
                    mbar_arrive_expect_tx(bar, bytes * (second ? 3 : 2));
                    bulk_load(sfb, pb + k0, bytes, bar);
                    if (second) bulk_load(sfb + P::kSfbBytes / 2, pc + k0, bytes, bar);
                    bulk_load(sfa, pa + k0, bytes, bar);
                }
                ++issued;
                if (++st == P::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        // the newest copy of each stage lands before the CTA leaves, whoever gave up
        for (int i = 0; i < min(issued, P::kStages); ++i) {
            if (--st < 0) {
                st = P::kStages - 1;
                ph ^= 1;
            }
            mbar_wait(smem_u32(&sh.full[st]), ph, 1 << 20, nullptr);
        }
    } else if (warp == 1) {
        // ---- MMAs
        const uint32_t leader = elect_one();
        int st = 0, acc = 0;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        const uint32_t sf0 = tmem + P::kAccs * BN;
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            // columns of the first weight row inside its scale row tile (32 rows a column)
            const uint32_t sub = P::kOutN % kScaleRows ? (uint32_t)(tile % n_tiles * P::kOutN % kScaleRows) / 32 : 0;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.acc_empty[acc]), aph ^ 1, a.wait_limit, abort));
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            for (int ks = ks0; ok && ks < ks1; ++ks) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.full[st]), ph, a.wait_limit, abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t base = smem0 + st * P::kCodeBytes;
                const uint32_t sfa = sf0 + st * P::kSfCols, sfb = sfa + 4 * P::kTilesK + sub;
                const uint32_t sfa_s = smem0 + P::kSfAt + st * P::kSfBytes, sfb_s = sfa_s + P::kSfaBytes;
#pragma unroll
                for (int j = 0; j < P::kTilesK; ++j) {
                    tmem_cp_scales<1>(sfa + 4 * j, desc_scales(sfa_s + j * kScaleTile), leader);
#pragma unroll
                    for (int c = 0; c < P::kChunks; ++c)
                        tmem_cp_scales<1>(sfa + 4 * (P::kTilesK + P::kChunks * j + c),
                                       desc_scales(sfb_s + (c * P::kTilesK + j) * kScaleTile), leader);
                }
                const uint64_t ad = desc_sw128(base), bd = desc_sw128(base + P::kABytes);
                const int kk = (a.K - ks * P::kStepK) / (P::kStepK / 4);          // instructions left along K
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // 32 bytes along K inside the swizzle atom
                    const uint32_t id = idesc_scaled<FMT>(128, P::kMmaN, P::kNv ? 0 : j), go = ks > ks0 || j > 0;
                    const uint32_t sa = sfa + (P::kNv ? 4 * j : 0), sb = sfb + (P::kNv ? 4 * P::kChunks * j : 0);
                    const uint32_t on = leader & (uint32_t)(j < kk);
                    mma_scaled<FMT, 1>(d, ad + 2 * j, bd + 2 * j, id, sa, sb, go, on);
                    if (P::kMmaN != BN)
                        mma_scaled<FMT, 1>(d + P::kMmaN, ad + 2 * j, bd + 2 * j + (P::kMmaN * kStepBytes >> 4), id, sa, sb + 4, go, on);
                }
                if (leader) mma_commit(smem_u32(&sh.empty[st]));
                if (++st == P::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
            if (leader) mma_commit(smem_u32(&sh.acc_full[acc]));
            if (++acc == P::kAccs) {
                acc = 0;
                aph ^= 1;
            }
        }
        // the products end before the CTA leaves, whoever gave up: an epilogue that did waits for none of them
        if (leader) {
            if (!ok) fail();
            mma_commit(smem_u32(&sh.drain));
        }
        __syncwarp();
        mbar_wait(smem_u32(&sh.drain), 0, 1 << 20, nullptr);
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- accumulators to outputs
        // two warps share a quarter of the rows, each with half of the tile's output columns
        constexpr int kCols = P::kOutN / 2;
        const int quad = warp & 3, half = (warp - 4) >> 2;
        int acc = 0;
        uint32_t aph = 0;
        for (int tile = first_tile; tile < total; tile += stride) {
            const Tile t = tile_at<kScaleRows>(a, sh, tile, n_tiles);
            const int r = quad * 32 + lane, col0 = t.nt * P::kOutN + half * kCols;
            const uint32_t d = tmem + acc * BN + half * kCols + ((uint32_t)(quad * 32) << 16);
            const bool any = quad * 32 < t.rows && col0 < a.N, live = any && r < t.rows;
            const size_t row = (size_t)t.row0 + r;
            // factors on their way under the products
            const float rs = live && a.a_row_scale ? a.a_row_scale[row] : 1.0f;
            const float s0 = rs * (a.alpha[0] ? a.alpha[0][t.g] : 1.0f);
            const float s1 = DUAL ? rs * (a.alpha[1] ? a.alpha[1][t.g] : 1.0f) : 1.0f;
            const float ginv = DUAL && P::kNv ? __fdiv_rn(1.0f, a.h_gscale[t.g]) : 1.0f;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.acc_full[acc]), aph, a.wait_limit, abort))) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            // the accumulators go to registers and are free for the next tile's products before anything is
            // computed from them or stored
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.acc_empty[acc]));
            };
            const float4 *part = nullptr;
            if constexpr (SPLIT) {
                // each CTA finishes half of the columns and hands the other half's sums over
                float4 *const mine = reinterpret_cast<float4 *>(smem + P::kPartAt) + quad * 8 * P::kPartCols;
                if (half != rank) {
                    if (any) {
                        const uint32_t to = mapa_u32(smem_u32(mine), rank ^ 1) + lane * 16;
#pragma unroll
                        for (int i = 0; i < P::kPartCols; i += 16) {
                            uint32_t u[16];
                            // a SwiGLU tile's up products follow its gate products of all the tile's columns
                            tmem_ld16(d + (DUAL && i >= kCols ? BN / 2 - kCols + i : i), u);
                            tmem_ld_wait();
#pragma unroll
                            for (int c = 0; c < 4; ++c) st_cluster_v4(to + (i / 4 + c) * 512, u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
                        }
                        fence_cluster();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa_u32(smem_u32(&sh.part[quad]), rank ^ 1));
                    }
                    release();
                    break;                                                // these columns are the other CTA's from here on
                }
                if (any) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(smem_u32(&sh.part[quad]), 0, a.wait_limit, abort))) {
                        if (lane == 0) fail();
                        break;
                    }
                    part = mine;
                }
            }
            if (!any) {
                release();
            } else if constexpr (!DUAL) {
                store_rows<kCols, P::kStaged>(a, d, (size_t)t.row0 + quad * 32, t.rows - quad * 32, col0, s0, lane,
                                  smem + P::kOutAt + (warp - 4) * (P::kOutBytes / 8), part, release);
            } else {
                uint32_t u[kCols / 16][16], u2[kCols / 16][16];          // gate and up products
#pragma unroll
                for (int i = 0; i < kCols / 16; ++i) {
                    tmem_ld16(d + 16 * i, u[i]);
                    tmem_ld16(d + BN / 2 + 16 * i, u2[i]);
                }
                tmem_ld_wait();
                release();
#pragma unroll
                for (int i = 0; i < kCols / 16; ++i) {
                    add_part(u[i], part, 16 * i, lane);
                    add_part(u2[i], part, kCols + 16 * i, lane);
                }
                const int hct = scaled_col_tiles(FMT, a.N);
                const long long srow = (long long)t.srow_tile * kScaleRows + r;
                constexpr int kBlk = scaled_block(FMT), kWords = kCols / (P::kNv ? 8 : 4);
                uint32_t q[kWords], word = 0;                   // codes and scale bytes of the warp's columns
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float h[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        h[i] = silu(__uint_as_float(u[(c + i) / 16][i % 16]) * s0) * (__uint_as_float(u2[(c + i) / 16][i % 16]) * s1);
#pragma unroll
                    for (int i0 = 0; i0 < 32; i0 += kBlk) {
                        uint32_t m = 0;
#pragma unroll
                        for (int i = 0; i < kBlk; ++i) m = max(m, __float_as_uint(h[i0 + i]) & 0x7FFFFFFFu);
                        uint32_t sc;
                        float inv;
                        if (P::kNv) {
                            sc = nvfp4_scale(m, ginv, inv);
                        } else {
                            sc = pow2_scale<MOE_SCALED_MXFP8>(m);
                            inv = pow2_inverse(sc);
                        }
                        word |= sc << (8 * ((c + i0) / kBlk));
#pragma unroll
                        for (int i = 0; i < kBlk; i += 8) {
                            float e[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) e[k] = h[i0 + i + k] * inv;
                            if (P::kNv) {
                                q[(c + i0 + i) / 8] = to_e2m1x8(e);
                            } else {
                                q[(c + i0 + i) / 4] = to_e4m3x2(e[1], e[0]) | ((uint32_t)to_e4m3x2(e[3], e[2]) << 16);
                                q[(c + i0 + i) / 4 + 1] = to_e4m3x2(e[5], e[4]) | ((uint32_t)to_e4m3x2(e[7], e[6]) << 16);
                            }
                        }
                    }
                }
                if (live) {
                    uint4 *p = reinterpret_cast<uint4 *>(a.h_codes + (P::kNv ? (row * a.N + col0) / 2 : row * a.N + col0));
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) p[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
                    uint8_t *ps = a.h_scales + scale_at(srow, col0 / kBlk, hct);
                    if (kCols / kBlk == 4) *reinterpret_cast<uint32_t *>(ps) = word;
                    else if (kCols / kBlk == 2) *reinterpret_cast<uint16_t *>(ps) = (uint16_t)word;
                    else *ps = (uint8_t)word;
                }
            }
            if (++acc == P::kAccs) {
                acc = 0;
                aph ^= 1;
            }
        }
    }
    __syncthreads();
    if (SPLIT) cluster_sync();                                        // no store of the second CTA is on its way any more
    if (warp == 3) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ a pair of CTAs on one tile
//
// Large groups: two SMs share a tile of 256 rows x 256 outputs (cta_group::2).  Each holds the codes of its own
// 128 rows and of half of the weights, so that a step brings an SM 38 KB in place of 54 KB for the same
// products, and five stages fit in place of three: the one-CTA kernel waits a third of its time for a refilled
// stage.  The first CTA issues the products of both; all copies of a stage complete on its barrier, and its
// commits arrive in both.

template <int FMT>
struct PairPlan {
    static constexpr bool kNv = FMT == MOE_SCALED_NVFP4;
    static constexpr int kStepK = kNv ? 256 : 128, kTilesK = kNv ? 4 : 1;
    static constexpr int kABytes = 128 * kStepBytes, kBBytes = 128 * kStepBytes;
    static constexpr int kBTxBytes = kNv ? kBBytes : kBBytes / 2;
    static constexpr int kSfBytes = kTilesK * kScaleTile;                   // one row tile's scales of a step
    static constexpr int kCodeBytes = kABytes + kBBytes;
    static constexpr int kStages = kNv ? 5 : 6;
    static constexpr int kSfCols = 4 * kTilesK * 3;
    static constexpr int kSfAt = kStages * kCodeBytes, kOutAt = kSfAt + kStages * 3 * kSfBytes;
    static constexpr int kSmem = kOutAt + 16384 + 1024;
    static_assert(256 + kStages * kSfCols <= 512, "tensor memory");
};
constexpr int kPairRows = 256;

struct PairMaps {
    CUtensorMap a, w, sa, sw;              // codes; scale tiles as rows of 128 words
};

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
scaled_pair_kernel(const __grid_constant__ ScaledGemmArgs a, const __grid_constant__ PairMaps maps)
{
    using P = PairPlan<FMT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    uint8_t *smem = align_smem_1024(smem_raw);
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), first_tile = blockIdx.x >> 1, stride = gridDim.x >> 1;
    const int n_tiles = (a.N + 255) / 256, n_steps = (a.K + P::kStepK - 1) / P::kStepK;
    const int ct = scaled_col_tiles(FMT, a.K), w_row_tiles = (a.N + kScaleRows - 1) / kScaleRows;

    pdl_trigger();
    if (threadIdx.x == 0) {
        prefetch_map(&maps.a);
        prefetch_map(&maps.w);
        prefetch_map(&maps.sa);
        prefetch_map(&maps.sw);
        for (int i = 0; i < P::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 2);                      // codes and scales (of both CTAs, in the first)
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        mbar_init(smem_u32(&sh.acc_full[0]), 1);
        mbar_init(smem_u32(&sh.acc_empty[0]), 16);                    // the epilogue warps of both CTAs
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = sh.gave_up = 0;
        sh.bad = 0;
        sh.row_tiles = (a.R + kPairRows - 1) / kPairRows;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc_pair(smem_u32(&sh.tmem), 512);
        tmem_relinquish_pair();
    }
    __syncthreads();
    pdl_wait();
    if (a.offsets) build_table<kPairRows>(a, sh, warp, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                                   // the barriers of both CTAs are there
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
    const int total = __shfl_sync(0xFFFFFFFFu, sh.row_tiles * n_tiles, 0);
    volatile int *abort = &sh.abort;
    const uint32_t smem0 = smem_u32(smem);
    auto fail = [&]() {
        record_status(a.status, MOE_ERR_TIMEOUT);
        *abort = 1;
    };
    auto tell_pair = [&]() {
        for (uint32_t c = 0; c < 2; ++c) st_cluster_u32(mapa_u32(smem_u32(&sh.gave_up), c), 1);
    };

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || warp == 2) {
        // ---- copies: warp 0 the codes, warp 2 the scales, each CTA its own; they complete on the first CTA's barrier
        const bool leader = elect_one();
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            const Tile t = tile_at<kPairRows>(a, sh, tile, n_tiles);
            const int n0 = t.nt * 256, wrow = t.g * a.N + n0 + rank * 128, arow = t.row0 + rank * 128;
            const int sa = (t.srow_tile + rank) * ct, sw = (t.g * w_row_tiles + n0 / kScaleRows) * ct;
            for (int ks = 0; ks < n_steps; ++ks) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.empty[st]), ph ^ 1, a.wait_limit, abort));
                if (!ok) {
                    if (leader) fail();
                    break;
                }
                const uint32_t base = smem0 + st * P::kCodeBytes, bar = mapa_u32(smem_u32(&sh.full[st]), 0);
                if (warp == 0) {
                    if (leader) {
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[st]), 2 * (P::kABytes + P::kBTxBytes));
                        tma_load_2d_pair(base + P::kABytes, &maps.w, P::kNv ? ks * kStepBytes : ks * P::kStepK, wrow, bar);
                        tma_load_2d_pair(base, &maps.a, ks * kStepBytes, arow, bar);
                    }
                } else if (leader) {
                    const uint32_t sf = smem0 + P::kSfAt + st * 3 * P::kSfBytes;
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[st]), 2 * 3 * P::kSfBytes);
                    tma_load_2d_pair(sf, &maps.sa, 0, sa + ks * P::kTilesK, bar);
                    tma_load_2d_pair(sf + P::kSfBytes, &maps.sw, 0, sw + ks * P::kTilesK, bar);
                    tma_load_2d_pair(sf + 2 * P::kSfBytes, &maps.sw, 0, sw + ct + ks * P::kTilesK, bar);
                }
                ++issued;
                if (++st == P::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (leader) {
            st_cluster_u32(mapa_u32(smem_u32(&sh.issued[rank][warp >> 1]), 0), issued);
            if (!ok) tell_pair();
        }
    } else if (warp == 1 && rank == 0) {
        // ---- MMAs of the pair
        const uint32_t leader = elect_one();
        int st = 0;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        const uint32_t sf0 = tmem + 256;
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(smem_u32(&sh.acc_empty[0]), aph ^ 1, a.wait_limit, abort));
            tc_fence_after();
            for (int ks = 0; ok && ks < n_steps; ++ks) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(smem_u32(&sh.full[st]), ph, a.wait_limit, abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t base = smem0 + st * P::kCodeBytes, sf = smem0 + P::kSfAt + st * 3 * P::kSfBytes;
                const uint32_t sfa = sf0 + st * P::kSfCols, sfb = sfa + 4 * P::kTilesK;
#pragma unroll
                for (int j = 0; j < P::kTilesK; ++j) {
                    tmem_cp_scales<2>(sfa + 4 * j, desc_scales(sf + j * kScaleTile), leader);
                    tmem_cp_scales<2>(sfb + 8 * j, desc_scales(sf + P::kSfBytes + j * kScaleTile), leader);
                    tmem_cp_scales<2>(sfb + 8 * j + 4, desc_scales(sf + 2 * P::kSfBytes + j * kScaleTile), leader);
                }
                const uint64_t ad = desc_sw128(base), bd = desc_sw128(base + P::kABytes);
                const int kk = (a.K - ks * P::kStepK) / (P::kStepK / 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_scaled<FMT, 2>(tmem, ad + 2 * j, bd + 2 * j, idesc_scaled<FMT>(256, 256, P::kNv ? 0 : j),
                                       sfa + (P::kNv ? 4 * j : 0), sfb + (P::kNv ? 8 * j : 0), ks > 0 || j > 0,
                                       leader & (uint32_t)(j < kk));
                if (leader) mma_commit_pair(smem_u32(&sh.empty[st]));
                if (++st == P::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
            if (leader) mma_commit_pair(smem_u32(&sh.acc_full[0]));
            aph ^= 1;
        }
        // the products end before the pair leaves, whoever gave up
        if (leader) {
            if (!ok) {
                fail();
                tell_pair();
            }
            mma_commit_pair(smem_u32(&sh.drain));
        }
        __syncwarp();
        mbar_wait(smem_u32(&sh.drain), 0, 1 << 20, nullptr);
    } else if (warp >= 4) {
        // ---- accumulators to outputs: each CTA its own rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int quad = warp & 3, half = (warp - 4) >> 2;
        uint32_t aph = 0;
        const uint32_t empty = mapa_u32(smem_u32(&sh.acc_empty[0]), 0);
        for (int tile = first_tile; tile < total; tile += stride) {
            const Tile t = tile_at<kPairRows>(a, sh, tile, n_tiles);
            const int r0 = rank * 128 + quad * 32, r = r0 + lane, col0 = t.nt * 256 + half * 128;
            const bool any = r0 < t.rows && col0 < a.N, live = any && r < t.rows;
            const size_t row = (size_t)t.row0 + r;
            const float s = (live && a.a_row_scale ? a.a_row_scale[row] : 1.0f) * (a.alpha[0] ? a.alpha[0][t.g] : 1.0f);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(smem_u32(&sh.acc_full[0]), aph, a.wait_limit, abort))) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(empty);
            };
            if (any)
                store_rows<128, 64>(a, tmem + half * 128 + ((uint32_t)(quad * 32) << 16), (size_t)t.row0 + r0, t.rows - r0, col0, s, lane,
                                smem + P::kOutAt + (warp - 4) * 2048, nullptr, release);
            else release();
            aph ^= 1;
        }
    }
    __syncthreads();
    cluster_sync();                                                   // nothing of the pair is issued any more
    // commits arrive in both CTAs: the last of them, of all products, is there before the second one's shared memory goes
    if (rank == 1 && warp == 1) mbar_wait(smem_u32(&sh.drain), 0, 1 << 20, nullptr);
    if (sh.gave_up) {
        // Where nobody gave up, the products have waited for every copy of both CTAs.  Else the newest copy of each stage may
        // still be on its way, whichever of the four warps asked for it: none is more than the stages ahead of another.  A
        // stage that not all four asked for does not complete, and its wait runs out long after its copies have landed.
        if (rank == 0 && warp == 0) {
            const int n = max(max(sh.issued[0][0], sh.issued[0][1]), max(sh.issued[1][0], sh.issued[1][1])), i = n - 1 - lane;
            if (lane < min(n, P::kStages)) mbar_wait(smem_u32(&sh.full[i % P::kStages]), i / P::kStages & 1, 1 << 20, nullptr);
        }
        __syncthreads();
        cluster_sync();
    }
    if (warp == 3) tmem_dealloc_pair(tmem, 512);
}

// Scale tiles as rows of 128 32-bit words, in boxes of `box` tiles.
bool make_map_scales(CUtensorMap *m, const uint8_t *p, uint64_t tiles, uint32_t box)
{
    return make_map_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, kScaleTile / 4, tiles, kScaleTile / 4, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int FMT>
cudaError_t launch_pair(const ScaledGemmArgs &a, int clusters, cudaStream_t st)
{
    using P = PairPlan<FMT>;
    PairMaps maps;
    const uint64_t ct = scaled_col_tiles(FMT, a.K), wrt = (a.N + kScaleRows - 1) / kScaleRows;
    bool ok = make_map_2d(&maps.a, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, P::kNv ? a.K / 2 : a.K, a.R, kStepBytes, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B) &&
              make_map_scales(&maps.sa, a.a_scales, (uint64_t)(a.R / kScaleRows + a.G) * ct, P::kTilesK) &&
              make_map_scales(&maps.sw, a.w_scales[0], (uint64_t)a.G * wrt * ct, P::kTilesK);
    ok = ok && (P::kNv ? make_map_2d(&maps.w, a.w_codes[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.K / 2, (uint64_t)a.G * a.N, kStepBytes,
                                     128, CU_TENSOR_MAP_SWIZZLE_128B)
                       : make_map_4bit(&maps.w, a.w_codes[0], a.K, (uint64_t)a.G * a.N, 128));
    if (!ok) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> ready{0};
    static_assert(P::kSmem + sizeof(Shared) <= 227 * 1024, "shared memory");
    const cudaError_t e = set_shared(scaled_pair_kernel<FMT>, P::kSmem, ready);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(scaled_pair_kernel<FMT>, 2 * clusters, 2, kThreads, P::kSmem, st, a, maps);
}

template <int FMT, bool DUAL, int BN, bool SPLIT = false>
cudaError_t launch_plan(const ScaledGemmArgs &a, const Maps &maps, int ctas, cudaStream_t st)
{
    using P = Plan<FMT, DUAL, BN, SPLIT>;
    auto k = scaled_gemm_kernel<FMT, DUAL, BN, SPLIT>;
    static_assert(P::kSmem + sizeof(Shared) <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = set_shared(k, P::kSmem, ready);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(k, ctas, SPLIT ? 2 : 1, kThreads, P::kSmem, st, a, maps);
}

template <int FMT, bool DUAL>
cudaError_t launch_fmt(const ScaledGemmArgs &a, cudaStream_t st)
{
    constexpr bool kNv = FMT == MOE_SCALED_NVFP4;
    const int sms = device_sm_count();
    // row tiles at most: every group's last one may be partial
    const long long mt = a.offsets ? a.R / kScaleRows + (a.G < a.R ? a.G : a.R) : (a.R + kScaleRows - 1) / kScaleRows;
    auto tiles = [&](int out_n) { return mt * ((a.N + out_n - 1) / out_n); };
    if constexpr (!DUAL) {
        // A pair of CTAs a tile: groups of 256 rows and more on average, a tile for every pair of SMs, and K steps
        // enough to pay for the longer way of a tile's first and last step.  us, one CTA / a pair: 8192 x 8192 x
        // 4096 NVFP4 (16 steps) 119 / 105, MXFP8 (32) 192 / 156, 8192 x 8192 x 2048 NVFP4 (8) 72.6 / 64.7, 4096 x 4096 x
        // 1024 MXFP8 (8) 20.3 / 19.8; 5627 x 3400 x 896 MXFP8 (7) 22.1 / 22.3, 8192 x 2048 x 512 (4) 13.7 / 15.4;
        // 1024 x 4096 x 4096 NVFP4 (64 pair tiles for 76 pairs) 10.6 / 11.0.
        using P = PairPlan<FMT>;
        const long long pairs = (a.R / kPairRows) * ((long long)(a.N + 255) / 256), ct = scaled_col_tiles(FMT, a.K);
        const bool coords = ((long long)a.G * ((a.N + kScaleRows - 1) / kScaleRows) + 1) * ct < 0x7FFFFFFFll &&
                            ((long long)a.R / kScaleRows + a.G + 1) * ct < 0x7FFFFFFFll;   // scale tiles as 32-bit coordinates
        if (a.R / a.G >= kPairRows && pairs >= sms / 2 && a.K >= 8 * P::kStepK && coords) return launch_pair<FMT>(a, sms / 2, st);
    }
    // The widest tile, or the narrowest of which there is at most one an SM.  us at 64 / 128 / 256 columns: 1 x 16384
    // x 2048 NVFP4 (256, 128, 64 tiles) 6.9 / 5.2 / 5.9, 512 x 4096 x 4096 (256, 128, 64) 11.6 / 7.9 / 10.4, 64 x 8192
    // x 4096 MXFP8 (128, 64, 32) 9.5 / 9.8 / 12.3, 256 x 4096 x 4096 (128, 64, 32) 7.3 / 7.5 / 9.0; experts of 512
    // tokens: the SwiGLU pair 56 us with 128, 51 with 256, the down products 39 with 128, 32 with 256.
    int bn = 256;
    if (tiles(DUAL ? 64 : 128) <= sms) bn = 128;
    if (!DUAL && tiles(64) <= sms) bn = 64;
    const long long n = tiles(DUAL ? bn / 2 : bn);
    const int ctas = (int)(n < sms ? n : sms);
    constexpr int kNarrow = DUAL ? 128 : 64, kStepK = kNv ? 256 : 128;
    // Half of the K steps on a second CTA, where they are worth the exchange (about 1 us, and the clusters start later
    // behind another launch).  us, one CTA / two, with the quantisation of the rows, at 14, 20 and 32 steps: 16 x 4096 NVFP4
    // 7.4 / 7.1, 9.2 / 8.2, 12.5 / 10.2, MXFP8 6.8 / 6.7, 8.1 / 7.4, 10.6 / 8.8; 301 x 1000 NVFP4 8.6 / 8.9, 10.8 / 9.8, 14.1 / 12.0, MXFP8
    // 7.5 / 8.1, 8.9 / 9.3, 11.6 / 10.8.
    const bool split = bn == kNarrow && 2 * n <= sms && a.K >= (a.R <= 64 ? 14 : 24) * kStepK;
    Maps maps;
    const uint64_t abytes = kNv ? a.K / 2 : a.K;
    bool ok = make_map_2d(&maps.a32, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, abytes, a.R, kStepBytes, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    maps.a128 = maps.a32;                                // up to 96 rows the kernel takes 32 at a time
    maps.w[1] = CUtensorMap{};
    if (a.R > 96)
        ok = ok && make_map_2d(&maps.a128, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, abytes, a.R, kStepBytes, 128,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    for (int i = 0; i < (DUAL ? 2 : 1); ++i) {
        const uint8_t *w = a.w_codes[i];
        const uint32_t box = DUAL ? bn / 2 : bn;
        if (kNv)
            ok = ok && make_map_2d(&maps.w[i], w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.K / 2, (uint64_t)a.G * a.N, kStepBytes,
                                   box, CU_TENSOR_MAP_SWIZZLE_128B);
        else
            ok = ok && make_map_4bit(&maps.w[i], w, a.K, (uint64_t)a.G * a.N, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (split) return launch_plan<FMT, DUAL, kNarrow, true>(a, maps, 2 * (int)n, st);
    if (bn == 256) return launch_plan<FMT, DUAL, 256>(a, maps, ctas, st);
    if (bn == 128) return launch_plan<FMT, DUAL, 128>(a, maps, ctas, st);
    if constexpr (!DUAL) return launch_plan<FMT, DUAL, 64>(a, maps, ctas, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_scaled_gemm(const ScaledGemmArgs &a, int fmt, bool swiglu, cudaStream_t st)
{
    // Few rows a row at a time (scaled_vec.cu): up to 10240 outputs, more where groups would share no tiles anyway.
    // us, tiles / rows: 1 x 4096 x 2048 (4096 outputs) NVFP4 4.5 / 2.8, MXFP8 5.9 / 2.8; 2 x 4096 x 2048 (8192) 4.5 / 3.8, 5.8 / 3.5;
    // 2 x 4096 x 8192 (8192) 8.5 / 8.5, 11.4 / 7.9; 4 x 4096 x 2048 (16384) 4.5 / 6.4, 5.9 / 5.9; the SwiGLU of 1, 2 and 3 tokens
    // of 9 experts each, inter 512 (9216, 18432, 27648 gate and up outputs) NVFP4 7.4 / 4.7, 7.9 / 6.7, 9.3 / 11.2; their down
    // products (18432, 36864, 55296) 4.4 / 3.8, 5.0 / 4.2, 6.2 / 6.1.  A single step (K <= 256) the same: K = 256, NVFP4, 1 x 4096
    // 2.4 / 1.7, 1 x 10240 2.6 / 2.2, 9 groups' rows x 2048 3.6 / 2.9, 40 x 1024 5.4 / 4.1; K = 128, MXFP8, 2.3 / 1.6, 2.5 / 2.0,
    // 3.5 / 2.7, 5.0 / 4.1; but where rows must share groups their tiles are few (1280 x 32 to 20 x 2048 in 3 groups 3.1 to 3.6 / 4.0,
    // at half as many outputs 3.1 to 3.6 / 3.2).  The SwiGLU alone keeps its single steps in tiles (one token's of inter 512 4.2 / 2.5): hidden <= 256 is
    // a test's size, and there a layer's bounded waits are to be met at one token too.
    const long long outputs = (long long)a.R * ((a.N + 31) / 32 * 32) * (swiglu ? 2 : 1);
    const int most = !a.offsets ? 10240 : a.K <= 512 && (a.K > 256 || a.G >= a.R) ? 40960 : 20480;
    if (outputs <= most && !(swiglu && a.K <= 256)) return launch_scaled_vec(a, fmt, swiglu, st);
    if (fmt == MOE_SCALED_NVFP4)
        return swiglu ? launch_fmt<MOE_SCALED_NVFP4, true>(a, st) : launch_fmt<MOE_SCALED_NVFP4, false>(a, st);
    return swiglu ? launch_fmt<MOE_SCALED_MXFP8, true>(a, st) : launch_fmt<MOE_SCALED_MXFP8, false>(a, st);
}

}  // namespace qmoe
