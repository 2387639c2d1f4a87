// Grouped products of bf16 rows with bf16 matrices on the tensor cores, with their epilogue, and their weight gradients.
//
//   NT  y[r, n]  = act(sum over the pairs of a[r] . w_g[n] + bias_g[n]) + residual[r, n]      w [G, N, K]
//       GLU: y[r, n] = act(a[r] . gate_g[n] + ..) (a[r] . up_g[n] + ..)
//   NN  the same with w [G, K, N]: the input gradient of an NT product
//   TN  dw_g[n, k] (+)= sum over group g's rows r of dy[r, n] x[r, k]
//
// All sums are fp32, in tensor memory.  An operand whose rows run along the sum (K-major: a, w of NT) is copied as rows of 64
// elements, one whose rows run across it (MN-major: w of NN, dy, x of TN) as blocks of 64 columns x 64 terms; either is 128-byte
// swizzled shared memory that tcgen05.mma reads in place, so no operand is ever transposed.
// Tiles of 128 outputs' rows x BN columns, 64 terms a step, in a ring of stages; two accumulators, so that a tile leaves
// tensor memory under the next one's products.  Where a group's rows end inside a tile the rest is computed and not
// written (NT, NN); where they end inside a step of a sum (TN) a warp overwrites the rest of both operands with zeros
// before the products read it, since those rows are other groups' and may hold anything.
//
// One CTA per SM walks over the tiles: warp 0 copies (TMA), warp 1 issues the products, warp 2 clears the ends of sums,
// warps 4-11 read the accumulators and write.  Few tiles share out their steps (SPLIT), large ones go to pairs of CTAs (PAIR).
//
// Bounds and measurements: 8192 x 8192 x 4096 with bias, GELU and residual 310 to 330 us (1.7 PFLOP/s; 291 to 297 without them, where the
// library's product alone takes 271 to 279): tensor cores, and what the epilogue takes from them.  Its tiles are
// 1,024 for 76 pairs of SMs; 4096 x 2048 x 4096 43 us for 39 of the library's, 128 tiles in two rounds of 76.
// Experts of 512 tokens (hidden 2048, inter 512, 257 groups): gated pair 165 us (171 with both products kept), down products 87, 6.4 and 6.2 TB/s of weights.  Of 4096
// tokens: input gradients 117 and 200 us (6.2 and 6.5 TB/s), weight gradients 139 to 141 each for 730 MB (5.2 TB/s, three
// quarters of it writes; groups of 3 rows, whose writes are all, 88 us).  There no unit is full (tensor pipe 21%, DRAM 40% where half of
// the output stays in L2): copies wait behind writes in a ring of four stages, and the write of a tile's 64 KB takes 2,100 of its
// 4,300 cycles.  301 x 1000 x 2184 9.9 us: 18 steps of 0.2 us on each of two CTAs a tile, 24 KB a step being near what an SM takes in,
// the exchange of their sums (2 us) and a launch.
#include "bf16.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kMaxGroups = 1024;
constexpr int kStep = 64;                          // terms of a step: 128 bytes of a K-major row
constexpr int kBlockBytes = 64 * 128;              // an MN-major block: 64 terms x 64 columns
constexpr int kSliceBytes = 16 * 128;              // one of 16 terms
// fp32 outputs: steps after which a tile's sums leave tensor memory, to be added up in registers.  The tensor cores' additions do not
// round to nearest, so that their error grows with the number of terms, not its root (2-norm, 512, 1024, 2048, 4096 and 8192 terms in
// one go: 4.7e-7, 1.0e-6, 2.1e-6, 2.1e-6, 4.4e-6; fp32 on the other units 1.6e-7 to 9.6e-7).
// bf16 outputs: 8192 terms of one sign lose at most 512 times 2^-24 of their sum, 1/64 of the rounding to come (262,144 in one go
// lost 6e-4, and a third of the outputs were rounded to the wrong value).
constexpr int kSegmentF32 = 12, kSegment16 = 128;
enum Kind { kNT, kNN, kTN };

template <int KIND, bool DUAL, int BN, bool PAIR, int SPLIT>
struct Plan {
    static constexpr int kOutN = DUAL ? BN / 2 : BN;                 // output columns of a tile
    static constexpr int kRows = PAIR ? 256 : 128;                   // output rows of a tile
    static constexpr int kHeld = PAIR ? BN / 2 : BN;                 // columns of the second operand in this CTA
    static constexpr int kABytes = 128 * 128, kBBytes = kHeld * 128, kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = PAIR ? 5 : BN == 256 ? 4 : BN == 128 ? (SPLIT > 1 ? 4 : 5) : 7;
    // an epilogue warp's 32 rows at a time: 128 bytes of each where the table of groups leaves room and a warp has them
    static constexpr int kRowBytes = (KIND != kTN && !PAIR && BN == 256) || kOutN == 64 || (DUAL && BN == 256) ? 64 : 128;
    static constexpr int kOutBytes = SPLIT > 1 ? 0 : 8 * 32 * kRowBytes;
    static constexpr int kMats = DUAL ? 2 : 1;
    static constexpr int kPartBytes = SPLIT > 1 ? kMats * kOutN * 128 * 4 : 0;   // all CTAs' sums of them
    static constexpr int kOutAt = kStages * kStageBytes, kPartAt = kOutAt + kOutBytes, kSmem = kPartAt + kPartBytes + 1024;
    static_assert(SPLIT == 1 || (kMats * kOutN <= 128 && !PAIR), "shared memory of the sums");
};

struct Maps {
    CUtensorMap a[2], a32[2], w[2];                  // first operand(s) in whole and in 32-row boxes, second operand(s)
    CUtensorMap a16, w16;                            // TN: both operands in boxes of 16 terms
    CUtensorMap y, pre[2];                           // outputs, in an epilogue warp's boxes of 32 rows
};

// What a launch computes.
struct ProductArgs {
    const int32_t *offsets;
    const uint16_t *bias[2], *residual;
    uint16_t *pre[2];
    void *y;
    int *status;
    int R, M, N, K, G;                               // rows; TN: output rows of a matrix; output columns; terms (NT, NN)
    int pairs, act, y_f32, accumulate;
    int blocks_a, blocks_w;                          // MN-major operands whose maps bring all of a tile's blocks in one copy
    long long wait_limit;
};

template <int KIND>
struct Shared {
    uint64_t full[8], empty[8], tail[8], cleared[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    int bad, groups, row_tiles;                      // malformed offsets; groups with rows; their row tiles
    int gave_up, issued[2];                          // a pair's: whether any of its waits ran out; copies of each CTA
    int2 warp_sum[kThreads / 32];
    int2 group[KIND == kTN ? 1 : kMaxGroups + 1];    // those groups: row tiles before it, start << 10 | group
};

constexpr int kGroupBits = 10;
static_assert(kMaxGroups == 1 << kGroupBits, "the table's packing");

struct Tile {
    int g, row0, rows, col0;                         // first output row (of all rows; TN: of the matrix), how many, first column
    int first, terms;                                // TN: first row of the sum, rows of it
};

// The groups with rows and the tiles before each (NT, NN); a check of the offsets alone (TN).  Every thread takes part.
template <int KIND, int ROWS>
__device__ __forceinline__ void build_table(const ProductArgs &a, Shared<KIND> &sh, int warp, int lane)
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
    if (KIND == kTN) {
        __syncthreads();
        if (threadIdx.x == 0 && sh.bad) {
            sh.row_tiles = 0;
            record_status(a.status, MOE_ERR_DEVICE);
        }
        return;
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
        if (o[i + 1] <= o[i] || sh.bad) continue;
        sh.group[base.y] = make_int2(base.x, o[i] << kGroupBits | (g0 + i));
        base.x += (o[i + 1] - o[i] + ROWS - 1) / ROWS;
        base.y += 1;
    }
    if (threadIdx.x == kThreads - 1) {
        sh.groups = base.y;
        sh.row_tiles = sh.bad ? 0 : base.x;
        if (!sh.bad) sh.group[base.y] = make_int2(base.x, (int)((uint32_t)a.R << kGroupBits));
        if (sh.bad) record_status(a.status, MOE_ERR_DEVICE);
    }
}

// Quotients by a divisor of the launch: floor(2^32 / d) is found once, and an estimate with it is one short at most.  (A tile found
// with divisions cost each role 1,000 to 1,300 cycles, as much as two steps of products.)
struct Divisor {
    uint32_t d, m;
    __device__ __forceinline__ explicit Divisor(int by) : d((uint32_t)by), m(0xFFFFFFFFu / (uint32_t)by) {}
    __device__ __forceinline__ int operator()(int x) const
    {
        const uint32_t q = __umulhi((uint32_t)x, m);
        return (int)(q + ((uint32_t)x - q * d >= d));
    }
};

// Tile `tile`: kBand row tiles of a column follow each other, then those of the next column, so that what the SMs work on at a
// time shares rows and columns.
// (Weight gradients of several groups by rows of tiles: the groups share nothing, and those worked on at a time are few; runs of tiles of
// equal cost for each CTA, or the tiles of a shared expert with all tokens first, were 138 to 195 us and no better where this takes 122 and 140.)
constexpr int kBand = 8;
struct TileShape {
    Divisor n, band, per;                                    // column tiles; those of a band of rows; TN: row tiles of a matrix
    __device__ __forceinline__ TileShape(int n_tiles, int row_tiles) : n(n_tiles), band(kBand * n_tiles), per(row_tiles) {}
};
template <int KIND, int ROWS, int OUT_N>
__device__ __forceinline__ Tile tile_at(const ProductArgs &a, const Shared<KIND> &sh, int tile, const TileShape &shape)
{
    int mt, nt;
    if (KIND == kTN && a.offsets) {
        mt = shape.n(tile);
        nt = tile - mt * (int)shape.n.d;
    } else {
        const int band = shape.band(tile), in = tile - band * (int)shape.band.d, high = sh.row_tiles - band * kBand;
        nt = high >= kBand ? in / kBand : in / high;
        mt = band * kBand + in - nt * min(high, kBand);
    }
    Tile t;
    t.col0 = nt * OUT_N;
    t.first = t.terms = 0;
    if (KIND == kTN) {
        t.g = shape.per(mt);
        t.row0 = (mt - t.g * (int)shape.per.d) * ROWS;
        t.rows = min(a.M - t.row0, ROWS);
        t.first = a.offsets ? a.offsets[t.g] : 0;
        t.terms = (a.offsets && t.g + 1 < a.G ? a.offsets[t.g + 1] : a.R) - t.first;
        return t;
    }
    if (!a.offsets) {
        t.g = 0;
        t.row0 = mt * ROWS;
        t.rows = min(a.R - t.row0, ROWS);
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
    return t;
}

// ------------------------------------------------------------------ descriptors

// An MN-major operand in the 128-byte swizzle: blocks of 64 columns (rows of 128 bytes, one term a row), 8 terms 1024 bytes
// apart (stride byte offset), the next 64 columns a block further (leading byte offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block = kBlockBytes)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// kind::f16 with bf16 operands: D f32 [4,6) = 1, A and B bf16 [7,10), [10,13) = 1, A and B MN-major [15], [16].
template <int KIND>
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t m, uint32_t n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (KIND == kTN ? 1u << 15 : 0u) | (KIND != kNT ? 1u << 16 : 0u) | ((n >> 3) << 17) |
           ((m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate, uint32_t issue)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::%6.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issue), "n"(CG)
        : "memory");
}
// A copy of up to four dimensions; PAIR: completes on a barrier of either CTA of the pair (a cluster address).
template <bool PAIR>
__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5}], "
            "[%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
            : "memory");
}
// BLOCKS blocks of 64 columns from column `col` on x TERMS terms from `row` on of matrix g: one copy where the map has the blocks as a
// dimension, else the first `some` of them one by one.
template <bool PAIR, int BLOCKS, int TERMS>
__device__ __forceinline__ void load_blocks(uint32_t dst, const CUtensorMap *map, bool at_once, int some, int col, int row, int g, uint32_t bar)
{
    if (at_once) {
        load_4d<PAIR>(dst, map, 0, row, col / 64, g, bar);
        return;
    }
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
        if (i < some) load_4d<PAIR>(dst + i * TERMS * 128, map, col + 64 * i, row, 0, g, bar);
}

// ------------------------------------------------------------------ epilogue

// 32 rows of B bytes (64 or 128), a lane a row in 16-byte chunks, into `stage`: row r's chunk k lies at k ^ r / 2 or k ^ r of the
// row (the 64- and 128-byte swizzles), so that no bank is met twice in a phase.  The copy engine has read what it was last
// given from there.
template <int B>
__device__ __forceinline__ int chunk_at(int r, int k) { return r * B + ((k ^ (B == 64 ? r >> 1 : r)) & (B / 16 - 1)) * 16; }
template <int B>
__device__ __forceinline__ void stage_rows(const uint32_t *w, int lane, uint8_t *stage)
{
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < B / 16; ++k)
        *reinterpret_cast<uint4 *>(stage + chunk_at<B>(lane, k)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}
// The first `rows` rows and `chunks` chunks of each to rows `pitch` bytes apart from `dst` on: 4 or 8 lanes write a row's bytes
// together.  ADD: fp32 values added to what is there.
template <int B, bool ADD>
__device__ __forceinline__ void store_staged(uint8_t *dst, size_t pitch, const uint32_t *w, int rows, int chunks, int lane, uint8_t *stage)
{
    constexpr int kLanes = B / 16;
    stage_rows<B>(w, lane, stage);
    __syncwarp();
    const int k = lane % kLanes;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
        const int r = (i * 32 + lane) / kLanes;
        uint4 v = *reinterpret_cast<const uint4 *>(stage + chunk_at<B>(r, k));
        if (r < rows && k < chunks) {
            uint4 *p = reinterpret_cast<uint4 *>(dst + r * pitch + 16 * k);
            if (ADD) {
                const uint4 o = *p;
                v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(o.x));
                v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(o.y));
                v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(o.z));
                v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(o.w));
            }
            *p = v;
        }
    }
    __syncwarp();
}
// The same through the copy engine, which leaves out what lies past the map's last row and column.  A lane of its own row
// touches 32 lines in every store, and through shared memory and back 64 wavefronts of the load/store unit are needed for 32
// columns; this way 16 (weight gradients of 64 experts, one step a tile: 5,000 cycles a tile with plain stores).
template <int KIND, int B>
__device__ __forceinline__ void store_box(const CUtensorMap *map, int col, int row, int g, const uint32_t *w, int lane, uint8_t *stage)
{
    stage_rows<B>(w, lane, stage);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (KIND == kTN)
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(map)),
                         "r"(col), "r"(row), "r"(g), "r"(smem_u32(stage))
                         : "memory");
        else
            tma_store_2d(map, col, row, smem_u32(stage));
        bulk_commit();
    }
}
// The other way: the lane's row of up to B bytes.
template <int B>
__device__ __forceinline__ void load_staged(uint32_t *w, const uint8_t *src, size_t pitch, int rows, int chunks, int lane, uint8_t *stage)
{
    constexpr int kLanes = B / 16;
    const int k = lane % kLanes;
    uint4 v[kLanes];
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
        const int r = (i * 32 + lane) / kLanes;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < rows && k < chunks) v[i] = *reinterpret_cast<const uint4 *>(src + r * pitch + 16 * k);
    }
#pragma unroll
    for (int i = 0; i < kLanes; ++i) *reinterpret_cast<uint4 *>(stage + chunk_at<B>((i * 32 + lane) / kLanes, k)) = v[i];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kLanes; ++j) {
        const uint4 u = *reinterpret_cast<const uint4 *>(stage + chunk_at<B>(lane, j));
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
    }
    __syncwarp();
}

// Adds the bias of N columns (of which `cols` exist) to a row.
template <int N>
__device__ __forceinline__ void add_bias(float *v, const uint16_t *bias, int cols)
{
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        if (8 * i >= cols) break;
        const uint4 b = reinterpret_cast<const uint4 *>(bias)[i];
        const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[8 * i + 2 * k] += bf16_lo(u[k]);
            v[8 * i + 2 * k + 1] += bf16_hi(u[k]);
        }
    }
}
template <int N>
__device__ __forceinline__ void apply(int act, float (&v)[N])
{
    switch (act) {
    case MOE_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value(MOE_ACT_SILU, v[i]);
        break;
    case MOE_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value(MOE_ACT_GELU, v[i]);
        break;
    case MOE_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value(MOE_ACT_RELU, v[i]);
        break;
    default: break;
    }
}
template <int N>
__device__ __forceinline__ void load_columns(uint32_t d, float (&v)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        uint32_t r[16];
        tmem_ld16(d + c, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c + i] = __uint_as_float(r[i]);
    }
}

// Adds N accumulator columns to the sums in registers.
template <int N>
__device__ __forceinline__ void add_columns(uint32_t d, float (&v)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 32) {
        float w[32];
        load_columns(d + c, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[c + i] += w[i];
    }
}

// The warp's 32 rows x COLS columns of a tile (v; u: the up products) to the outputs.  row: the first row's index (TN: in its
// matrix), of which `rows` exist; whole: no row of another group follows within the 32.
template <int KIND, bool DUAL, int COLS, int B>
__device__ __forceinline__ void finish(const ProductArgs &a, const Maps &maps, float (&v)[COLS], float (&u)[DUAL ? COLS : 1], int g, int row, int rows,
                                       bool whole, int col0, int lane, uint8_t *stage)
{
    const size_t n = a.N;
    const size_t first = KIND == kTN ? (size_t)g * a.M + row : (size_t)row;
    constexpr int kC = B / 2, kF = B / 4;                            // bf16 and fp32 columns of B bytes
    auto put16 = [&](const CUtensorMap *map, uint16_t *out, const float *from, int c, int cols) {
        uint32_t w[kC / 2];
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) w[i] = pack_bf16(from[2 * i], from[2 * i + 1]);
        if (whole) store_box<KIND, B>(map, col0 + c, row, g, w, lane, stage);
        else store_staged<B, false>(reinterpret_cast<uint8_t *>(out + first * n + col0 + c), n * 2, w, rows, cols / 8, lane, stage);
    };
    if (KIND != kTN) {
#pragma unroll
        for (int c = 0; c < COLS; c += kC) {
            const int cols = a.N - col0 - c;
            if (cols <= 0) break;
            if (a.bias[0]) add_bias<kC>(v + c, a.bias[0] + g * n + col0 + c, cols);
            if (a.pre[0]) put16(&maps.pre[0], a.pre[0], v + c, c, cols);
            if constexpr (DUAL) {
                if (a.bias[1]) add_bias<kC>(u + c, a.bias[1] + g * n + col0 + c, cols);
                if (a.pre[1]) put16(&maps.pre[1], a.pre[1], u + c, c, cols);
            }
        }
        apply(a.act, v);
        if constexpr (DUAL) {
#pragma unroll
            for (int i = 0; i < COLS; ++i) v[i] *= u[i];
        }
    }
#pragma unroll
    for (int c = 0; c < COLS; c += kC) {
        const int cols = a.N - col0 - c;
        if (cols <= 0) break;
        if (KIND != kTN && !DUAL && a.residual) {
            uint32_t w[kC / 2];
            load_staged<B>(w, reinterpret_cast<const uint8_t *>(a.residual + first * n + col0 + c), n * 2, rows, cols / 8, lane, stage);
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
                v[c + 2 * i] += bf16_lo(w[i]);
                v[c + 2 * i + 1] += bf16_hi(w[i]);
            }
        }
        if (DUAL || !a.y_f32) {
            put16(&maps.y, static_cast<uint16_t *>(a.y), v + c, c, cols);
            continue;
        }
        if constexpr (!DUAL) {
#pragma unroll
            for (int h = 0; h < kC; h += kF) {
                if (h >= cols) break;
                uint32_t w[kF];
#pragma unroll
                for (int i = 0; i < kF; ++i) w[i] = __float_as_uint(v[c + h + i]);
                uint8_t *y = reinterpret_cast<uint8_t *>(static_cast<float *>(a.y) + first * n + col0 + c + h);
                if (KIND == kTN && a.accumulate) store_staged<B, true>(y, n * 4, w, rows, (cols - h) / 4, lane, stage);
                else if (whole) store_box<KIND, B>(&maps.y, col0 + c + h, row, g, w, lane, stage);
                else store_staged<B, false>(y, n * 4, w, rows, (cols - h) / 4, lane, stage);
            }
        }
    }
}

// A split tile's columns that this CTA finishes, from all CTAs' sums: part[(source, matrix, column / 4)][row] of four columns.
template <int KIND, bool DUAL, int COLS, int SPLIT>
__device__ __forceinline__ void finish_split(const ProductArgs &a, const float4 *part, const Tile &t, int col0)
{
    constexpr int kMats = DUAL ? 2 : 1, kSegs = COLS / 8;
    const size_t n = a.N, first = KIND == kTN ? (size_t)t.g * a.M + t.row0 : (size_t)t.row0;
    for (int i = threadIdx.x; i < t.rows * kSegs; i += kThreads) {
        const int r = i / kSegs, seg = i - r * kSegs, col = col0 + 8 * seg;
        if (col >= a.N) continue;
        float v[kMats][8];
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[m][e] = 0.f;
#pragma unroll
            for (int s = 0; s < SPLIT; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 p = part[((s * kMats + m) * (COLS / 4) + 2 * seg + h) * 128 + r];
                    v[m][4 * h] += p.x;
                    v[m][4 * h + 1] += p.y;
                    v[m][4 * h + 2] += p.z;
                    v[m][4 * h + 3] += p.w;
                }
        }
        const size_t at = (first + r) * n + col;
        auto add16 = [&](float (&x)[8], const uint16_t *p) {
            const uint4 b = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] += bf16_lo(w[k]);
                x[2 * k + 1] += bf16_hi(w[k]);
            }
        };
        auto put16 = [&](uint16_t *p, const float (&x)[8]) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        };
        if (KIND != kTN) {
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
                if (a.bias[m]) add16(v[m], a.bias[m] + t.g * n + col);
                if (a.pre[m]) put16(a.pre[m] + at, v[m]);
            }
            apply(a.act, v[0]);
            if (DUAL) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[0][e] *= v[kMats - 1][e];
            }
            if (!DUAL && a.residual) add16(v[0], a.residual + at);
        }
        if (DUAL || !a.y_f32) {
            put16(static_cast<uint16_t *>(a.y) + at, v[0]);
            continue;
        }
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(a.y) + at);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 o = make_float4(v[0][4 * h], v[0][4 * h + 1], v[0][4 * h + 2], v[0][4 * h + 3]);
            if (KIND == kTN && a.accumulate) {
                const float4 p = y[h];
                o = make_float4(o.x + p.x, o.y + p.y, o.z + p.z, o.w + p.w);
            }
            y[h] = o;
        }
    }
}

// ------------------------------------------------------------------ the kernel
//
// SPLIT: few tiles, where the steps one after the other are the time: a cluster of SPLIT CTAs shares out a tile's steps;
// each CTA finishes its part of the tile's columns from all CTAs' sums, which meet in its shared memory, in their order.
//
// PAIR: two SMs share a tile of 256 x 256 (cta_group::2): each holds its own 128 rows of the first operand and half of the
// second's columns, so that a step brings an SM 32 KB in place of 48 KB for the same products.  The first CTA issues the
// products of both; a stage's copies complete on its barrier, and its commits arrive in both.  A step whose end has to
// be cleared completes on each CTA's own barrier first, and counts once both have cleared their part.

template <int KIND, bool DUAL, int BN, bool PAIR, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ Maps maps)
{
    using P = Plan<KIND, DUAL, BN, PAIR, SPLIT>;
    constexpr int kCluster = PAIR ? 2 : SPLIT;
    [[maybe_unused]] constexpr int kPartCols = P::kOutN / SPLIT;     // columns that this CTA of a split tile finishes
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared<KIND> sh;
    uint8_t *smem = align_smem_1024(smem_raw);
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0, part = SPLIT > 1 ? (int)cluster_ctarank() : 0;
    const int first_tile = blockIdx.x / kCluster, stride = gridDim.x / kCluster;
    const int n_tiles = (a.N + P::kOutN - 1) / P::kOutN, k_steps = (a.K + kStep - 1) / kStep;
    const TileShape shape(n_tiles, KIND == kTN ? (a.M + P::kRows - 1) / P::kRows : 1);

    pdl_trigger();
    if (threadIdx.x == 0) {
        prefetch_map(&maps.a[0]);
        prefetch_map(&maps.w[0]);
        if (DUAL) prefetch_map(&maps.w[1]);
        for (int i = 0; i < P::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            mbar_init(smem_u32(&sh.tail[i]), 1);
            mbar_init(smem_u32(&sh.cleared[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), PAIR ? 16 : 8);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = sh.gave_up = 0;
        sh.bad = 0;
        sh.row_tiles = KIND == kTN ? a.G * ((a.M + P::kRows - 1) / P::kRows) : (a.R + P::kRows - 1) / P::kRows;
        fence_mbar_init();
    }
    if (warp == 3) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(&sh.tmem), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&sh.tmem), 512);
            tmem_relinquish();
        }
    }
    __syncthreads();
    if (kCluster > 1) cluster_arrive();
    pdl_wait();
    if (a.offsets) build_table<KIND, P::kRows>(a, sh, warp, lane);
    tc_fence_before();
    __syncthreads();
    if (kCluster > 1) cluster_wait();                                 // the barriers of all its CTAs are there
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
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, PAIR ? mbar_wait_cluster(bar, parity, a.wait_limit, abort) : mbar_wait(bar, parity, a.wait_limit, abort));
    };
    auto steps_of = [&](const Tile &t) { return KIND == kTN ? (t.terms + kStep - 1) / kStep : a.pairs * k_steps; };
    // this CTA's steps of a tile
    auto first_step = [&](int steps) { return SPLIT > 1 ? steps * part / SPLIT : 0; };
    auto last_step = [&](int steps) { return SPLIT > 1 ? steps * (part + 1) / SPLIT : steps; };
    // whether it has the last step of a sum that ends inside it, before the last of all rows (past which the copies bring zeros)
    auto to_clear = [&](const Tile &t) {
        return KIND == kTN && t.terms % kStep != 0 && t.first + t.terms < a.R &&
               (SPLIT == 1 || (last_step(steps_of(t)) == steps_of(t) && first_step(steps_of(t)) < steps_of(t)));
    };

    // A role's warp walks its loop as a whole and only the issuing instructions are one lane's (scaled_gemm.cu).
    // registers: 384 x 168 at launch, redistributed by warpgroup to 104 and 2 x 200 (the same total)
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0) {
        // ---- copies, each CTA its own.  What a step costs this one warp in instructions delays the copy: the place in the ring is
        // carried on, whole steps have a loop of their own.
        const bool leader = elect_one();
        int st = 0, issued = 0;
        uint32_t ph = 0, base = smem0;
        bool ok = true;
        // the next stage, once its last products are done
        auto acquire = [&]() {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.empty[0]) + 8 * st, ph ^ 1, a.wait_limit, abort));
            if (!ok && leader) fail();
            return ok;
        };
        auto advance = [&]() {
            ++issued;
            base += P::kStageBytes;
            if (++st == P::kStages) {
                st = 0;
                ph ^= 1;
                base = smem0;
            }
        };
        const uint32_t full0 = PAIR ? mapa_u32(smem_u32(&sh.full[0]), 0) : smem_u32(&sh.full[0]);   // copies complete there
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            const Tile t = tile_at<KIND, P::kRows, P::kOutN>(a, sh, tile, shape);
            const int steps = steps_of(t), ks0 = first_step(steps), ks1 = last_step(steps), row = t.row0 + rank * 128, mine = t.rows - rank * 128;
            // the second operand's columns of this CTA, and how many blocks of 64 of them exist
            const int c0 = t.col0 + rank * P::kHeld, blocks = PAIR || a.blocks_w ? P::kHeld / 64 : min(P::kHeld / 64, (a.N - c0 + 63) / 64);
            if constexpr (KIND == kTN) {
                const int ablocks = a.blocks_a || PAIR || mine > 64 ? 2 : 1, bytes = (ablocks + blocks) * kBlockBytes, whole = min(ks1, t.terms / kStep);
                int r = t.first + ks0 * kStep;
#pragma unroll 1
                for (int ks = ks0; ks < whole; ++ks, r += kStep) {
                    if (!acquire()) break;
                    if (leader) {
                        const uint32_t bar = full0 + 8 * st;
                        if (!PAIR) mbar_arrive_expect_tx(bar, bytes);
                        else if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[0]) + 8 * st, 2 * P::kStageBytes);
                        load_blocks<PAIR, 2, kStep>(base, &maps.a[0], a.blocks_a, ablocks, row, r, 0, bar);
                        load_blocks<PAIR, P::kHeld / 64, kStep>(base + P::kABytes, &maps.w[0], a.blocks_w, blocks, c0, r, 0, bar);
                    }
                    advance();
                }
                if (ok && ks0 < ks1 && ks1 > whole && acquire()) {
                    // the end of a sum, in slices of 16 terms: those that have some
                    if (leader) {
                        const bool tail = to_clear(t);
                        const int slices = (t.terms - whole * kStep + 15) / 16, part = (ablocks + blocks) * slices * kSliceBytes;
                        const uint32_t local = smem_u32(tail ? &sh.tail[st] : &sh.full[st]), bar = PAIR ? mapa_u32(local, tail ? rank : 0) : local;
                        if (!PAIR || tail) mbar_arrive_expect_tx(local, part);
                        else if (rank == 0) mbar_arrive_expect_tx(local, 2 * part);
                        for (int j = 0; j < slices; ++j) {
                            load_blocks<PAIR, 2, 16>(base + j * 2 * kSliceBytes, &maps.a16, a.blocks_a, ablocks, row, r + 16 * j, 0, bar);
                            load_blocks<PAIR, P::kHeld / 64, 16>(base + P::kABytes + j * (P::kHeld / 64) * kSliceBytes, &maps.w16, a.blocks_w, blocks, c0,
                                                                 r + 16 * j, 0, bar);
                        }
                    }
                    advance();
                }
            } else {
                const int boxes = mine > 96 || PAIR ? 4 : (mine + 31) / 32, wrow = t.g * a.N + (PAIR && DUAL ? t.col0 : c0);
                const int bytes = boxes * 32 * 128 + (KIND == kNN ? blocks * kBlockBytes : P::kBBytes);
                int pair = ks0 >= k_steps, k = (ks0 - pair * k_steps) * kStep;
#pragma unroll 1
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!acquire()) break;
                    if (leader) {
                        const uint32_t bar = full0 + 8 * st, w = base + P::kABytes;
                        if (!PAIR) mbar_arrive_expect_tx(bar, bytes);
                        else if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[0]) + 8 * st, 2 * P::kStageBytes);
                        if (KIND == kNN) {
                            load_blocks<PAIR, P::kHeld / 64, kStep>(w, &maps.w[pair], a.blocks_w, blocks, c0, k, t.g, bar);
                        } else if (PAIR) {
                            tma_load_2d_pair(w, &maps.w[DUAL ? rank : pair], k, wrow, bar);
                        } else {
                            tma_load_2d(w, &maps.w[DUAL ? 0 : pair], k, wrow, bar);
                            if (DUAL) tma_load_2d(w + P::kBBytes / 2, &maps.w[1], k, wrow, bar);
                        }
                        if (PAIR)
                            tma_load_2d_pair(base, &maps.a[pair], k, row, bar);
                        else if (boxes == 4)
                            tma_load_2d(base, &maps.a[pair], k, row, bar);
                        else
                            for (int i = 0; i < boxes; ++i) tma_load_2d(base + i * 32 * 128, &maps.a32[pair], k, row + 32 * i, bar);
                    }
                    advance();
                    k += kStep;
                    if (ks + 1 == k_steps) {
                        pair = 1;
                        k = 0;
                    }
                }
            }
        }
        if (PAIR) {
            if (leader) {
                st_cluster_u32(mapa_u32(smem_u32(&sh.issued[rank]), 0), issued);
                if (!ok) tell_pair();
            }
        } else {
            // the newest copy of each stage lands before the CTA leaves, whoever gave up
            for (int i = 0; i < min(issued, P::kStages); ++i) {
                if (--st < 0) {
                    st = P::kStages - 1;
                    ph ^= 1;
                }
                mbar_wait(smem_u32(&sh.full[st]), ph, 1 << 20, nullptr);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- products
        const uint32_t leader = elect_one();
        int st = 0, acc = 0;
        uint32_t ph = 0, aph = 0, cph = 0;                              // cph: a bit a stage
        bool ok = true;
        const uint64_t ad0 = KIND == kTN ? desc_mn(smem0) : desc_sw128(smem0);
        const uint64_t bd0 = KIND == kNT ? desc_sw128(smem0 + P::kABytes) : desc_mn(smem0 + P::kABytes);
        constexpr uint32_t kNextA = KIND == kTN ? kSliceBytes >> 4 : 2, kNextB = KIND == kNT ? 2 : kSliceBytes >> 4;   // from instruction to instruction
        auto commit = [&](uint32_t bar) {
            if (leader) {
                if (PAIR) mma_commit_pair(bar);
                else mma_commit(bar);
            }
        };
        for (int tile = first_tile; ok && tile < total; tile += stride) {
            const Tile t = tile_at<KIND, P::kRows, P::kOutN>(a, sh, tile, shape);
            const int steps = steps_of(t), ks0 = first_step(steps), ks1 = last_step(steps);
            // columns past the last are not multiplied (whole instructions of 16)
            const uint32_t id = idesc_bf16<KIND>(P::kRows, PAIR || DUAL ? BN : min(BN, (a.N - t.col0 + 15) & ~15));
            ok = wait(smem_u32(&sh.acc_empty[acc]), aph ^ 1);
            tc_fence_after();
            uint32_t d = tmem + acc * BN, more = 0;                   // more: there are sums in the accumulators
            // the accumulators are the epilogue's, and the next ones this warp's
            auto hand_over = [&]() {
                commit(smem_u32(&sh.acc_full[acc]));
                if (++acc == 2) {
                    acc = 0;
                    aph ^= 1;
                }
            };
            auto leave_stage = [&]() {
                commit(smem_u32(&sh.empty[0]) + 8 * st);
                if (++st == P::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            };
            // whole steps
            const int whole = KIND == kTN ? min(ks1, t.terms / kStep) : ks1;
            const int segment = !DUAL && a.y_f32 ? kSegmentF32 : kSegment16;
            int left = segment;
#pragma unroll 1
            for (int ks = ks0; ok && ks < whole; ++ks) {
                if (left-- == 0) {
                    hand_over();
                    ok = wait(smem_u32(&sh.acc_empty[acc]), aph ^ 1);
                    if (!ok) break;
                    tc_fence_after();
                    d = tmem + acc * BN;
                    more = 0;
                    left = segment - 1;
                }
                ok = wait(smem_u32(&sh.full[0]) + 8 * st, ph);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = ad0 + st * (P::kStageBytes >> 4), bd = bd0 + st * (P::kStageBytes >> 4);
                // instructions of 16 terms: 32 bytes along K-major rows, 16 rows of MN-major blocks; the last step of K may have fewer
                int kk = 4;
                if (KIND != kTN && (ks + 1 == k_steps || ks + 1 == 2 * k_steps)) kk = (a.K - (k_steps - 1) * kStep + 15) / 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_bf16<PAIR ? 2 : 1>(d, ad + j * kNextA, bd + j * kNextB, id, more, KIND == kTN ? leader : leader & (uint32_t)(j < kk));
                    more = 1;
                }
                leave_stage();
            }
            if (KIND == kTN && ok && ks0 < ks1 && ks1 > whole) {
                // the end of a sum, in slices of 16 terms, a block of each behind the other
                if (left == 0) {
                    hand_over();
                    ok = wait(smem_u32(&sh.acc_empty[acc]), aph ^ 1);
                    tc_fence_after();
                    d = tmem + acc * BN;
                    more = 0;
                }
                ok = ok && wait(smem_u32(&sh.full[st]), ph);
                if (PAIR && ok && to_clear(t)) {
                    ok = wait(smem_u32(&sh.cleared[st]), cph >> st & 1);
                    cph ^= 1u << st;
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t base = smem0 + st * P::kStageBytes;
                const uint64_t ad = desc_mn(base, kSliceBytes), bd = desc_mn(base + P::kABytes, kSliceBytes);
                const int slices = (t.terms - whole * kStep + 15) / 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_bf16<PAIR ? 2 : 1>(d, ad + j * (2 * kSliceBytes >> 4), bd + j * ((P::kHeld / 64) * kSliceBytes >> 4), id, more,
                                           leader & (uint32_t)(j < slices));
                    more = 1;
                }
                leave_stage();
            }
            if (!ok) break;
            hand_over();
        }
        // the products end before the CTA leaves, whoever gave up
        if (leader) {
            if (!ok) {
                fail();
                if (PAIR) tell_pair();
            }
            if (PAIR) mma_commit_pair(smem_u32(&sh.drain));
            else mma_commit(smem_u32(&sh.drain));
        }
        __syncwarp();
        mbar_wait(smem_u32(&sh.drain), 0, 1 << 20, nullptr);
    } else if (warp == 2 && KIND == kTN) {
        // ---- zeros for what the last step of a sum holds of other groups' rows; its copies complete on a barrier of their
        // own, and the stage's is this warp's to complete
        int it = 0;
        uint32_t tph = 0;                                               // a bit a stage
        for (int tile = first_tile; tile < total; tile += stride) {
            const Tile t = tile_at<KIND, P::kRows, P::kOutN>(a, sh, tile, shape);
            it += last_step(steps_of(t)) - first_step(steps_of(t));
            if (!to_clear(t)) continue;
            const int st = (int)((uint32_t)(it - 1) % P::kStages);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sh.tail[st]), tph >> st & 1, a.wait_limit, abort))) {
                if (lane == 0) {
                    fail();
                    if (PAIR) tell_pair();
                }
                break;
            }
            tph ^= 1u << st;
            // terms up to the end of the last slice, 8 lanes a row
            const int lo = t.terms % kStep, slice = lo / 16;
            uint8_t *const base = smem + st * P::kStageBytes + lane % 8 * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lo % 16 + lane / 8 + 4 * i;
                if (r < 16 && lo % 16) {
#pragma unroll
                    for (int block = 0; block < 2; ++block)
                        *reinterpret_cast<uint4 *>(base + (slice * 2 + block) * kSliceBytes + r * 128) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int block = 0; block < P::kHeld / 64; ++block)
                        *reinterpret_cast<uint4 *>(base + P::kABytes + (slice * (P::kHeld / 64) + block) * kSliceBytes + r * 128) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster(mapa_u32(smem_u32(&sh.cleared[st]), 0));
                if (rank == 0) mbar_arrive(smem_u32(&sh.full[st]));
            }
        }
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- accumulators to outputs: two warps share a quarter of the rows, each with half of the output columns
        constexpr int kCols = P::kOutN / 2;
        const int quad = warp & 3, half = (warp - 4) >> 2;
        uint8_t *const stage = smem + P::kOutAt + (warp - 4) * (P::kOutBytes / 8);
        int acc = 0;
        uint32_t aph = 0;
        for (int tile = first_tile; tile < total; tile += stride) {
            const Tile t = tile_at<KIND, P::kRows, P::kOutN>(a, sh, tile, shape);
            const int r0 = rank * 128 + quad * 32, col0 = t.col0 + half * kCols;
            const int steps = last_step(steps_of(t)) - first_step(steps_of(t));
            const int segments = max(1, !DUAL && a.y_f32 ? (steps + kSegmentF32 - 1) / kSegmentF32 : (steps + kSegment16 - 1) / kSegment16);
            const bool any = r0 < t.rows && (SPLIT > 1 || col0 < a.N);
            float v[kCols], u[DUAL ? kCols : 1];
            if (KIND != kTN && !DUAL && any && a.residual && lane < t.rows - r0) {
                // on its way to L2 under the products
                const uint16_t *p = a.residual + (size_t)(t.row0 + r0 + lane) * a.N + col0;
                for (int c = 0; c < min(kCols, a.N - col0); c += 64) prefetch_l2_line(p + c);
            }
            bool ok = true;
            for (int seg = 0; seg < segments; ++seg) {
                ok = wait(smem_u32(&sh.acc_full[acc]), aph);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN + half * kCols + ((uint32_t)(quad * 32) << 16);
                if (any) {
                    // to registers before anything is computed from them or stored: free for later products
                    if (seg) {
                        add_columns(d, v);
                        if constexpr (DUAL) add_columns(d + BN / 2, u);
                    } else {
                        load_columns(d, v);
                        if constexpr (DUAL) load_columns(d + BN / 2, u);
                        tmem_ld_wait();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(mapa_u32(smem_u32(&sh.acc_empty[acc]), 0));
                    else mbar_arrive(smem_u32(&sh.acc_empty[acc]));
                }
                if (++acc == 2) {
                    acc = 0;
                    aph ^= 1;
                }
            }
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            if (!any) continue;
            if (steps == 0) {
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    v[i] = 0.f;
                    if (DUAL) u[DUAL ? i : 0] = 0.f;
                }
            }
            if constexpr (SPLIT > 1) {
                const uint32_t parts = smem_u32(smem + P::kPartAt) + (quad * 32 + lane) * 16;
#pragma unroll
                for (int m = 0; m < P::kMats; ++m)
#pragma unroll
                    for (int j = 0; j < kCols / 4; ++j) {
                        const int c = half * kCols + 4 * j, to = c / kPartCols, at = c % kPartCols / 4;
                        const float *const f = m ? u : v;
                        st_cluster_v4(mapa_u32(parts + ((part * P::kMats + m) * (kPartCols / 4) + at) * 128 * 16, to), __float_as_uint(f[4 * j]),
                                      __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3]));
                    }
            } else {
                finish<KIND, DUAL, kCols, P::kRowBytes>(a, maps, v, u, t.g, t.row0 + r0, t.rows - r0,
                                                        KIND == kTN || t.rows - r0 >= 32 || t.row0 + t.rows == a.R, col0, lane, stage);
            }
        }
        if (SPLIT == 1 && lane == 0) bulk_wait<0>();                  // what was written through the copy engine is there
    }
    __syncthreads();
    if constexpr (SPLIT > 1) {
        cluster_sync();                                               // all CTAs' sums are there
        if (first_tile < total && !*abort) {
            const Tile t = tile_at<KIND, P::kRows, P::kOutN>(a, sh, first_tile, shape);
            finish_split<KIND, DUAL, kPartCols, SPLIT>(a, reinterpret_cast<const float4 *>(smem + P::kPartAt), t, t.col0 + part * kPartCols);
        }
    }
    if (PAIR) {
        cluster_sync();                                               // nothing of the pair is issued any more
        // commits arrive in both CTAs: the last of them, of all products, is there before the second one's shared memory goes
        if (rank == 1 && warp == 1) mbar_wait(smem_u32(&sh.drain), 0, 1 << 20, nullptr);
        if (sh.gave_up) {
            // Where nobody gave up, the products have waited for every copy of both CTAs.  Else the newest copy of each stage
            // may still be on its way, of either CTA: neither is more than the stages ahead of the other.  A stage that not
            // both asked for does not complete, and its wait runs out long after its copies have landed.
            if (rank == 0 && warp == 0) {
                const int n = max(sh.issued[0], sh.issued[1]), i = n - 1 - lane;
                if (lane < min(n, P::kStages)) mbar_wait(smem_u32(&sh.full[i % P::kStages]), i / P::kStages & 1, 1 << 20, nullptr);
            }
            __syncthreads();
            cluster_sync();
        }
    }
    if (warp == 3) {
        if (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// Rows of outputs in boxes of 32 rows x `bytes`: [rows, cols], or with G > 0 [G, rows, cols].
bool map_out(CUtensorMap *m, void *p, bool f32, uint64_t cols, uint64_t rows, uint64_t G, uint32_t bytes)
{
    const CUtensorMapSwizzle swz = bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType type = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint32_t size = f32 ? 4 : 2;
    if (!G) return make_map_2d(m, p, type, size, cols, rows, bytes / size, 32, swz);
    const uint64_t dims[3] = {cols, rows, G}, strides[2] = {cols * size, cols * rows * size};
    const uint32_t box[3] = {bytes / size, 32, 1};
    return make_map_3d(m, p, type, dims, strides, box, swz);
}

template <int KIND, bool DUAL, int BN, bool PAIR, int SPLIT = 1>
cudaError_t launch_plan(const ProductArgs &a, Maps &maps, int ctas, cudaStream_t st)
{
    using P = Plan<KIND, DUAL, BN, PAIR, SPLIT>;
    if (SPLIT == 1) {
        bool ok = map_out(&maps.y, a.y, a.y_f32, a.N, KIND == kTN ? a.M : a.R, KIND == kTN ? a.G : 0, P::kRowBytes);
        for (int i = 0; i < 2; ++i)
            if (a.pre[i]) ok = ok && map_out(&maps.pre[i], a.pre[i], false, a.N, a.R, 0, P::kRowBytes);
        if (!ok) return cudaErrorInvalidValue;
    }
    auto k = product_kernel<KIND, DUAL, BN, PAIR, SPLIT>;
    static_assert(P::kSmem + sizeof(Shared<KIND>) <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = set_shared(k, P::kSmem, ready);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(k, ctas, PAIR ? 2 : SPLIT, kThreads, P::kSmem, st, a, maps);
}
// How few tiles of about `steps` steps run: on one CTA each or shared out to S, of 64 columns or (long sums, not DUAL) of 128.
// us, 1 / 2 / 4 / 8 CTAs a tile: 16 rows x 1024 (16 tiles), K = 512 4.4 / 4.6 / 4.4 / -, 1024 6.2 / 5.4 / 4.9 / -, 2048 9.5 / 7.2 / 5.6 / -, 4096 16.4 /
// 10.8 / 7.5 / -; 128 rows x 512 (8 tiles), K = 512 4.6 / 5.2 / 4.6 / 4.6, 1024 6.4 / 6.1 / 5.1 / 4.9, 4096 16.4 / 11.3 / 7.7 / 6.1.  Clusters
// of 8 beyond 64 CTAs do not all find room at once (16 x 1024 x 1024 8.7).  128 columns exchange twice the sums: 301 x 1000 x 1024 6.3 with
// 64 columns on two CTAs, 7.6 with 128 on four; gradients of 1024 x 512 from 2048 rows 8.7 and 9.2, from 8192 rows 18.4 and 14.8.
struct Split {
    int bn, ways;
};
template <class Tiles>
Split split_of(Tiles tiles, bool wide, int steps, int sms)
{
    Split best{64, 1};
    int least = steps;                                     // of a CTA
    for (int bn = 64; bn <= (wide && steps >= 64 ? 128 : 64); bn *= 2)
        for (int s = 2; s <= 8; s *= 2) {
            const long long n = tiles(bn) * s;
            if (n > (s == 8 ? 64 : s == 4 ? 128 : sms) || steps < (s == 2 ? 10 : s == 4 ? 9 : 16)) continue;
            if ((steps + s - 1) / s < least) {
                least = (steps + s - 1) / s;
                best = Split{bn, s};
            }
        }
    return best;
}
template <int KIND, bool DUAL>
cudaError_t launch_narrow(const ProductArgs &a, Maps &maps, long long tiles, Split how, int sms, cudaStream_t st)
{
    constexpr int kBn = DUAL ? 128 : 64;
    const int ctas = (int)tiles * how.ways;
    if (!DUAL && how.bn == 128) {
        if constexpr (!DUAL) {
            if (how.ways == 2) return launch_plan<KIND, false, 128, false, 2>(a, maps, ctas, st);
            if (how.ways == 4) return launch_plan<KIND, false, 128, false, 4>(a, maps, ctas, st);
            return launch_plan<KIND, false, 128, false, 8>(a, maps, ctas, st);
        }
    }
    if (how.ways == 2) return launch_plan<KIND, DUAL, kBn, false, 2>(a, maps, ctas, st);
    if (how.ways == 4) return launch_plan<KIND, DUAL, kBn, false, 4>(a, maps, ctas, st);
    if (how.ways == 8) return launch_plan<KIND, DUAL, kBn, false, 8>(a, maps, ctas, st);
    return launch_plan<KIND, DUAL, kBn, false>(a, maps, (int)(tiles < sms ? tiles : sms), st);
}

// An MN-major operand, G matrices [terms, cols], in boxes of `box_terms` x 64 columns, or, where the columns are whole blocks of 64,
// of `blocks` of those at once: a copy costs its issue about 100 cycles (gradients of 257 groups of 143 rows, 2048 x 512, three steps of
// six copies a tile: of 3,940 cycles a tile the copies' warp had 2,350 of its own).
bool map_mn(CUtensorMap *m, const void *p, uint64_t cols, uint64_t terms, uint64_t G, uint32_t box_terms, uint32_t blocks, int *at_once)
{
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    *at_once = cols % 64 == 0;
    cuuint64_t dims[4] = {cols, terms, 1, G}, strides[3] = {cols * 2, cols * terms * 2, cols * terms * 2};
    cuuint32_t box[4] = {64, box_terms, 1, 1}, each[4] = {1, 1, 1, 1};
    if (*at_once) {
        dims[0] = 64;
        dims[2] = cols / 64;
        strides[1] = 128;
        box[2] = blocks;
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_2d(CUtensorMap *m, const void *p, uint64_t cols, uint64_t rows, uint32_t box_rows)
{
    return make_map_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, cols, rows, kStep, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// ------------------------------------------------------------------ column sums

// db_g (+)= sum over the group's rows of dy: a cluster of `parts` CTAs has 256 columns of one group, each a part of its rows; a
// warp reads 8 columns a lane of every kSumWarps-th row.  The parts meet in the first CTA in a fixed order.  Many warps, since
// the compiler keeps few of a thread's loads on their way (4096 x 4096 with 8 warps 34 us).
struct BiasArgs {
    const uint16_t *dy;
    const int32_t *offsets;
    void *db;
    int *status;
    int R, N, G, f32, accumulate, parts;
};
constexpr int kSumWarps = 32;

__global__ void __launch_bounds__(32 * kSumWarps) column_sum_kernel(const __grid_constant__ BiasArgs a)
{
    __shared__ float part[kSumWarps][256 + 8];
    __shared__ float total[8][256];                        // of each CTA of the cluster, in the first
    pdl_trigger();
    if (a.parts > 1) cluster_arrive();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = a.parts > 1 ? (int)cluster_ctarank() : 0;
    const int blocks = (a.N + 255) / 256, cluster = blockIdx.x / a.parts, g = cluster / blocks, n0 = (cluster - g * blocks) * 256;
    bool bad = false;
    int lo = 0, hi = a.R;
    if (a.offsets) {
        int b = 0;
        for (int i = threadIdx.x; i < a.G; i += 32 * kSumWarps) {
            const int o = a.offsets[i], next = i + 1 < a.G ? a.offsets[i + 1] : a.R;
            b |= o < 0 || o > a.R || next < o;
        }
        bad = __syncthreads_or(b);
        lo = a.offsets[g];
        hi = g + 1 < a.G ? a.offsets[g + 1] : a.R;
    }
    const int col = n0 + 8 * lane;
    float acc[8] = {};
    if (!bad && col < a.N) {
        const uint16_t *p = a.dy + col;
#pragma unroll 4
        for (int r = lo + rank * kSumWarps + warp; r < hi; r += kSumWarps * a.parts) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + (size_t)r * a.N);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[2 * e] += bf16_lo(w[e]);
                acc[2 * e + 1] += bf16_hi(w[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][8 * lane + e] = acc[e];
    __syncthreads();
    float s = 0.f;
    if (threadIdx.x < 256) {
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) s += part[i][threadIdx.x];
    }
    if (a.parts > 1) {
        cluster_wait();                                    // the first CTA is there
        if (threadIdx.x < 256) st_cluster_u32(mapa_u32(smem_u32(&total[rank][threadIdx.x]), 0), __float_as_uint(s));
        cluster_sync();
        if (rank) return;
        s = 0.f;
        if (threadIdx.x < 256)
            for (int i = 0; i < a.parts; ++i) s += total[i][threadIdx.x];
    }
    const int c = n0 + threadIdx.x;
    if (bad || threadIdx.x >= 256 || c >= a.N) return;
    const size_t at = (size_t)g * a.N + c;
    if (a.f32) {
        float *p = static_cast<float *>(a.db) + at;
        *p = a.accumulate ? *p + s : s;
    } else {
        static_cast<uint16_t *>(a.db)[at] = float_to_bf16_bits(s);
    }
}

template <int KIND, bool DUAL>
cudaError_t launch_rows_product(const GemmArgs &g, cudaStream_t st)
{
    ProductArgs a{};
    a.offsets = g.offsets;
    for (int i = 0; i < 2; ++i) {
        a.bias[i] = g.bias[i];
        a.pre[i] = g.pre[i];
    }
    a.residual = g.residual;
    a.y = g.y;
    a.status = g.status;
    a.R = g.R;
    a.N = g.N;
    a.K = g.K;
    a.G = g.G;
    a.pairs = g.pairs;
    a.act = g.act;
    a.y_f32 = g.y_f32;
    a.wait_limit = g.wait_limit;
    const int sms = device_sm_count();
    auto row_tiles = [&](int rows) -> long long {          // at most: every group's last one may be partial
        return a.offsets ? a.R / rows + (a.G < a.R ? a.G : a.R) : (a.R + rows - 1) / rows;
    };
    auto tiles = [&](int out_n) { return row_tiles(128) * ((a.N + out_n - 1) / out_n); };
    const long long pairs = (a.R / 256) * (long long)((a.N + (DUAL ? 127 : 255)) / (DUAL ? 128 : 256));
    // A pair of CTAs a tile: groups of 512 rows on average, a tile for every pair, and long sums or several tiles for each.  us, one CTA / a
    // pair: rows x N x K 4096 x 2048 x 512 10.3 / 11.6, x 1024 15.2 / 16.4, x 2048 24.8 / 25.0, x 4096 49.2 / 45.8; 16384 x 2048 x 512 (512
    // tiles) 30.2 / 28.1, x 1024 51.5 / 46.1; 1024 x 8192 x 8192 93.9 / 87.3; 64 groups of 256 x 2048 x 512 39.5 / 40.5, of 384 54.2 / 60.6,
    // of 512 x 512 x 2048 66.7 / 63.8 (gated pairs 66.0 / 71.5, 87.5 / 121.9, 103.9 / 93.1).
    const bool pair = a.R / a.G >= 512 && pairs >= sms / 2 && ((long long)a.K * a.pairs >= 2048 || pairs >= 3 * sms / 2);
    int bn = 256;
    // Else the widest tiles, or the narrowest of which there is about one an SM (groups of fewer rows than a tile have one row tile each).  us at
    // 64 / 128 / 256 columns: 512 rows x 2048 x 1024 (128, 64, 32 tiles) 7.5 / 7.6 / 9.6, x 4096 (256, 128, 64) 11.6 / 8.2 / 10.2, x 8192
    // (512, 256, 128) 19.2 / 12.3 / 10.2; 16 groups of 100 x 1024 x 1024 (256, 128, 64) 13.0 / 10.3 / 12.4; 64 of 3 x 1032 x 264 (1088, 576, 320) 17.1 /
    // 12.2 / 13.6, x 512 x 2048 (512, 256, 128) 35.5 / 27.9 / 27.9.
    const long long likely = a.offsets && a.R / a.G < 128 ? (a.G < a.R ? a.G : a.R) : row_tiles(128);
    auto about = [&](int out_n) { return likely * ((a.N + out_n - 1) / out_n); };
    Split how{64, 1};
    if (!pair) {
        if (about(DUAL ? 64 : 128) <= sms) {
            bn = 128;
            how = split_of(tiles, !DUAL, a.pairs * ((a.K + kStep - 1) / kStep), sms);
        }
        if (!DUAL && (how.ways > 1 || about(64) <= sms)) bn = how.bn;
    }
    Maps maps{};
    bool ok = true;
    for (int i = 0; i < g.pairs; ++i) {
        ok = ok && map_2d(&maps.a32[i], g.a[i], a.K, a.R, 32);
        maps.a[i] = maps.a32[i];
        if (a.R > 96) ok = ok && map_2d(&maps.a[i], g.a[i], a.K, a.R, 128);
    }
    for (int i = 0; i < (DUAL ? 2 : g.pairs); ++i) {
        if (KIND == kNN) {
            ok = ok && map_mn(&maps.w[i], g.w[i], a.N, a.K, a.G, kStep, pair ? 2 : bn / 64, &a.blocks_w);
        } else {
            ok = ok && map_2d(&maps.w[i], g.w[i], a.K, (uint64_t)a.G * a.N, pair ? 128 : DUAL ? bn / 2 : bn);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    if (pair) return launch_plan<KIND, DUAL, 256, true>(a, maps, sms / 2 * 2, st);
    const long long n = tiles(DUAL ? bn / 2 : bn);
    const int ctas = (int)(n < sms ? n : sms);
    if (how.ways > 1 || bn == (DUAL ? 128 : 64)) return launch_narrow<KIND, DUAL>(a, maps, n, how, sms, st);
    if constexpr (!DUAL)
        if (bn == 128) return launch_plan<KIND, DUAL, 128, false>(a, maps, ctas, st);
    return launch_plan<KIND, DUAL, 256, false>(a, maps, ctas, st);
}

}  // namespace

cudaError_t launch_gemm(const GemmArgs &g, cudaStream_t st)
{
    // Few rows without tiles (bf16_vec.cu): up to 8 of one group; of groups, up to a number of outputs that grows with K, since a
    // tile's steps follow each other.  us, tiles / without: 1 to 8 x 4096 x 2048 9.9 / 4.9 to 5.1, x 8192 x 4096 17.1 / 13.2 to 14.3,
    // x 2048 x 512 4.0 / 2.6 to 2.9; 9 and 16 x 4096 x 2048 9.9 / 7.9, 8.3, x 8192 x 4096 17.0 / 22.1, 23.8.  Experts (257, hidden 2048,
    // inter 512), 1, 2, 4, 8 and 16 tokens: the gated pair 11.8 / 8.0, 14.9 / 13.8, 25.7 / 25.1, 42.9 / 42.1, 69.6 / 71.9 (73,728
    // outputs at 8 tokens), the down products 6.8 / 5.4, 9.4 / 9.6 (18,432 and 36,864).
    const long long outputs = (long long)g.R * g.N * (g.glu ? 2 : 1), most = g.K < 512 ? 20480 : g.K < 2048 ? 40ll * g.K : 81920;
    if (!g.w_kn && (g.offsets ? outputs <= most : g.R <= 8)) return launch_gemm_vec(g, st);
    if (g.glu) return launch_rows_product<kNT, true>(g, st);
    return g.w_kn ? launch_rows_product<kNN, false>(g, st) : launch_rows_product<kNT, false>(g, st);
}

cudaError_t launch_wgrad(const WgradArgs &g, cudaStream_t st)
{
    ProductArgs a{};
    a.offsets = g.offsets;
    a.y = g.dw;
    a.status = g.status;
    a.R = g.R;
    a.M = g.N;
    a.N = g.K;
    a.G = g.G;
    a.y_f32 = g.f32;
    a.accumulate = g.accumulate;
    a.wait_limit = g.wait_limit;
    const int sms = device_sm_count();
    auto tiles = [&](int rows, int cols) { return (long long)a.G * ((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols); };
    // A pair of CTAs a tile from 384 rows a group on, where there is a tile for every pair.  us, one CTA / a pair, 2048 x 512: 64 groups of 256
    // rows 43 / 54, of 384 56 / 56, of 512 69 / 61, of 1024 111 / 102, 16 of 4096 106 / 101; 4096 x 4096 from 512 rows 18.0 / 16.4, from
    // 4096 91 / 86.
    const bool pair = a.R / a.G >= 384 && tiles(256, 256) >= sms / 2;
    int bn = 256;
    Split how{64, 1};
    if (!pair) {
        if (tiles(128, 128) <= sms) {
            bn = 128;
            how = split_of([&](int cols) { return tiles(128, cols); }, true, (a.R / a.G + kStep - 1) / kStep, sms);
        }
        if (how.ways > 1 || tiles(128, 64) <= sms) bn = how.bn;
    }
    Maps maps{};
    // (the 128-column plans spill 12 to 32 bytes of an epilogue warp's registers, the 256-column one 8)
    const int blocks = pair ? 2 : bn / 64;
    if (!map_mn(&maps.a[0], g.dy, a.M, a.R, 1, kStep, 2, &a.blocks_a) || !map_mn(&maps.a16, g.dy, a.M, a.R, 1, 16, 2, &a.blocks_a) ||
        !map_mn(&maps.w[0], g.x, a.N, a.R, 1, kStep, blocks, &a.blocks_w) || !map_mn(&maps.w16, g.x, a.N, a.R, 1, 16, blocks, &a.blocks_w))
        return cudaErrorInvalidValue;
    const long long n = tiles(128, bn);
    const int ctas = (int)(n < sms ? n : sms);
    if (g.db) {
        // first, so that the products find dy in L2
        const long long blocks = (long long)g.G * ((g.N + 255) / 256);
        const int parts = blocks * 8 <= 2 * sms && g.R / g.G >= 256 ? 8 : 1;
        const BiasArgs b{g.dy, g.offsets, g.db, g.status, g.R, g.N, g.G, g.f32, g.accumulate, parts};
        const cudaError_t e = launch_dependent_clusters(column_sum_kernel, (unsigned)(blocks * parts), parts, 32 * kSumWarps, 0, st, b);
        if (e != cudaSuccess) return e;
    }
    if (pair) return launch_plan<kTN, false, 256, true>(a, maps, sms / 2 * 2, st);
    if (how.ways > 1 || bn == 64) return launch_narrow<kTN, false>(a, maps, n, how, sms, st);
    if (bn == 128) return launch_plan<kTN, false, 128, false>(a, maps, ctas, st);
    return launch_plan<kTN, false, 256, false>(a, maps, ctas, st);
}

}  // namespace qmoe
