// C entry points of the block-scaled operators: argument checks and launches (contract: include/moe.h).
#include "scaled.cuh"

using namespace qmoe;

namespace {

constexpr long long kWaitPolls = 1ll << 20;   // bound of every wait inside a kernel, about a second
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxProductRows = 1 << 21;      // start rows share a word with their group in the kernels' table
constexpr int kMaxGroups = 1024;              // with N <= 2^20 a stack's rows stay 32-bit copy coordinates
constexpr int kMaxRowLength = 16384;          // rows that a kernel keeps in registers whole

bool aligned(const void *p, unsigned a = 16) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool aligned_or_null(const void *p, unsigned a = 16) { return p == nullptr || aligned(p, a); }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool activation_format(int f) { return f == MOE_SCALED_NVFP4 || f == MOE_SCALED_MXFP8; }
bool known_format(int f) { return activation_format(f) || f == MOE_SCALED_MXFP4; }

// Destination or source rows: NVFP4 rows may carry factors, the power-of-two formats never do.
bool rows_ok(const moe_scaled_rows *q, int fmt)
{
    if (!q || !aligned(q->codes) || !aligned(q->scales)) return false;
    return fmt == MOE_SCALED_NVFP4 ? aligned_or_null(q->row_scale) : q->row_scale == nullptr;
}

bool mat_ok(const moe_scaled_mat *w, int fmt)
{
    return w && aligned(w->codes, fmt == MOE_SCALED_MXFP8 ? 32 : 16) && aligned(w->scales) && aligned_or_null(w->alpha, 4);
}

int check_ws(void *ws, size_t bytes)
{
    if (!aligned(ws)) return MOE_ERR_INVALID_ARG;
    return bytes < MOE_SCALED_WS_BYTES ? MOE_ERR_WORKSPACE : MOE_OK;
}

// Sizes of a product over R rows, N outputs, K inputs and G groups.
int check_product(int fmt, int R, int N, int K, int G, const int32_t *offsets, int n_unit)
{
    if (R < 0 || N <= 0 || K <= 0 || G <= 0 || R > kMaxProductRows) return MOE_ERR_INVALID_ARG;
    if (!aligned_or_null(offsets, 4) || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
    if (!activation_format(fmt) || G > kMaxGroups) return MOE_ERR_UNSUPPORTED;
    if (K % (fmt == MOE_SCALED_NVFP4 ? 64 : 128) || K > 65536 || N % n_unit || N > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_add_rmsnorm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float weight_offset, float eps,
                    int T, int n, uint16_t *sum_out, uint16_t *y_out, int format, const moe_scaled_rows *q, void *stream)
{
    if (T < 0 || n <= 0 || T > kMaxRows || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if (format != 0 && !activation_format(format)) return MOE_ERR_UNSUPPORTED;
    if (n > kMaxRowLength || n % (format ? scaled_block(format) : 8)) return MOE_ERR_UNSUPPORTED;
    if (!aligned(x) || !aligned_or_null(residual) || !aligned_or_null(weight) || !aligned_or_null(sum_out) ||
        !aligned_or_null(y_out))
        return MOE_ERR_INVALID_ARG;
    if (format ? !rows_ok(q, format) || (format == MOE_SCALED_NVFP4 && !q->row_scale) : q != nullptr) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    RowArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.weight_offset = weight_offset;
    a.eps = eps;
    a.sum_out = sum_out;
    a.y_out = y_out;
    if (q) {
        a.codes = q->codes;
        a.scales = q->scales;
        a.row_scale = q->row_scale;
    }
    a.T = T;
    a.n = n;
    return cuda_rc(launch_rows(a, format, true, static_cast<cudaStream_t>(stream)));
}

int moe_quantize(int format, const void *x, int x_f32, int T, int n, int groups, const float *gscale,
                 const moe_scaled_rows *q, void *stream)
{
    if (T < 0 || n <= 0 || groups <= 0 || T > kMaxRows || (x_f32 != 0 && x_f32 != 1) || T % groups) return MOE_ERR_INVALID_ARG;
    if (!known_format(format)) return MOE_ERR_UNSUPPORTED;
    if (n % scaled_block(format) || n > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (format == MOE_SCALED_NVFP4 && !gscale && n > kMaxRowLength) return MOE_ERR_UNSUPPORTED;
    if (!aligned(x) || !rows_ok(q, format) || !aligned_or_null(gscale, 4)) return MOE_ERR_INVALID_ARG;
    if (format == MOE_SCALED_NVFP4 ? (gscale == nullptr) == (q->row_scale == nullptr) : gscale != nullptr)
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    RowArgs a{};
    a.x = x;
    a.x_f32 = x_f32;
    a.codes = q->codes;
    a.scales = q->scales;
    a.row_scale = q->row_scale;
    a.gscale = gscale;
    a.T = T;
    a.n = n;
    a.rows_per_group = groups > 1 ? T / groups : 0;
    return cuda_rc(launch_rows(a, format, false, static_cast<cudaStream_t>(stream)));
}

int moe_quantize_routed(int format, const uint16_t *x, int T, int n, int k, int E, int has_shared, const int32_t *ids,
                        const int32_t *inv_perm, const int32_t *offsets, const moe_scaled_rows *q, void *ws,
                        size_t ws_bytes, void *stream)
{
    if (T < 0 || n <= 0 || k <= 0 || E <= 0 || T > kMaxTokens || (has_shared != 0 && has_shared != 1)) return MOE_ERR_INVALID_ARG;
    if (!activation_format(format) || k > kMaxTopK || E + has_shared > kMaxGroups) return MOE_ERR_UNSUPPORTED;
    if (n % scaled_block(format) || n > (format == MOE_SCALED_NVFP4 ? kMaxRowLength : 1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (!aligned(x) || !aligned(ids, 4) || !aligned(inv_perm, 4) || !aligned(offsets, 4) || !rows_ok(q, format))
        return MOE_ERR_INVALID_ARG;
    if (format == MOE_SCALED_NVFP4 && !q->row_scale) return MOE_ERR_INVALID_ARG;
    const int rc = check_ws(ws, ws_bytes);
    if (rc) return rc;
    if (T == 0) return MOE_OK;
    RowArgs a{};
    a.x = x;
    a.codes = q->codes;
    a.scales = q->scales;
    a.row_scale = q->row_scale;
    a.ids = ids;
    a.inv_perm = inv_perm;
    a.offsets = offsets;
    a.status = static_cast<int *>(ws);
    a.T = T;
    a.n = n;
    a.k = k;
    a.E = E;
    a.has_shared = has_shared;
    return cuda_rc(launch_rows(a, format, false, static_cast<cudaStream_t>(stream)));
}

int moe_tile_scales(int format, const uint8_t *src, int G, int N, int n, uint8_t *dst, void *stream)
{
    if (G < 0 || N <= 0 || n <= 0) return MOE_ERR_INVALID_ARG;
    if (!known_format(format)) return MOE_ERR_UNSUPPORTED;
    if (n % scaled_block(format) || n > (1 << 20) || (long long)G * N > 0x7FFFFFFFll - 256) return MOE_ERR_UNSUPPORTED;
    if (src == nullptr || !aligned(dst)) return MOE_ERR_INVALID_ARG;
    if (G == 0) return MOE_OK;
    return cuda_rc(launch_tile_scales(src, dst, format, G, N, n, static_cast<cudaStream_t>(stream)));
}

int moe_scaled_gemm(int format, const moe_scaled_rows *a, const moe_scaled_mat *w, int R, int N, int K, int G,
                    const int32_t *offsets, void *y, int y_f32, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_product(format, R, N, K, G, offsets, 8);
    if (rc) return rc;
    if (!rows_ok(a, format) || !mat_ok(w, format) || !aligned(y) || (y_f32 != 0 && y_f32 != 1)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (R == 0) return MOE_OK;
    ScaledGemmArgs g{};
    g.a_codes = a->codes;
    g.a_scales = a->scales;
    g.a_row_scale = a->row_scale;
    g.w_codes[0] = w->codes;
    g.w_scales[0] = w->scales;
    g.alpha[0] = w->alpha;
    g.offsets = offsets;
    g.y = y;
    g.y_f32 = y_f32;
    g.status = static_cast<int *>(ws);
    g.R = R;
    g.N = N;
    g.K = K;
    g.G = G;
    g.wait_limit = kWaitPolls;
    return cuda_rc(launch_scaled_gemm(g, format, false, static_cast<cudaStream_t>(stream)));
}

int moe_scaled_swiglu(int format, const moe_scaled_rows *a, const moe_scaled_mat *gate, const moe_scaled_mat *up, int R,
                      int inter, int K, int G, const int32_t *offsets, const float *h_scale, const moe_scaled_rows *h,
                      void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_product(format, R, inter, K, G, offsets, format == MOE_SCALED_NVFP4 ? 64 : 128);
    if (rc) return rc;
    if (!rows_ok(a, format) || !mat_ok(gate, format) || !mat_ok(up, format) || !rows_ok(h, format) || h->row_scale)
        return MOE_ERR_INVALID_ARG;
    if (format == MOE_SCALED_NVFP4 ? !aligned(h_scale, 4) : h_scale != nullptr) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (R == 0) return MOE_OK;
    ScaledGemmArgs g{};
    g.a_codes = a->codes;
    g.a_scales = a->scales;
    g.a_row_scale = a->row_scale;
    const moe_scaled_mat *w[2] = {gate, up};
    for (int i = 0; i < 2; ++i) {
        g.w_codes[i] = w[i]->codes;
        g.w_scales[i] = w[i]->scales;
        g.alpha[i] = w[i]->alpha;
    }
    g.offsets = offsets;
    g.h_codes = h->codes;
    g.h_scales = h->scales;
    g.h_gscale = h_scale;
    g.status = static_cast<int *>(ws);
    g.R = R;
    g.N = inter;
    g.K = K;
    g.G = G;
    g.wait_limit = kWaitPolls;
    return cuda_rc(launch_scaled_gemm(g, format, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
