// C entry points of the 16-bit operators: argument checks and launches (contract: include/moe.h).
#include "bf16.cuh"

using namespace qmoe;

namespace {

constexpr long long kWaitPolls = 1ll << 20;   // bound of every wait inside a kernel, about a second
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxProductRows = 1 << 21;      // start rows share a word with their group in the kernels' table
constexpr int kMaxGroups = 1024;              // with N <= 2^20 a stack's rows stay 32-bit copy coordinates

bool aligned(const void *p, unsigned a = 16) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool aligned_or_null(const void *p, unsigned a = 16) { return p == nullptr || aligned(p, a); }
// Rows: there when there are any.
bool rows_ok(const void *p, int rows) { return rows == 0 ? aligned_or_null(p) : aligned(p); }
bool flag(int v) { return v == 0 || v == 1; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int check_ws(void *ws, size_t bytes)
{
    if (!aligned(ws)) return MOE_ERR_INVALID_ARG;
    return bytes < MOE_SCALED_WS_BYTES ? MOE_ERR_WORKSPACE : MOE_OK;
}

// Sizes of a product over R rows, N outputs, K inputs and G groups.
int check_product(int R, int N, int K, int G, const int32_t *offsets)
{
    if (R < 0 || N <= 0 || K <= 0 || G <= 0 || R > kMaxProductRows) return MOE_ERR_INVALID_ARG;
    if (!aligned_or_null(offsets, 4) || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
    if (G > kMaxGroups || N % 8 || K % 8 || K > 65536 || N > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_act(int act)
{
    if (act < MOE_ACT_NONE || act > MOE_ACT_SIGMOID) return MOE_ERR_INVALID_ARG;
    return act == MOE_ACT_SIGMOID ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows routed to k picks each.
int check_routed(int T, int n, int k, int has_shared, const int32_t *inv_perm)
{
    if (T < 0 || n <= 0 || k <= 0 || T > kMaxTokens || !flag(has_shared)) return MOE_ERR_INVALID_ARG;
    if (k > kMaxTopK || n % 8 || n > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return T ? (aligned(inv_perm, 4) ? MOE_OK : MOE_ERR_INVALID_ARG) : (aligned_or_null(inv_perm, 4) ? MOE_OK : MOE_ERR_INVALID_ARG);
}

int check_gated_norm(const uint16_t *x, const uint16_t *gate, int gate_shape, int gate_act, float scale, int post_norm,
                     const uint16_t *post_weight, const uint16_t *pre_weight, float eps, int T, int n)
{
    if (T < 0 || n <= 0 || T > kMaxRows || !(eps >= 0.f) || !flag(post_norm) || scale != scale) return MOE_ERR_INVALID_ARG;
    if (gate_shape < MOE_GATE_NONE || gate_shape > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
    if (gate_act != MOE_ACT_NONE && gate_act != MOE_ACT_SILU && gate_act != MOE_ACT_SIGMOID) return MOE_ERR_UNSUPPORTED;
    if (gate_shape == MOE_GATE_NONE && (gate != nullptr || gate_act != MOE_ACT_NONE)) return MOE_ERR_INVALID_ARG;
    if (n % 8 || n > kNormMaxN) return MOE_ERR_UNSUPPORTED;
    if (!rows_ok(x, T) || !aligned_or_null(post_weight) || !aligned_or_null(pre_weight) || (post_weight && !post_norm))
        return MOE_ERR_INVALID_ARG;
    if (gate_shape != MOE_GATE_NONE && !rows_ok(gate, gate_shape == MOE_GATE_CHANNEL ? n : T)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_gemm(const uint16_t *a, const uint16_t *w, const uint16_t *a2, const uint16_t *w2, int w_transposed, int R, int N, int K,
             int G, const int32_t *offsets, const uint16_t *bias, int act, const uint16_t *residual, uint16_t *pre_out, void *y,
             int y_f32, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_product(R, N, K, G, offsets);
    if (rc || (rc = check_act(act))) return rc;
    if (!rows_ok(a, R) || !aligned(w) || !aligned_or_null(a2) || !aligned_or_null(w2) || !flag(w_transposed) || !flag(y_f32) ||
        !aligned_or_null(bias) || !aligned_or_null(residual) || !aligned_or_null(pre_out) || !rows_ok(y, R))
        return MOE_ERR_INVALID_ARG;
    if (w2 ? !rows_ok(a2, R) : a2 != nullptr) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (R == 0) return MOE_OK;
    GemmArgs g{};
    g.a[0] = a;
    g.a[1] = a2;
    g.w[0] = w;
    g.w[1] = w2;
    g.pairs = w2 ? 2 : 1;
    g.w_kn = w_transposed;
    g.offsets = offsets;
    g.bias[0] = bias;
    g.residual = residual;
    g.pre[0] = pre_out;
    g.y = y;
    g.y_f32 = y_f32;
    g.act = act;
    g.status = static_cast<int *>(ws);
    g.R = R;
    g.N = N;
    g.K = K;
    g.G = G;
    g.wait_limit = kWaitPolls;
    return cuda_rc(launch_gemm(g, static_cast<cudaStream_t>(stream)));
}

int moe_gemm_glu(const uint16_t *a, const uint16_t *gate, const uint16_t *up, const uint16_t *gate_bias, const uint16_t *up_bias,
                 int act, int R, int inter, int K, int G, const int32_t *offsets, uint16_t *gate_out, uint16_t *up_out,
                 uint16_t *h, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_product(R, inter, K, G, offsets);
    if (rc || (rc = check_act(act))) return rc;
    if (!rows_ok(a, R) || !aligned(gate) || !aligned(up) || !aligned_or_null(gate_bias) || !aligned_or_null(up_bias) ||
        !aligned_or_null(gate_out) || !aligned_or_null(up_out) || !rows_ok(h, R))
        return MOE_ERR_INVALID_ARG;
    if ((gate_out == nullptr) != (up_out == nullptr)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (R == 0) return MOE_OK;
    GemmArgs g{};
    g.a[0] = g.a[1] = a;
    g.w[0] = gate;
    g.w[1] = up;
    g.pairs = 1;
    g.glu = 1;
    g.offsets = offsets;
    g.bias[0] = gate_bias;
    g.bias[1] = up_bias;
    g.pre[0] = gate_out;
    g.pre[1] = up_out;
    g.y = h;
    g.act = act;
    g.status = static_cast<int *>(ws);
    g.R = R;
    g.N = inter;
    g.K = K;
    g.G = G;
    g.wait_limit = kWaitPolls;
    return cuda_rc(launch_gemm(g, static_cast<cudaStream_t>(stream)));
}

int moe_gemm_wgrad(const uint16_t *dy, const uint16_t *x, int R, int N, int K, int G, const int32_t *offsets, int accumulate,
                   void *dw, void *db, int f32, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_product(R, N, K, G, offsets);
    if (rc) return rc;
    if (!rows_ok(dy, R) || !rows_ok(x, R) || !aligned(dw) || !aligned_or_null(db) || !flag(f32) || !flag(accumulate))
        return MOE_ERR_INVALID_ARG;
    if (accumulate && !f32) return MOE_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits (a stack this large fits no GPU's memory unless N or K is a few elements)
    if ((long long)G * ((N + 63) / 64) * ((K + 63) / 64) > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0) {
        if (accumulate) return MOE_OK;
        const size_t size = f32 ? 4 : 2;
        cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)G * N * K * size, st);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)G * N * size, st);
        return cuda_rc(e);
    }
    WgradArgs g{};
    g.dy = dy;
    g.x = x;
    g.offsets = offsets;
    g.dw = dw;
    g.db = db;
    g.f32 = f32;
    g.accumulate = accumulate;
    g.status = static_cast<int *>(ws);
    g.R = R;
    g.N = N;
    g.K = K;
    g.G = G;
    g.wait_limit = kWaitPolls;
    return cuda_rc(launch_wgrad(g, st));
}

int moe_act_grad(int act, const uint16_t *dy, const uint16_t *pre, const uint16_t *up, int R, int N, uint16_t *dpre, uint16_t *dup,
                 void *stream)
{
    if (R < 0 || N <= 0 || R > kMaxRows) return MOE_ERR_INVALID_ARG;
    const int rc = check_act(act);
    if (rc) return rc;
    if (N % 8 || N > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (!rows_ok(dy, R) || !rows_ok(pre, R) || !aligned_or_null(up) || !rows_ok(dpre, R) || !aligned_or_null(dup)) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if ((up == nullptr) != (dup == nullptr) || dup == dpre) return MOE_ERR_INVALID_ARG;
    ActGradArgs g{dy, pre, up, dpre, dup, (size_t)R * N, act};
    return cuda_rc(launch_act_grad(g, static_cast<cudaStream_t>(stream)));
}

int moe_dispatch(const uint16_t *x, int T, int n, int k, int has_shared, const int32_t *inv_perm, uint16_t *y, void *ws,
                 size_t ws_bytes, void *stream)
{
    int rc = check_routed(T, n, k, has_shared, inv_perm);
    if (rc) return rc;
    if (!rows_ok(x, T) || !rows_ok(y, T)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (T == 0) return MOE_OK;
    RoutedArgs g{};
    g.x = x;
    g.inv_perm = inv_perm;
    g.y = y;
    g.status = static_cast<int *>(ws);
    g.T = T;
    g.n = n;
    g.k = k;
    g.has_shared = has_shared;
    return cuda_rc(launch_dispatch(g, static_cast<cudaStream_t>(stream)));
}

int moe_weighted_sum(const uint16_t *rows, int T, int n, int k, int has_shared, const int32_t *inv_perm, const uint16_t *p,
                     const uint16_t *w_shared, uint16_t *y, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_routed(T, n, k, has_shared, inv_perm);
    if (rc) return rc;
    if (!rows_ok(rows, T) || !rows_ok(y, T) || !aligned_or_null(p) || !aligned_or_null(w_shared)) return MOE_ERR_INVALID_ARG;
    if (T && (w_shared != nullptr) != (has_shared && p)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (T == 0) return MOE_OK;
    RoutedArgs g{};
    g.x = rows;
    g.inv_perm = inv_perm;
    g.p = p;
    g.w_shared = w_shared;
    g.y = y;
    g.status = static_cast<int *>(ws);
    g.T = T;
    g.n = n;
    g.k = k;
    g.has_shared = has_shared;
    return cuda_rc(launch_weighted_sum(g, static_cast<cudaStream_t>(stream)));
}

int moe_weighted_sum_grad(const uint16_t *dy, const uint16_t *rows, int T, int n, int k, int has_shared, const int32_t *inv_perm,
                          const uint16_t *p, const uint16_t *w_shared, uint16_t *drows, float *dp, float *dw_shared, void *ws,
                          size_t ws_bytes, void *stream)
{
    int rc = check_routed(T, n, k, has_shared, inv_perm);
    if (rc) return rc;
    if (!rows_ok(dy, T) || !aligned_or_null(rows) || !rows_ok(p, T) || !aligned_or_null(w_shared) || !rows_ok(drows, T) ||
        !aligned_or_null(dp) || !aligned_or_null(dw_shared))
        return MOE_ERR_INVALID_ARG;
    if (T && ((w_shared != nullptr) != (has_shared != 0) || ((dp || dw_shared) && !rows))) return MOE_ERR_INVALID_ARG;
    if (dw_shared && !has_shared) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (T == 0) return MOE_OK;
    RoutedArgs g{};
    g.x = rows;
    g.dy = dy;
    g.inv_perm = inv_perm;
    g.p = p;
    g.w_shared = w_shared;
    g.y = drows;
    g.dp = dp;
    g.dw_shared = dw_shared;
    g.status = static_cast<int *>(ws);
    g.T = T;
    g.n = n;
    g.k = k;
    g.has_shared = has_shared;
    return cuda_rc(launch_weighted_sum_grad(g, static_cast<cudaStream_t>(stream)));
}

int moe_gated_norm(const uint16_t *x, const uint16_t *residual, const uint16_t *gate, int gate_shape, int gate_act, float scale,
                   int post_norm, const uint16_t *post_weight, const uint16_t *pre_weight, float weight_offset, float eps, int T,
                   int n, uint16_t *sum_out, uint16_t *y_out, void *stream)
{
    const int rc = check_gated_norm(x, gate, gate_shape, gate_act, scale, post_norm, post_weight, pre_weight, eps, T, n);
    if (rc) return rc;
    if (!aligned_or_null(residual) || !aligned_or_null(sum_out) || !aligned_or_null(y_out)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    GatedNormArgs a{};
    a.x = x;
    a.residual = residual;
    a.gate = gate;
    a.post_weight = post_weight;
    a.pre_weight = pre_weight;
    a.sum = sum_out;
    a.y = y_out;
    a.T = T;
    a.n = n;
    a.gate_shape = gate_shape;
    a.act = gate_act;
    a.post_norm = post_norm;
    a.scale = scale;
    a.weight_offset = weight_offset;
    a.eps = eps;
    return cuda_rc(launch_gated_norm(a, static_cast<cudaStream_t>(stream)));
}

int moe_gated_norm_workspace_size(int T, int n, size_t *bytes)
{
    if (T < 0 || n <= 0 || T > kMaxRows || !bytes) return MOE_ERR_INVALID_ARG;
    if (n % 8 || n > kNormMaxN) return MOE_ERR_UNSUPPORTED;
    *bytes = MOE_SCALED_WS_BYTES + gated_norm_partials(T, n) * sizeof(float);
    return MOE_OK;
}

int moe_gated_norm_grad(const uint16_t *x, const uint16_t *sum, const uint16_t *gate, int gate_shape, int gate_act, float scale,
                        int post_norm, const uint16_t *post_weight, const uint16_t *pre_weight, float weight_offset, float eps,
                        int T, int n, const uint16_t *dy, const uint16_t *dsum, uint16_t *dx, uint16_t *dresidual, void *dgate,
                        float *dpost_weight, float *dpre_weight, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_gated_norm(x, gate, gate_shape, gate_act, scale, post_norm, post_weight, pre_weight, eps, T, n);
    if (rc) return rc;
    if (!rows_ok(sum, T) || !aligned_or_null(dy) || !aligned_or_null(dsum) || !rows_ok(dx, T) || !aligned_or_null(dresidual) ||
        !aligned_or_null(dgate) || !aligned_or_null(dpost_weight) || !aligned_or_null(dpre_weight))
        return MOE_ERR_INVALID_ARG;
    if ((dgate && gate_shape == MOE_GATE_NONE) || (dpost_weight && !post_norm)) return MOE_ERR_INVALID_ARG;
    if (T && ((!dy && !dsum) || (dpre_weight && !dy) || dresidual == dx)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes))) return rc;
    if (ws_bytes < MOE_SCALED_WS_BYTES + gated_norm_partials(T, n) * sizeof(float)) return MOE_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        float *const sums[3] = {dpost_weight, dpre_weight, gate_shape == MOE_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr};
        for (float *s : sums)
            if (s && e == cudaSuccess) e = cudaMemsetAsync(s, 0, (size_t)n * sizeof(float), st);
        return cuda_rc(e);
    }
    GatedNormArgs a{};
    a.x = x;
    a.gate = gate;
    a.post_weight = post_weight;
    a.pre_weight = pre_weight;
    a.sum = const_cast<uint16_t *>(sum);
    a.dy = dy;
    a.dsum = dsum;
    a.dx = dx;
    a.dresidual = dresidual;
    a.dgate = dgate;
    a.dpost_weight = dpost_weight;
    a.dpre_weight = dpre_weight;
    a.status = static_cast<int *>(ws);
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + MOE_SCALED_WS_BYTES);
    a.T = T;
    a.n = n;
    a.gate_shape = gate_shape;
    a.act = gate_act;
    a.post_norm = post_norm;
    a.scale = scale;
    a.weight_offset = weight_offset;
    a.eps = eps;
    return cuda_rc(launch_gated_norm_grad(a, st));
}

}  // extern "C"
