// The 16-bit operators (bf16 rows and matrices, 32-bit sums) and their gradients: activation functions and the
// argument blocks of the kernels.  Launches and loads follow scaled.cuh: every kernel may start while its predecessor still
// writes, waits for it, and reads by plain loads.
#pragma once

#include "scaled.cuh"

namespace qmoe {

// ---------------------------------------------------------------- functions

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// 1 / (1 + exp(-v)) and v / (1 + exp(-v)): the fast exponential and division are off by a few 2^-22 for |v| < 20 and by at
// most |v| 2^-23 beyond (where the result is next to 0 or 1), far inside the 2^-9 of the bf16 that is written.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }
__device__ __forceinline__ float times_sigmoid(float v, float z) { return __fdividef(v, 1.0f + __expf(-z)); }

// tanh form of GELU: v (1 + tanh(u)) / 2 = v sigmoid(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3).
constexpr float kGelu2 = 1.5957691216057308f, kGelu3 = 0.044715f;      // 2 sqrt(2 / pi)
__device__ __forceinline__ float act_value(int act, float v)
{
    switch (act) {
    case MOE_ACT_SILU: return times_sigmoid(v, v);
    case MOE_ACT_GELU: return times_sigmoid(v, kGelu2 * (v + kGelu3 * v * v * v));
    case MOE_ACT_RELU: return v > 0.f ? v : (v != v ? v : 0.f);
    case MOE_ACT_SIGMOID: return sigmoid(v);
    default: return v;
    }
}
// The logistic function's value and slope, s and s (1 - s), from e = exp(-|v|): the smaller of s and 1 - s is e / (1 + e), where 1 - s
// would lose its digits to s (all of them past 17).
__device__ __forceinline__ float2 sigmoid_slope(float v)
{
    const float e = __expf(-fabsf(v)), r = __fdividef(1.0f, 1.0f + e), small = e * r;
    return make_float2(v < 0.f ? small : r, small * r);
}
// A function's value and derivative.
__device__ __forceinline__ float2 act_slope(int act, float v)
{
    switch (act) {
    case MOE_ACT_SILU: {
        const float s = sigmoid(v);
        return make_float2(v * s, s + v * s * (1.0f - s));
    }
    case MOE_ACT_GELU: {
        // past +-10 the slope is 1 or 0 to 30 digits, and v^2 would leave fp32's range; the value is v or 0 (1e-38 of 3e38 would not be)
        const float c = fminf(fmaxf(v, -10.0f), 10.0f), s = sigmoid(kGelu2 * (c + kGelu3 * c * c * c));
        return make_float2(v * (v < -10.0f ? 0.0f : s), v != v ? v : s + c * s * (1.0f - s) * (kGelu2 * (1.0f + 3.0f * kGelu3 * c * c)));
    }
    case MOE_ACT_RELU: {
        const float f = v <= 0.f ? 0.f : v;                  // (NaN stays, here and in the slope)
        return make_float2(f, f > 0.f ? 1.f : f);
    }
    case MOE_ACT_SIGMOID: return sigmoid_slope(v);
    default: return make_float2(v, 1.f);
    }
}

// ---------------------------------------------------------------- kernel arguments

// y = act(sum over the pairs of a w^T + bias) + residual; GLU: y = act(a w[0]^T + bias[0]) (a w[1]^T + bias[1]).
struct GemmArgs {
    const uint16_t *a[2], *w[2];         // [R, K]; [G, N, K], or [G, K, N] with w_kn
    const int32_t *offsets;              // [G] first row of each group (the last group ends at R), or null (G == 1)
    const uint16_t *bias[2];             // [G, N] or null
    const uint16_t *residual;            // [R, N] or null
    uint16_t *pre[2];                    // [R, N] or null: the products with their bias
    void *y;                             // [R, N] bf16 or fp32 (y_f32)
    int *status;
    int R, N, K, G, w_kn, pairs, glu, act, y_f32;
    long long wait_limit;
};
cudaError_t launch_gemm(const GemmArgs &a, cudaStream_t st);
cudaError_t launch_gemm_vec(const GemmArgs &a, cudaStream_t st);      // few rows, w [G, N, K] (bf16_vec.cu)

// dw_g (+)= dy_g^T x_g, db_g (+)= column sums of dy_g.
struct WgradArgs {
    const uint16_t *dy, *x;              // [R, N], [R, K]
    const int32_t *offsets;
    void *dw, *db;                       // [G, N, K], [G, N] (or null): bf16 or fp32 (f32)
    int *status;
    int R, N, K, G, f32, accumulate;
    long long wait_limit;
};
cudaError_t launch_wgrad(const WgradArgs &a, cudaStream_t st);

struct ActGradArgs {
    const uint16_t *dy, *pre, *up;
    uint16_t *dpre, *dup;
    size_t n;                            // elements, a multiple of 8
    int act;
};
cudaError_t launch_act_grad(const ActGradArgs &a, cudaStream_t st);

// Token rows and their expert-sorted copies.
struct RoutedArgs {
    const uint16_t *x;                   // dispatch: [T, n]; sum, sum_grad: rows [T k + T, n]
    const uint16_t *dy;                  // sum_grad: [T, n]
    const int32_t *inv_perm;
    const uint16_t *p, *w_shared;        // null: ones
    uint16_t *y;                         // dispatch: rows; sum: [T, n]; sum_grad: drows
    float *dp, *dw_shared;               // sum_grad, or null
    int *status;
    int T, n, k, has_shared;
};
cudaError_t launch_dispatch(const RoutedArgs &a, cudaStream_t st);
cudaError_t launch_weighted_sum(const RoutedArgs &a, cudaStream_t st);
cudaError_t launch_weighted_sum_grad(const RoutedArgs &a, cudaStream_t st);

// Norms around a block (bf16_norm.cu).
struct GatedNormArgs {
    const uint16_t *x, *residual, *gate, *post_weight, *pre_weight;
    uint16_t *sum, *y;                   // forward: written; backward: sum read
    const uint16_t *dy, *dsum;           // backward
    uint16_t *dx, *dresidual;
    void *dgate;
    float *dpost_weight, *dpre_weight;
    float *partial;                      // workspace: column sums of each block
    int *status;                         // backward
    int T, n, gate_shape, act, post_norm;
    float scale, weight_offset, eps;
};
constexpr int kNormMaxN = 8192;
size_t gated_norm_partials(int T, int n);    // floats of `partial`
cudaError_t launch_gated_norm(const GatedNormArgs &a, cudaStream_t st);
cudaError_t launch_gated_norm_grad(const GatedNormArgs &a, cudaStream_t st);

}  // namespace qmoe
