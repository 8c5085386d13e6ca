// What the kernels of the gated feed-forward product share: the activations
// and how a product is described.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace olc {
namespace gated {

// ---- activations ------------------------------------------------------------

// act(g) and act'(g).  EXACT: float32 functions of full accuracy (FLOAT
// tensors); otherwise the fast forms, for results that are rounded to 16 bits:
// sigmoid is good to about 2^-21 of itself, GELU's distribution function to
// 2^-18 of itself down to g = -5 and 2^-17 where it ends (the products multiply
// its tail by any u, so an absolute bound would not do).
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float g) {
    if constexpr (EXACT) return 1.0f / (1.0f + expf(-g));
    return __fdividef(1.0f, 1.0f + __expf(-g));
}
// The normal distribution function Phi(g) and e^(-g^2 / 2).  On the negative side
// Phi(g) = erfc(x) / 2, x = |g| / sqrt 2, with erfc(x) = e^(-x^2) t P(t) for t =
// 1 / (1 + 3 x / 8) in (0, 1]: the P of degree 6 whose largest relative error is
// least (2^-20.6 for x <= 9.6, a linear program over 2400 points); the rounding
// of x^2 in the exponent is the larger part beyond.
__device__ __forceinline__ float normal_cdf_fast(float g, float& bell) {
    const float t = __fdividef(1.0f, fmaf(0.26516504f, fabsf(g), 1.0f));
    float q = fmaf(-0.13513307f, t, 0.38809144f);
    q = fmaf(q, t, -0.12984459f);
    q = fmaf(q, t, 0.28325987f);
    q = fmaf(q, t, 0.16658108f);
    q = fmaf(q, t, 0.21570666f);
    q = fmaf(q, t, 0.21133803f);
    bell = __expf(-0.5f * g * g);
    const float tail = 0.5f * (q * t) * bell;
    return g >= 0.f ? 1.0f - tail : tail;                // NaN takes the second arm
}
template <bool EXACT, int ACT>
__device__ __forceinline__ float gate_value(float g) {
    if constexpr (ACT == OLC_GATE_SILU) return g * sigmoid<EXACT>(g);
    else if constexpr (ACT == OLC_GATE_GELU) {
        if constexpr (EXACT) return 0.5f * g * erfcf(g * -0.70710678118654752f);
        float bell;
        return g * normal_cdf_fast(g, bell);
    }
    else if constexpr (ACT == OLC_GATE_RELU) return g < 0.f ? 0.f : g;
    else return sigmoid<EXACT>(g);
}
template <bool EXACT, int ACT>
__device__ __forceinline__ void gate_slope(float g, float& value, float& slope) {
    if constexpr (ACT == OLC_GATE_SILU) {
        const float s = sigmoid<EXACT>(g);
        value = g * s;
        slope = s * (1.0f + g * (1.0f - s));
    } else if constexpr (ACT == OLC_GATE_GELU) {
        // Phi(g) + g phi(g)
        float cdf, bell;
        if constexpr (EXACT) {
            cdf = 0.5f * erfcf(g * -0.70710678118654752f);
            bell = expf(-0.5f * g * g);
        } else {
            cdf = normal_cdf_fast(g, bell);
        }
        value = g * cdf;
        slope = fmaf(g, 0.39894228040143268f * bell, cdf);
    } else if constexpr (ACT == OLC_GATE_RELU) {
        value = g < 0.f ? 0.f : g;
        slope = g > 0.f ? 1.f : 0.f;
    } else {
        // s(|g|) = 1 / (1 + e) with e = e^-|g| leaves 1 - s = e s, which 1 - s itself would cancel
        const float e = EXACT ? expf(-fabsf(g)) : __expf(-fabsf(g));
        const float s = EXACT ? 1.0f / (1.0f + e) : __fdividef(1.0f, 1.0f + e);
        value = g < 0.f ? e * s : s;
        slope = e * s * s;
    }
}
// f(the activation as a constant): one branch around a whole
// run of elements instead of one at each
template <typename F>
__device__ __forceinline__ void by_activation(int act, F&& f) {
    switch (act) {
        case OLC_GATE_SILU: f(std::integral_constant<int, OLC_GATE_SILU>{}); break;
        case OLC_GATE_GELU: f(std::integral_constant<int, OLC_GATE_GELU>{}); break;
        case OLC_GATE_RELU: f(std::integral_constant<int, OLC_GATE_RELU>{}); break;
        default: f(std::integral_constant<int, OLC_GATE_SIGMOID>{});
    }
}

// ---- products -------------------------------------------------------------------

enum Mode { FWD = 0, DX = 1, DW = 2 };

// A stored matrix (16-bit elements that the TMA reads: base on a 16-byte
// boundary, pitch a multiple of 8).
struct Stored {
    const void* base;
    int64_t rows, cols, pitch;
};

struct Product {
    int mode;
    int64_t M, N, K;
    Stored a[2], b[2];
    bool a_mn, b_k;
    void* Y[3];
    int act;
};

// few rows, FWD operands: gated_few.cu.  Up to 32 rows, and up to 64 where the
// single CTAs' 64-column tiles would take more than a round (BF16, us, few-row
// kernel and tiles: 32 rows [1024] x [1024, 2816] 7.6 and 8.5, [4096] x [4096,
// 14336] 40.0 and 47.3; 64 rows 10.1 and 8.4, 43.0 and 47.5; 64 rows [2048] x
// [2048, 5632] 17.3 and 14.2).
inline bool takes_few(int64_t M, int64_t F, int sm_count) {
    return M <= 32 || (M <= 64 && ceil_div(F, 64) > sm_count);
}
cudaError_t launch_few(olc_dtype dt, const Product& w, int sm_count, cudaStream_t s);

// FLOAT: gated_float.cu; operands of any alignment to their elements.
// sums: float_sum_bytes of device memory; counters: float_counter_bytes
// of it, zero before the first call (and after every call).
size_t float_sum_bytes(int mode, int64_t M, int64_t N, int64_t K, int sm_count);
size_t float_counter_bytes(int sm_count);
cudaError_t launch_float(const Product& w, void* sums, unsigned int* counters, int sm_count, cudaStream_t s);

}  // namespace gated
}  // namespace olc
