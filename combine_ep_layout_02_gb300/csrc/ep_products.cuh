// ep_products.cuh -- what the BF16 products of an expert layer share: their
// arguments, the activations and their derivatives, and the launchers.
#pragma once

#include "ep_experts.cuh"

namespace ep {

// The three products of rows [rows, K] or [rows, N] with weights [E, N, K]:
//   kForward  out[r, n] = sum_k x[r, k] w[e, n, k]
//   kInput    dx[r, k]  = sum_n dy[r, n] w[e, n, k]
//   kWeight   dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]
enum ProductKind { kForward = 0, kInput = 1, kWeight = 2 };

struct ProductArgs {
    // operands: kForward x, w; kInput dy, w; kWeight dy, x
    const uint16_t* a;
    const uint16_t* b;
    int64_t rows;  // of the buffers
    int64_t N, K;  // rows and width of an expert's weights; with SwiGLU N counts gate and up rows
    int E;
    // segments; counts == nullptr: one expert with all rows
    const int32_t* counts;
    const int32_t* offsets;
    int kind, capacity;
    // epilogue
    int activation;       // kForward: EP_ACT_*; kInput: EP_ACT_SWIGLU gives dz from z
    const void* bias;     // [N] or nullptr
    int bias_type;
    const void* residual; // of out_type, or nullptr
    const void* add;      // kWeight: of out_type, or nullptr
    void* out;
    int out_type;
    uint16_t* z;          // kForward: pre-activations out or nullptr; kInput with SwiGLU: in
    uint32_t* status;
    // one expert: columns of a tile at most (0: 256); kForward: parts of the summed
    // index, each with its own fp32 [rows, N] in `out`; kWeight: rows of a part
    // (0: all), each of E parts with its own fp32 [N, K]
    int most, splits;
    int64_t part_rows;
};

// How a dense product of more than EP_LINEAR_FEW_TOKENS tokens is cut.
struct DensePlan {
    int most, splits;
};
DensePlan dense_plan(int64_t M, int64_t K, int64_t channels, bool gated, bool split);
// The same for the gradient of [N, K] weights from M rows.
DensePlan weight_plan(int64_t M, int64_t N, int64_t K, bool split);

// Rows of expert e (of the whole buffer where there are no experts).
__device__ __forceinline__ Segment product_segment(const ProductArgs& p, int e) {
    if (p.counts == nullptr) {
        if (p.part_rows == 0) return Segment{0, p.rows, false};
        const int64_t first = e * p.part_rows;
        return Segment{first, first + p.part_rows < p.rows ? p.part_rows : p.rows - first, false};
    }
    return expert_segment(e, p.counts, p.offsets, p.kind, p.capacity, p.rows);
}

// 1 / (1 + exp(-v)), the exponential and the quotient each good to 2 ulp; far
// below zero the divisor reaches 2^126, for which the quotient is 0, the limit.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, __fadd_rn(1.0f, expf(-v))); }

// Good to 1 and 2 ulp for arguments in the normal range.
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Tail of the normal distribution beyond a = |v|, from 1 to 15, and e = exp(-v^2 / 2),
// good to some 10 parts in 2^24.  With z = |v| / sqrt 2 the tail is erfc(z) / 2 =
// exp(-z^2) erfcx(z) / 2, and erfcx(z) / 2 = t p(t) for t = 1 / (1 + 0.4 z), p being
// smooth: a polynomial fitted to the relative error (7e-8) with z from 0.7 to 10.6.
// The exponent -v^2 / 2 log2(e) is taken with its rounding error, which the power
// of two would otherwise multiply; kNarrow: v is a bf16 value and its square
// exact.  From |v| = 15 on e is 0.  (With normcdff and a second exp the elementwise
// pass of 16,384 x 4,096 took 218 us.)
template <bool kNarrow>
__device__ __forceinline__ float normal_tail(float a, float& e) {
    const float t = rcp_approx(fmaf(a, 0.28284271247461901f, 1.0f));
    float p = 0.00450075557f;
    p = fmaf(p, t, -0.0721399933f);
    p = fmaf(p, t, 0.139903709f);
    p = fmaf(p, t, -0.00842234679f);
    p = fmaf(p, t, 0.111561485f);
    p = fmaf(p, t, 0.0982244909f);
    p = fmaf(p, t, 0.113490656f);
    p = fmaf(p, t, 0.112806149f);
    // -log2(e) / 2 = kHi + kLo
    constexpr float kHi = -0.72134752044448169f;
    constexpr float kLo = (float)(-0.72134752044448169 - (double)kHi);
    const float square = a * a;
    const float power = square * kHi;
    float rest = fmaf(square, kLo, fmaf(square, kHi, -power));
    if (!kNarrow) rest = fmaf(fmaf(a, a, -square), kHi, rest);
    e = exp2_approx(power);
    e = fmaf(e, rest * 0.69314718055994531f, e);
    return t * p * e;
}

// Normal distribution function; below |v| = 1, where 1/2 is the larger part, with
// an odd polynomial (7e-10).
__device__ __forceinline__ float normal_cdf(float v) {
    const float a = fminf(fabsf(v), 15.0f), square = a * a;
    float e;
    const float tail = normal_tail<false>(a, e);
    float near = -7.65419899e-06f;
    near = fmaf(near, square, 0.000113486348f);
    near = fmaf(near, square, -0.00118632992f);
    near = fmaf(near, square, 0.0099733234f);
    near = fmaf(near, square, -0.0664903599f);
    near = fmaf(near, square, 0.39894228f);
    return a < 1.0f ? fmaf(v, near, 0.5f) : v < 0.0f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;  // keeps NaN
        case EP_ACT_SILU: return v * sigmoid(v);
        case EP_ACT_GELU: return v * normal_cdf(v);
        default: return v;
    }
}

// Derivative of v Phi(v) times dy, both v and dy being bf16.  Below |v| = 1 it is
// dy v q(v^2) + dy / 2, where dy v and dy / 2 are exact and q is smooth (fitted to
// 6e-9): one rounding is left near v = 0, where most values lie.  At v = -0.752, where
// the two terms cancel, the rounding of q is what would be left, and is added.  (From
// the distribution function and v e: 116 us for 16,384 x 4,096, here 129; but 240 of
// 8.4 million gradients rounded to the other bf16 neighbour, here 65, none of them
// large, and the weights' gradient 2e-6 to 6e-6 off, here 6e-7.)
__device__ __forceinline__ float gelu_back(float v, float dy) {
    const float a = fminf(fabsf(v), 15.0f), square = a * a;
    float e;
    const float tail = normal_tail<true>(a, e);
    float r = 9.34694708e-06f;
    r = fmaf(r, square, -0.000117826632f);
    r = fmaf(r, square, 0.00116243132f);
    r = fmaf(r, square, -0.00950479601f);
    r = fmaf(r, square, 0.0598436482f);
    r = fmaf(r, square, -0.265961915f);
    constexpr float kFirst = 0.797884583f;
    const float q = fmaf(r, square, kFirst), left = fmaf(r, square, kFirst - q), both = dy * v;
    const float near = fmaf(both, left, fmaf(both, q, 0.5f * dy));
    const float far = dy * fmaf(v * 0.39894228040143268f, e, v < 0.0f ? tail : 1.0f - tail);
    return a < 1.0f && fabsf(dy) < INFINITY ? near : far;  // an infinite dy: no inf - inf
}

// d act / d v, times dy.  The tails are those of the functions: both factors of
// GELU's second term vanish far from zero.
__device__ __forceinline__ float activate_back(float v, float dy, int act) {
    switch (act) {
        case EP_ACT_RELU: return v > 0.0f ? dy : v == v ? 0.0f : v;
        case EP_ACT_SILU: {
            const float s = sigmoid(v);
            return dy * s * fmaf(v, 1.0f - s, 1.0f);
        }
        case EP_ACT_GELU: return gelu_back(v, dy);
        default: return dy;
    }
}

// Gradients of gate and up of h = silu(g) u.
__device__ __forceinline__ void swiglu_back(float g, float u, float dh, float& dg, float& du) {
    const float s = sigmoid(g);
    const float ds = dh * s;
    dg = ds * u * fmaf(g, 1.0f - s, 1.0f);
    du = ds * g;
}

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)pack_bf16x2_rn(v, 0.0f); }
__device__ __forceinline__ float load_typed(const void* p, int type, int64_t i) {
    return type == EP_TYPE_F32 ? __ldg(static_cast<const float*>(p) + i)
                               : bf16_value(__ldg(static_cast<const uint16_t*>(p) + i));
}

// ---- launchers (host) ------------------------------------------------------

cudaError_t launch_product(const ProductArgs& p, ProductKind kind, cudaStream_t stream);

// kForward of one expert for up to EP_LINEAR_FEW_TOKENS tokens
cudaError_t launch_linear_few(const ProductArgs& p, cudaStream_t stream);

// the epilogue over the parts' sums [splits, rows, N]
cudaError_t launch_linear_finish(const ProductArgs& p, const float* parts, int splits, cudaStream_t stream);

// add (or nothing) and the parts' sums [splits, count] to `out`
cudaError_t launch_weight_finish(const float* parts, int splits, int64_t count, const void* add, void* out, int type,
                                 cudaStream_t stream);

// dz (unless nullptr) and column sums of the unrounded dz (unless nullptr)
cudaError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, int64_t M, int64_t N,
                                int activation, uint16_t* dz, float* dbias, cudaStream_t stream);

cudaError_t launch_combine_backward(const void* dout, const void* y, const float* topk_w,
                                    const int32_t* dst_row, int64_t T, int64_t H, int k,
                                    int64_t rows, void* dy, float* dw, uint32_t* status,
                                    cudaStream_t stream);

}  // namespace ep
