// ep_route.cu -- the router's choice: top-k experts of each token's logits and
// their weights.  For each token t:
//     key_e  = fl32(logit_e + bias_e)             (bias optional: choice only)
//     an expert whose key is NaN or -inf is not eligible
//     groups: with G groups of E/G experts, only the experts of the
//             groups_per_token groups with the largest key maxima remain
//     idx    = the k largest remaining keys, ties to the lower expert id
//     w      = softmax of the chosen logits, or sigmoid / their sum
//              (renormalize), else softmax over all E logits, or sigmoid;
//              times scale
// A place without an eligible expert holds id -1 and weight 0.
//
// One warp per token, expert i * 32 + lane in register i.  A key becomes an
// unsigned word of the same order (0: not eligible), so that a round of the
// selection is a maximum over the lane's registers, one redux.max for the
// key and one redux.min for the lowest id that holds it.
#include "ep_internal.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;  // tokens per block

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}

// Order-preserving word of a key; 0 for NaN and -inf (not eligible).  Adding
// +0 first makes -0 and +0 one key, as they compare equal.
__device__ __forceinline__ uint32_t ordered(float key) {
    const uint32_t b = __float_as_uint(__fadd_rn(key, 0.0f));
    if (!(key > -INFINITY)) return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// l - m where m is the largest logit: 0 for l == m, also when both are +inf.
__device__ __forceinline__ float below(float l, float m) {
    return l == m ? 0.0f : __fadd_rn(l, -m);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

__device__ __forceinline__ float sigmoid(float l) {
    return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l)));
}

template <int NV, typename L>
__global__ void __launch_bounds__(kWarps * 32)
route_kernel(const L* __restrict__ logits, const float* __restrict__ bias, int64_t T, int E, int k,
             int groups, int groups_per_token, int scoring, int renormalize, float scale,
             int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
             uint32_t* __restrict__ status) {
    __shared__ uint32_t group_best[kWarps][EP_MAX_GROUPS];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= T) return;  // warp-uniform
    const L* row = logits + t * E;

    uint32_t key[NV];
    float top = -INFINITY;  // largest logit of this lane, and after warp_max of the token
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0u;
        if (e < E) {
            const float l = load_logit(row + e);
            const float c = bias ? __fadd_rn(l, __ldg(bias + e)) : l;
            bad |= c != c;
            key[i] = ordered(c);
            top = fmaxf(top, l);  // fmaxf passes over a NaN
        }
    }
    warp_flag(status, bad, EP_FLAG_BAD_LOGIT);

    if (groups_per_token < groups) {
        const int per = E / groups;
        uint32_t* best = group_best[warp];
        best[lane] = 0u;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = i * 32 + lane;
            if (e < E && key[i]) atomicMax(best + e / per, key[i]);
        }
        __syncwarp();
        uint32_t mine = best[lane], chosen = 0u;
        for (int r = 0; r < groups_per_token; ++r) {
            const uint32_t m = __reduce_max_sync(kFullMask, mine);
            if (m == 0u) break;
            const int g = __ffs(__ballot_sync(kFullMask, mine == m)) - 1;
            chosen |= 1u << g;
            if (lane == g) mine = 0u;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = i * 32 + lane;
            if (e < E && !((chosen >> (e / per)) & 1u)) key[i] = 0u;
        }
    }

    int my_idx = -1;  // lane j: the j-th choice
    for (int j = 0; j < k; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(kFullMask, m);
        if (m == 0u) break;
        int e = INT32_MAX;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
            if (key[i] == m) e = i * 32 + lane;
        e = __reduce_min_sync(kFullMask, e);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * 32 + lane == e) key[i] = 0u;
        if (lane == j) my_idx = e;
    }

    const bool live = my_idx >= 0;
    const float l = live ? load_logit(row + my_idx) : -INFINITY;
    float p;
    if (scoring == EP_SCORE_SOFTMAX) {
        // renormalised: the softmax over the chosen logits alone, so that
        // nothing is lost when a bias chooses experts far below the maximum
        const float m = warp_max(renormalize ? l : top);
        p = live ? expf(below(l, m)) : 0.0f;
        if (!renormalize) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = i * 32 + lane;
                if (e < E) {
                    const float v = load_logit(row + e);
                    if (v == v) s = __fadd_rn(s, expf(below(v, m)));
                }
            }
            s = warp_sum(s);
            p = live ? __fdiv_rn(p, s) : 0.0f;
        }
    } else {
        p = live ? sigmoid(l) : 0.0f;
    }
    if (renormalize) {
        const float s = warp_sum(p);
        p = s > 0.0f ? __fdiv_rn(p, s) : 0.0f;
    }
    if (lane < k) {
        topk_idx[t * k + lane] = my_idx;
        topk_w[t * k + lane] = live ? __fmul_rn(p, scale) : 0.0f;
    }
}

template <typename L>
cudaError_t launch(const L* logits, const float* bias, int64_t T, int E, int k, int groups,
                   int groups_per_token, int scoring, int renormalize, float scale,
                   int32_t* topk_idx, float* topk_w, uint32_t* status, cudaStream_t stream) {
    const dim3 grid((unsigned)((T + kWarps - 1) / kWarps)), block(kWarps * 32);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, stream, logits, bias, T, E, k, groups,
                          groups_per_token, scoring, renormalize, scale, topk_idx, topk_w, status);
    };
    if (E <= 32) return go(route_kernel<1, L>);
    if (E <= 64) return go(route_kernel<2, L>);
    if (E <= 128) return go(route_kernel<4, L>);
    if (E <= 256) return go(route_kernel<8, L>);
    if (E <= 512) return go(route_kernel<16, L>);
    return go(route_kernel<32, L>);
}

}  // namespace

cudaError_t launch_route(const void* logits, int type, const float* bias, int64_t T, int E, int k,
                         int groups, int groups_per_token, int scoring, int renormalize,
                         float scale, int32_t* topk_idx, float* topk_w, uint32_t* status,
                         cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    if (type == EP_TYPE_F32)
        return launch(static_cast<const float*>(logits), bias, T, E, k, groups, groups_per_token,
                      scoring, renormalize, scale, topk_idx, topk_w, status, stream);
    return launch(static_cast<const uint16_t*>(logits), bias, T, E, k, groups, groups_per_token,
                  scoring, renormalize, scale, topk_idx, topk_w, status, stream);
}

}  // namespace ep
