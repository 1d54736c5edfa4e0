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
// unsigned word of the same order (0: not eligible).  The k-th largest of the
// 32 lanes' maxima is at most the k-th largest key, so that every choice is
// among the keys that reach it: usually a dozen, which move one to a lane
// (in the order of their ids) and are ranked against each other.  Where more
// than 32 reach it (many equal keys, or k near 32) k rounds of a maximum over
// the warp find the choices instead.
//
// Bound by the ALU: MEASURED_ROUTE.
#include "ep_internal.cuh"

namespace ep {
namespace {

#ifndef EP_ROUTE_WARPS
#define EP_ROUTE_WARPS 8
#endif
constexpr int kWarps = EP_ROUTE_WARPS;  // tokens per block

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

// The key of a non-zero word.
__device__ __forceinline__ float unordered(uint32_t w) {
    return __uint_as_float((w & 0x80000000u) ? (w ^ 0x80000000u) : ~w);
}

// Group of expert e < 2^10 for groups of `per` <= 2^10: e / per by a
// multiplication with ceil(2^20 / per), exact because e * per < 2^20.
__device__ __forceinline__ int group_of(int e, uint32_t inverse) { return (int)(((uint32_t)e * inverse) >> 20); }

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
    __shared__ uint2 list[kWarps][32];  // candidates: key, id; the groups' best keys before that
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= T) return;  // warp-uniform
    const L* row = logits + t * E;
    uint2* mine = list[warp];

    uint32_t key[NV];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        float c = -INFINITY;
        if (e < E) {
            c = load_logit(row + e);
            if (bias) c = __fadd_rn(c, __ldg(bias + e));
        }
        bad |= c != c;
        key[i] = ordered(c);
    }
    warp_flag(status, bad, EP_FLAG_BAD_LOGIT);

    if (groups_per_token < groups) {
        const int per = E / groups;
        const uint32_t inverse = ((1u << 20) + per - 1) / per;
        uint32_t best = 0u;  // lane g: the best key of group g
        if (per % 32 == 0) {  // a register's 32 experts lie in one group
            const int regs = per / 32;
            int g = 0, left = regs;
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                m = max(m, key[i]);
                if (--left == 0) {
                    m = __reduce_max_sync(kFullMask, m);
                    if (lane == g) best = m;
                    ++g;
                    left = regs;
                    m = 0u;
                }
            }
        } else {
            mine[lane].x = 0u;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (key[i]) atomicMax(&mine[group_of(i * 32 + lane, inverse)].x, key[i]);
            __syncwarp();
            best = mine[lane].x;
            __syncwarp();
        }
        // a group's rank: how many are better, or as good and earlier
        int rank = 0;
        for (int g = 0; g < groups; ++g) {
            const uint32_t other = __shfl_sync(kFullMask, best, g);
            rank += other > best || (other == best && g < lane);
        }
        const unsigned chosen = __ballot_sync(kFullMask, rank < groups_per_token);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = group_of(per % 32 == 0 ? i * 32 : i * 32 + lane, inverse);
            if (!((chosen >> (g & 31)) & 1u)) key[i] = 0u;
        }
    }

    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = max(top, key[i]);
    uint32_t reach = 1u;  // every eligible key, where there are fewer than k lanes with one
    for (int j = 0; j < k; ++j) {
        const uint32_t m = __reduce_max_sync(kFullMask, top);
        reach = max(m, 1u);
        if (m == 0u) break;
        if (top == m) top = 0u;
    }
    int count = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const unsigned b = __ballot_sync(kFullMask, key[i] >= reach);
        const int at = count + __popc(b & lanemask_lt());
        if (key[i] >= reach && at < 32) mine[at] = make_uint2(key[i], i * 32 + lane);
        count += __popc(b);
    }
    __syncwarp();

    int idx = -1, place = lane;  // this lane's choice and its place among the k
    uint32_t word = 0u;
    if (count <= 32) {
        place = 32;
        if (lane < count) {
            const uint2 c = mine[lane];
            word = c.x;
            place = 0;
            for (int q = 0; q < count; ++q) {
                const uint32_t other = mine[q].x;
                place += other > word || (other == word && q < lane);
            }
            idx = place < k ? (int)c.y : -1;
        }
        const int found = min(count, k);
        if (idx < 0) place = lane >= found && lane < k ? lane : 32;  // places left over hold no candidate
    } else {
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
            if (lane == j) {
                idx = e;
                word = m;
            }
        }
    }

    const bool live = idx >= 0;
    const float l = !live ? -INFINITY : bias ? load_logit(row + idx) : unordered(word);
    float p;
    if (scoring == EP_SCORE_SOFTMAX) {
        if (renormalize) {
            // the softmax over the chosen logits alone, so that nothing is lost
            // when a bias chooses experts far below the maximum
            const float m = warp_max(l);
            p = live ? expf(below(l, m)) : 0.0f;
        } else {
            float m = -INFINITY, s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * 32 + lane < E) m = fmaxf(m, load_logit(row + i * 32 + lane));  // passes over a NaN
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * 32 + lane < E) {
                    const float v = load_logit(row + i * 32 + lane);
                    if (v == v) s = __fadd_rn(s, expf(below(v, m)));
                }
            }
            s = warp_sum(s);
            p = live ? __fdiv_rn(expf(below(l, m)), s) : 0.0f;
        }
    } else {
        p = live ? sigmoid(l) : 0.0f;
    }
    if (renormalize) {
        const float s = warp_sum(p);
        p = s > 0.0f ? __fdiv_rn(p, s) : 0.0f;
    }
    if (place < k) {
        topk_idx[t * k + place] = idx;
        topk_w[t * k + place] = live ? __fmul_rn(p, scale) : 0.0f;
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
