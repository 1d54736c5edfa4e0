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
// One warp per token.  Where E is 32 times a register count, lane l holds the
// experts [l * NV, (l + 1) * NV), read as whole vectors; otherwise register i
// holds expert i * 32 + lane.  A key becomes an unsigned word of the same order (0: not eligible).  The k-th largest of the
// 32 lanes' maxima is at most the k-th largest key, so that every choice is
// among the keys that reach it: usually a dozen, which move one to a lane
// and are ranked against each other.  Where more
// than 32 reach it (many equal keys, or k near 32) k rounds of a maximum over
// the warp find the choices instead.
//
// Bound by the instructions of one token (about 510 per warp; 85 % of the
// issue slots): 65,536 x 256 logits, 4 of 8 groups, k = 8: 33 us, 2.1 TB/s.  k
// rounds over all registers instead of the candidates took 103 us.  Of the 510
// the keys take 110, the groups 45, the threshold 50, collecting the candidates
// 110, ranking them 100, weights and output 90.
#include "ep_experts.cuh"

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
// N values from p, aligned to all of them or to 16 bytes.
template <int N>
__device__ __forceinline__ void load_logits(float (&v)[N], const float* p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
    }
}
template <int N>
__device__ __forceinline__ void load_logits(float (&v)[N], const uint16_t* p) {
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + i));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + 2 * j] = bf16lo_to_f32(w[j]), v[i + 2 * j + 1] = bf16hi_to_f32(w[j]);
        }
    } else if constexpr (N == 4) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
        v[0] = bf16lo_to_f32(q.x), v[1] = bf16hi_to_f32(q.x), v[2] = bf16lo_to_f32(q.y), v[3] = bf16hi_to_f32(q.y);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = load_logit(p + i);
    }
}

// Order-preserving word of a key; 0 for NaN and -inf (not eligible).  Adding
// +0 first makes -0 and +0 one key, as they compare equal; fmaxf turns a NaN
// into -inf, whose word 0x007fffff is the origin.
constexpr uint32_t kOrigin = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered(float key) {
    const int32_t b = __float_as_int(fmaxf(__fadd_rn(key, 0.0f), -INFINITY));
    return ((uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u)) - kOrigin;
}
// The key of a word.
__device__ __forceinline__ float unordered(uint32_t w) {
    w += kOrigin;
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

// The choice of groups, with its divisions made on the host.
struct GroupChoice {
    int groups, chosen;
    uint32_t inverse;  // group_of()'s
    int span_log2;     // whole vectors per lane: lanes of a group, if a power of two (else -1)
};

template <int NV, bool FULL, typename L>
__global__ void __launch_bounds__(kWarps * 32)
route_kernel(const L* __restrict__ logits, const float* __restrict__ bias, int64_t T, int E, int k,
             GroupChoice gc, int scoring, int renormalize, float scale,
             int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
             uint32_t* __restrict__ status) {
    // candidates as (word, ~id), in the order of the choice; the groups' best keys before that
    __shared__ uint64_t list[kWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t t = blockIdx.x * kWarps + warp;  // T * k < 2^31
    if (t >= (uint32_t)T) return;  // warp-uniform
    const L* row = logits + (uint64_t)t * (uint32_t)E;
    uint64_t* mine = list[warp];

    auto id = [lane](int i) { return FULL ? lane * NV + i : i * 32 + lane; };
    float v[NV];
    if constexpr (FULL) {
        load_logits<NV>(v, row + lane * NV);
        if (bias) {
            float w[NV];
            load_logits<NV>(w, bias + lane * NV);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = __fadd_rn(v[i], w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = id(i) < E ? load_logit(row + id(i)) : -INFINITY;
        if (bias) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (id(i) < E) v[i] = __fadd_rn(v[i], __ldg(bias + id(i)));
        }
    }
    if (status) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) bad |= v[i] != v[i];
        warp_flag(status, bad, EP_FLAG_BAD_LOGIT);
    }
    uint32_t key[NV], top = 0u;  // the largest key of this lane
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        key[i] = ordered(v[i]);
        top = max(top, key[i]);
    }

    bool in = true;  // FULL: whether the lane's experts are in a chosen group
    if (gc.chosen < gc.groups) {
        if (FULL && gc.span_log2 >= 0) {  // the groups are equal runs of lanes
            const int span = 1 << gc.span_log2, group = lane >> gc.span_log2;
            uint32_t best = top;  // of this lane's group, 0 once it is chosen
            for (int o = 1; o < span; o <<= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
            in = false;
            for (int r = 0; r < gc.chosen; ++r) {
                const uint32_t m = __reduce_max_sync(kFullMask, best);
                const int first = __ffs(__ballot_sync(kFullMask, best == m)) - 1;
                if (group == first >> gc.span_log2) {
                    in = true;
                    best = 0u;
                }
            }
            if (!in) top = 0u;
        } else {
            uint32_t* bests = reinterpret_cast<uint32_t*>(mine);
            bests[lane] = 0u;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (key[i]) atomicMax(bests + group_of(id(i), gc.inverse), key[i]);
            __syncwarp();
            const uint32_t best = bests[lane];  // of group `lane`
            __syncwarp();
            int rank = 0;  // how many groups are better, or as good and earlier
#pragma unroll 4
            for (int g = 0; g < gc.groups; ++g) {
                const uint32_t other = __shfl_sync(kFullMask, best, g);
                rank += other > best || (other == best && g < lane);
            }
            const unsigned chosen = __ballot_sync(kFullMask, rank < gc.chosen);
            top = 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!((chosen >> (group_of(id(i), gc.inverse) & 31)) & 1u)) key[i] = 0u;
                top = max(top, key[i]);
            }
        }
    }

    uint32_t reach = 0u;  // 0 at the end where fewer than k lanes have a key
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
        reach = __reduce_max_sync(kFullMask, top);
        if (top == reach) top = 0u;
    }
    const uint32_t bar = in ? max(reach, 1u) : 0xffffffffu;  // no key is that large
    int own = 0;  // candidates of this lane, then of the lanes up to it
#pragma unroll
    for (int i = 0; i < NV; ++i) own += key[i] >= bar;
    int at = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(kFullMask, at, o);
        if (lane >= o) at += below;
    }
    const int count = __shfl_sync(kFullMask, at, 31);
    if (count <= 32 && own > 0) {
        at -= own;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] >= bar) mine[at++] = ((uint64_t)key[i] << 32) | ~(uint32_t)id(i);
    }
    __syncwarp();

    int idx = -1, place = lane;  // this lane's choice and its place among the k
    uint32_t word = 0u;
    if (count <= 32) {
        place = 32;
        if (lane < count) {
            const uint64_t c = mine[lane];
            word = (uint32_t)(c >> 32);
            place = 0;
#pragma unroll 4
            for (int q = 0; q < count; ++q) place += mine[q] > c;
            idx = place < k ? (int)~(uint32_t)c : -1;
        }
        const int found = min(count, k);
        if (idx < 0) place = lane >= found && lane < k ? lane : 32;  // places left over hold no candidate
    } else {
        for (int j = 0; j < k; ++j) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) m = max(m, in ? key[i] : 0u);
            m = __reduce_max_sync(kFullMask, m);
            if (m == 0u) break;
            int e = INT32_MAX;
#pragma unroll
            for (int i = NV - 1; i >= 0; --i)
                if (in && key[i] == m) e = id(i);
            e = __reduce_min_sync(kFullMask, e);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (id(i) == e) key[i] = 0u;
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
            const float m = unordered(__reduce_max_sync(kFullMask, live ? ordered(l) : 0u));
            p = live ? expf(below(l, m)) : 0.0f;
            const float s = warp_sum(p);  // 1 to k, or 0 without a choice
            p = live ? __fdividef(p, s) : 0.0f;
        } else {
            float m = -INFINITY, s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (id(i) < E) m = fmaxf(m, load_logit(row + id(i)));  // passes over a NaN
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (id(i) < E) {
                    const float w = load_logit(row + id(i));
                    if (w == w) s = __fadd_rn(s, expf(below(w, m)));
                }
            }
            s = warp_sum(s);
            p = live ? __fdiv_rn(expf(below(l, m)), s) : 0.0f;
        }
    } else {
        p = live ? sigmoid(l) : 0.0f;
        if (renormalize) {
            const float s = warp_sum(p);
            p = s > 0.0f ? __fdiv_rn(p, s) : 0.0f;
        }
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
    const int per = E / groups;
    GroupChoice gc{groups, groups_per_token, ((1u << 20) + per - 1) / per, -1};
    if ((groups & (groups - 1)) == 0 && E % 32 == 0)  // 32 / groups lanes each
        for (gc.span_log2 = 0; (groups << gc.span_log2) < 32;) ++gc.span_log2;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, stream, logits, bias, T, E, k, gc, scoring,
                          renormalize, scale, topk_idx, topk_w, status);
    };
    // Whole vectors per lane where a row is 32 lanes of a power of two of
    // registers and lies on 16 bytes.  Other rows take single loads, and the
    // groups' maxima by atomics in shared memory, in the next power of two of
    // registers: 65,536 tokens, fp32, k = 8, without groups and with 4 of 8, in us:
    // 96 experts 22 and 31 (128: 22 and 28), 160 experts 27 and 45 (256: 26 and
    // 32), 384 experts 37 and 100 (512: 35 and 40).
    const bool vectors = ((uintptr_t)logits | (uintptr_t)bias) % 16 == 0;
    if (vectors && E == 64) return go(route_kernel<2, true, L>);
    if (vectors && E == 128) return go(route_kernel<4, true, L>);
    if (vectors && E == 256) return go(route_kernel<8, true, L>);
    if (vectors && E == 512) return go(route_kernel<16, true, L>);
    if (vectors && E == 1024) return go(route_kernel<32, true, L>);
    if (E <= 32) return go(route_kernel<1, false, L>);
    if (E <= 64) return go(route_kernel<2, false, L>);
    if (E <= 128) return go(route_kernel<4, false, L>);
    if (E <= 256) return go(route_kernel<8, false, L>);
    if (E <= 512) return go(route_kernel<16, false, L>);
    return go(route_kernel<32, false, L>);
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
