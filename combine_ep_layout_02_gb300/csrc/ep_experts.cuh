// ep_experts.cuh -- what the router, the experts' products and the few-token
// layer share, and their launchers.
#pragma once

#include "ep_internal.cuh"

namespace ep {

// gate / (1 + exp(-gate)) * up, the exponential and the quotient each good to
// 2 ulp (the IEEE quotient measured 18 % more time for a whole prefill product:
// 653 against 540 us).  A gate far below zero gives a divisor of 2^126 and
// more, for which the quotient is -0, the limit.
__device__ __forceinline__ float swiglu(float gate, float up) {
    return __fmul_rn(__fdividef(gate, __fadd_rn(1.0f, expf(-gate))), up);
}

// Rows of expert e in a dispatched buffer of `rows` rows: contiguous from
// offsets[e], masked from e * capacity (a count above the capacity is the
// layout's overflow: only capacity rows exist).  A segment that reaches out
// of the buffer is cut to it and reported.
struct Segment {
    int64_t first;
    int64_t count;
    bool bad;
};
__device__ __forceinline__ Segment expert_segment(int e, const int32_t* __restrict__ counts,
                                                  const int32_t* __restrict__ offsets, int kind,
                                                  int capacity, int64_t rows) {
    int64_t n = __ldg(counts + e);
    Segment s;
    if (kind == EP_LAYOUT_MASKED) {
        s.bad = n < 0;
        s.first = (int64_t)e * capacity;  // E * capacity <= rows was checked on the host
        s.count = n < 0 ? 0 : (n < capacity ? n : capacity);
        return s;
    }
    s.first = __ldg(offsets + e);
    s.bad = n < 0 || s.first < 0 || s.first + n > rows;
    s.count = n < 0 || s.first < 0 || s.first >= rows ? 0 : (s.first + n > rows ? rows - s.first : n);
    if (s.count == 0) s.first = 0;
    return s;
}

// Exclusive scan, by a whole warp, of the experts' tiles of `most` rows into
// tiles[0..E].  Segments that overlap can make more than 31 bits of them: then
// there are none, and the answer is false.
__device__ __forceinline__ bool scan_tiles(const int* count, int E, int most, int* tiles) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int64_t n = e0 + lane < E ? ((int64_t)count[e0 + lane] + most - 1) / most : 0;
        int64_t s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(kFullMask, s, o);
            if (lane >= o) s += v;
        }
        if (e0 + lane < E) tiles[e0 + lane] = (int)(base + s - n);
        base += __shfl_sync(kFullMask, s, 31);
    }
    const bool fits = base <= INT32_MAX;
    if (lane == 0) tiles[E] = fits ? (int)base : 0;
    return fits;
}

// ---- launchers (host) ------------------------------------------------------

// the router's top-k choice
cudaError_t launch_route(const void* logits, int type, const float* bias, int64_t T, int E, int k,
                         int groups, int groups_per_token, int scoring, int renormalize,
                         float scale, int32_t* topk_idx, float* topk_w, uint32_t* status,
                         cudaStream_t stream);

// the experts' FP8 products; out (bf16) or, with the SwiGLU epilogue, out_q / out_scale
cudaError_t launch_group_gemm(const uint8_t* a_q, const float* a_scale, int64_t rows, int64_t K,
                              const uint8_t* w_q, const float* w_scale, int64_t N, int E,
                              const int32_t* counts, const int32_t* offsets, int kind,
                              int capacity, void* out, uint8_t* out_q, float* out_scale,
                              uint32_t* status, cudaStream_t stream);

// the whole expert layer for a few tokens; workspace: moe_few_bytes()
size_t moe_few_bytes(int64_t T, int k, int I);
cudaError_t launch_moe_few(const void* x, int T, int H, int k, const int32_t* topk_idx,
                           const float* topk_w, const uint8_t* w13, const float* s13,
                           const uint8_t* w2, const float* s2, int I, int E, void* out,
                           uint32_t* status, void* workspace, cudaStream_t stream);

}  // namespace ep
