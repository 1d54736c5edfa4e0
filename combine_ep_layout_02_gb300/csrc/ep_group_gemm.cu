// ep_group_gemm.cu -- the experts' products over a dispatched FP8 buffer.
// Row r of expert e, with K channels in blocks of 128 (b = k / 128):
//     y[r, n] = sum_b a_scale[r, b] * w_scale[e, n/128, b]
//                     * sum_{k in b} a[r, k] * w[e, n, k]
// e4m3 codes, the block's sum and the sum over blocks in fp32.  Two forms:
//   plain   out[r, n] = bf16_rne(y[r, n])
//   swiglu  the expert's rows n < I are the gate, I <= n < 2I the up
//           projection: h = gate / (1 + exp(-gate)) * up in fp32, then the
//           e4m3 cast of ep_dispatch_fp8 per row and 128 channels of h.
#include "ep_internal.cuh"

namespace ep {
namespace {

constexpr int kRows = 8;  // rows of one expert per pass of a block

template <bool SWIGLU>
__global__ void __launch_bounds__(128)
group_gemm_kernel(const uint8_t* __restrict__ a_q, const float* __restrict__ a_scale, int64_t rows,
                  int64_t K, const uint8_t* __restrict__ w_q, const float* __restrict__ w_scale,
                  int64_t N, const int32_t* __restrict__ counts,
                  const int32_t* __restrict__ offsets, int kind, int capacity,
                  uint16_t* __restrict__ out, uint8_t* __restrict__ out_q,
                  float* __restrict__ out_scale, uint32_t* __restrict__ status) {
    __shared__ float as[kRows][128];
    __shared__ float ss[kRows];
    __shared__ float warp_amax[4];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y, tid = threadIdx.x;
    const Segment seg = expert_segment(e, counts, offsets, kind, capacity, rows);
    if (seg.bad && blockIdx.x == 0 && tid == 0 && status) atomicOr(status, EP_FLAG_BAD_ROW);
    const int64_t n = (int64_t)blockIdx.x * 128 + tid;
    const int64_t kb = K / 128, nb = (N + 127) / 128;
    const int64_t wrows = SWIGLU ? 2 * N : N, wnb = SWIGLU ? 2 * nb : nb;
    const bool live = n < N;
    const uint8_t* wg = w_q + ((int64_t)e * wrows + (live ? n : 0)) * K;
    const float* sg = w_scale + ((int64_t)e * wnb + blockIdx.x) * kb;
    for (int64_t r0 = 0; r0 < seg.count; r0 += kRows) {
        float acc[kRows], up[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r] = up[r] = 0.0f;
        for (int64_t b = 0; b < kb; ++b) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                as[r][tid] = r0 + r < seg.count
                                 ? e4m3_to_f32(a_q[(seg.first + r0 + r) * K + b * 128 + tid])
                                 : 0.0f;
            if (tid < kRows)
                ss[tid] = r0 + tid < seg.count ? a_scale[(seg.first + r0 + tid) * kb + b] : 0.0f;
            __syncthreads();
#pragma unroll
            for (int half = 0; half < (SWIGLU ? 2 : 1); ++half) {
                float p[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) p[r] = 0.0f;
                const uint8_t* w = wg + half * N * K + b * 128;
                for (int c = 0; c < 128; c += 16) {
                    const uint4 v = *reinterpret_cast<const uint4*>(w + c);
                    const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float f = e4m3_to_f32((uint8_t)(wv[i / 4] >> (8 * (i % 4))));
#pragma unroll
                        for (int r = 0; r < kRows; ++r) p[r] = __fmaf_rn(as[r][c + i], f, p[r]);
                    }
                }
                const float sb = sg[half * nb * kb + b];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float& to = half ? up[r] : acc[r];
                    to = __fmaf_rn(p[r], __fmul_rn(ss[r], sb), to);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r0 + r >= seg.count) break;
            const int64_t row = seg.first + r0 + r;
            if (!SWIGLU) {
                if (live) out[row * N + n] = (uint16_t)pack_bf16x2_rn(acc[r], acc[r]);
                continue;
            }
            const float h = swiglu(acc[r], up[r]);
            float amax = fabsf(h);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
            __syncthreads();
            if ((tid & 31) == 0) warp_amax[tid >> 5] = amax;
            __syncthreads();
            const float a = fmaxf(fmaxf(fmaxf(warp_amax[0], warp_amax[1]),
                                        fmaxf(warp_amax[2], warp_amax[3])), 1e-4f);
            const float inv = __fdiv_rn(448.0f, a);
            out_q[row * N + n] = (uint8_t)cvt_e4m3x2_rn_sat(__fmul_rn(h, inv), 0.0f);
            if (tid == 0) out_scale[row * nb + blockIdx.x] = __fdiv_rn(a, 448.0f);
        }
    }
}

}  // namespace

cudaError_t launch_group_gemm(const uint8_t* a_q, const float* a_scale, int64_t rows, int64_t K,
                              const uint8_t* w_q, const float* w_scale, int64_t N, int E,
                              const int32_t* counts, const int32_t* offsets, int kind,
                              int capacity, void* out, uint8_t* out_q, float* out_scale,
                              uint32_t* status, cudaStream_t stream) {
    const dim3 grid((unsigned)((N + 127) / 128), (unsigned)E);
    return launch_pdl(out ? group_gemm_kernel<false> : group_gemm_kernel<true>, grid, dim3(128), 0,
                      stream, a_q, a_scale, rows, K, w_q, w_scale, N, counts, offsets, kind,
                      capacity, static_cast<uint16_t*>(out), out_q, out_scale, status);
}

}  // namespace ep
