// ep_act_backward.cu -- the elementwise half of a dense layer's backward pass:
//     dz[m, n]  = dy[m, n] * act'(z[m, n])        (SwiGLU: both halves)
//     dbias[n]  = sum_m dz[m, n], of the unrounded values
//
// One block per 64 columns walks all rows, its warps every 8th; their sums meet
// in shared memory in a fixed order.
#include "ep_products.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32)
act_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, int64_t M,
                    int64_t N, int activation, uint16_t* __restrict__ dz,
                    float* __restrict__ dbias) {
    __shared__ float sums[kWarps][2][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    float sg = 0.0f, su = 0.0f;
    if (n < N) {
        for (int64_t m = warp; m < M; m += kWarps) {
            const float d = bf16_value(dy[m * N + n]);
            if (activation == EP_ACT_SWIGLU) {
                float dg, du;
                swiglu_back(bf16_value(z[m * 2 * N + n]), bf16_value(z[m * 2 * N + N + n]), d, dg, du);
                dz[m * 2 * N + n] = bf16_bits(dg);
                dz[m * 2 * N + N + n] = bf16_bits(du);
                sg += dg;
                su += du;
            } else {
                const float v = activation == EP_ACT_NONE ? d : activate_back(bf16_value(z[m * N + n]), d, activation);
                if (dz) dz[m * N + n] = bf16_bits(v);
                sg += v;
            }
        }
    }
    sums[warp][0][lane] = sg;
    sums[warp][1][lane] = su;
    __syncthreads();
    if (warp == 0 && n < N && dbias) {
        for (int w = 1; w < kWarps; ++w) {
            sg += sums[w][0][lane];
            su += sums[w][1][lane];
        }
        dbias[n] = sg;
        if (activation == EP_ACT_SWIGLU) dbias[N + n] = su;
    }
}

}  // namespace

cudaError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, int64_t M, int64_t N,
                                int activation, uint16_t* dz, float* dbias, cudaStream_t stream) {
    return launch_pdl(act_backward_kernel, dim3((unsigned)((N + 31) / 32)), dim3(kWarps * 32), 0, stream, dy, z, M,
                      N, activation, dz, dbias);
}

}  // namespace ep
