// ep_combine_backward.cu -- gradients of the weighted combine.  For every pair
// (t, j) with a row r = dst_row[t, j]:
//     dy[r, :] = bf16(w[t, j] * dout[t, :])
//     dw[t, j] = sum_h dout[t, h] * y[r, h]
//
// One warp per token: it reads its row of dout once per pair and y's row beside
// it; a lane's products are added in order of h, the lanes by a butterfly.
#include "ep_products.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                        const float* __restrict__ topk_w, const int32_t* __restrict__ dst_row,
                        int64_t T, int64_t nvec, int k, int64_t rows, uint4* __restrict__ dy,
                        float* __restrict__ dw, uint32_t* __restrict__ status) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= T) return;  // warp-uniform
    const int my_row = load_dst_row(dst_row, t, k, rows, status);
    const float my_w = lane < k ? __ldg(topk_w + t * k + lane) : 0.0f;
    for (int j = 0; j < k; ++j) {
        const int r = __shfl_sync(kFullMask, my_row, j);
        const float w = __shfl_sync(kFullMask, my_w, j);
        float sum = 0.0f;
        if (r >= 0) {
            for (int64_t v = lane; v < nvec; v += 32) {
                const uint4 d = dout[t * nvec + v];
                const uint4 q = dw ? y[r * nvec + v] : make_uint4(0, 0, 0, 0);
                const uint32_t dd[4] = {d.x, d.y, d.z, d.w}, qq[4] = {q.x, q.y, q.z, q.w};
                uint32_t o[4];
                for (int i = 0; i < 4; ++i) {
                    const float lo = bf16lo_to_f32(dd[i]), hi = bf16hi_to_f32(dd[i]);
                    sum = fmaf(lo, bf16lo_to_f32(qq[i]), sum);
                    sum = fmaf(hi, bf16hi_to_f32(qq[i]), sum);
                    o[i] = pack_bf16x2_rn(w * lo, w * hi);
                }
                st_v4(dy + r * nvec + v, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        if (dw && lane == 0) dw[t * k + j] = sum;
    }
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* y, const float* topk_w,
                                    const int32_t* dst_row, int64_t T, int64_t H, int k,
                                    int64_t rows, void* dy, float* dw, uint32_t* status,
                                    cudaStream_t stream) {
    return launch_pdl(combine_backward_kernel, dim3((unsigned)((T + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0,
                      stream, static_cast<const uint4*>(dout), static_cast<const uint4*>(y), topk_w, dst_row, T,
                      H / 8, k, rows, static_cast<uint4*>(dy), dw, status);
}

}  // namespace ep
