// ep_products.cu -- BF16 products grouped by expert, with their gradients.
//
// One block per 64 x 64 outputs of an expert, 4 x 4 per thread, fp32 FMAs from
// shared memory: right for every case, and bound by those FMAs.
#include "ep_products.cuh"

namespace ep {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <ProductKind KIND, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) product_kernel(const __grid_constant__ ProductArgs p) {
    // m: rows of the buffer (kWeight: of the weights); n: output channels; c: the summed index
    constexpr bool pair = SWIGLU && KIND == kForward;
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1], su[pair ? kStep : 1][kTile + 1];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.z;
    const Segment s = product_segment(p, e);
    if (s.bad && p.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        atomicOr(p.status, EP_FLAG_BAD_ROW);
    const int64_t half = pair ? p.N / 2 : 0;
    const int64_t nn = KIND == kForward ? (pair ? half : p.N) : p.K;  // output channels
    const int64_t mm = KIND == kWeight ? p.N : s.count;
    const int64_t cc = KIND == kForward ? p.K : KIND == kInput ? p.N : s.count;
    const uint16_t* w = p.b + (int64_t)e * p.N * p.K;
    const int64_t n0 = (int64_t)blockIdx.x * kTile;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    for (int64_t m0 = (int64_t)blockIdx.y * kTile; m0 < mm; m0 += (int64_t)gridDim.y * kTile) {
        float acc[4][4] = {}, accu[4][4] = {};
        for (int64_t c0 = 0; c0 < cc; c0 += kStep) {
            for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
                // the index that is contiguous in memory varies fastest over the threads
                const int mc = KIND == kWeight ? i / kTile : i % kStep, mx = KIND == kWeight ? i % kTile : i / kStep;
                const int64_t m = m0 + mx, c = c0 + mc;
                float v = 0.0f;
                if (m < mm && c < cc)
                    v = KIND == kWeight ? bf16_value(p.a[(s.first + c) * p.N + m])
                                        : bf16_value(p.a[(s.first + m) * cc + c]);
                sa[mc][mx] = v;
            }
            for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
                const int nc = KIND == kForward ? i % kStep : i / kTile, nx = KIND == kForward ? i / kStep : i % kTile;
                const int64_t n = n0 + nx, c = c0 + nc;
                float v = 0.0f, u = 0.0f;
                if (n < nn && c < cc) {
                    if (KIND == kForward) {
                        v = bf16_value(w[n * p.K + c]);
                        if (pair) u = bf16_value(w[(half + n) * p.K + c]);
                    } else if (KIND == kInput) {
                        v = bf16_value(w[c * p.K + n]);
                    } else {
                        v = bf16_value(p.b[(s.first + c) * p.K + n]);
                    }
                }
                sb[nc][nx] = v;
                if (pair) su[nc][nx] = u;
            }
            __syncthreads();
            for (int c = 0; c < kStep; ++c)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = fmaf(sa[c][tm + i], sb[c][tn + j], acc[i][j]);
                        if (pair) accu[i][j] = fmaf(sa[c][tm + i], su[c][tn + j], accu[i][j]);
                    }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + tm + i, n = n0 + tn + j;
                if (m >= mm || n >= nn) continue;
                const int64_t row = s.first + m;
                float v = acc[i][j];
                if (KIND == kWeight) {
                    const int64_t at = ((int64_t)e * p.N + m) * p.K + n;
                    if (p.add)
                        v += p.out_type == EP_TYPE_F32 ? static_cast<const float*>(p.add)[at]
                                                       : bf16_value(static_cast<const uint16_t*>(p.add)[at]);
                    if (p.out_type == EP_TYPE_F32) static_cast<float*>(p.out)[at] = v;
                    else static_cast<uint16_t*>(p.out)[at] = bf16_bits(v);
                    continue;
                }
                if (KIND == kInput) {
                    uint16_t* out = static_cast<uint16_t*>(p.out);
                    if (!SWIGLU) {
                        out[row * nn + n] = bf16_bits(v);
                    } else {
                        const int64_t at = row * 2 * nn + n;
                        float dg, du;
                        swiglu_back(bf16_value(p.z[at]), bf16_value(p.z[at + nn]), v, dg, du);
                        out[at] = bf16_bits(dg);
                        out[at + nn] = bf16_bits(du);
                    }
                    continue;
                }
                if (p.bias) v += load_typed(p.bias, p.bias_type, n);
                if (pair) {
                    float u = accu[i][j];
                    if (p.bias) u += load_typed(p.bias, p.bias_type, nn + n);
                    if (p.z) {
                        p.z[row * 2 * nn + n] = bf16_bits(v);
                        p.z[row * 2 * nn + nn + n] = bf16_bits(u);
                    }
                    v = swiglu(v, u);
                } else {
                    if (p.z) p.z[row * nn + n] = bf16_bits(v);
                    v = activate(v, p.activation);
                }
                const int64_t at = row * nn + n;
                if (p.residual)
                    v += p.out_type == EP_TYPE_F32 ? static_cast<const float*>(p.residual)[at]
                                                   : bf16_value(static_cast<const uint16_t*>(p.residual)[at]);
                if (p.out_type == EP_TYPE_F32) static_cast<float*>(p.out)[at] = v;
                else static_cast<uint16_t*>(p.out)[at] = bf16_bits(v);
            }
    }
}

}  // namespace

cudaError_t launch_product(const ProductArgs& p, ProductKind kind, cudaStream_t stream) {
    const bool swiglu = p.activation == EP_ACT_SWIGLU;
    const int64_t nn = kind == kForward ? (swiglu ? p.N / 2 : p.N) : p.K;
    const int64_t mm = kind == kWeight ? p.N : p.rows;
    const int64_t tiles = (mm + kTile - 1) / kTile;
    const dim3 grid((unsigned)((nn + kTile - 1) / kTile), (unsigned)(tiles < 64 ? tiles : 64), (unsigned)p.E);
    auto kernel = kind == kForward ? (swiglu ? product_kernel<kForward, true> : product_kernel<kForward, false>)
                  : kind == kInput ? (swiglu ? product_kernel<kInput, true> : product_kernel<kInput, false>)
                                   : product_kernel<kWeight, false>;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace ep
