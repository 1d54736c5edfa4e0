// ep_combine_backward.cu -- gradients of the weighted combine.  For every pair
// (t, j) with a row r = dst_row[t, j]:
//     dy[r, :] = bf16(w[t, j] * dout[t, :])
//     dw[t, j] = sum_h dout[t, h] * y[r, h]
//
// Bound by bytes: y's rows are read and dy's written once, dout's once per
// batch of eight pairs.  A block has one token (or, with few channels, several),
// its warps take groups of channels in turn: per group a lane loads 8
// channels of dout and of all rows of the batch before it computes, so that up to
// nine 16-byte loads are in flight per lane, and keeps a sum per pair.  The
// lanes' sums meet in a butterfly and the warps' in shared memory, in a fixed
// order.  16,384 tokens of 7,168 channels, k 8: 593 us, 6.74 TB/s (a plain copy
// 6.78); pair after pair, one warp per token, took 835 us.  128 tokens of 2,048:
// 4 us, the call 7 us.
#include "ep_products.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;

// `share` warps per token (1, 2, 4 or 8).
__global__ void __launch_bounds__(kWarps * 32)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                        const float* __restrict__ topk_w, const int32_t* __restrict__ dst_row,
                        int64_t T, int64_t nvec, int k, int64_t rows, int share,
                        uint4* __restrict__ dy, float* __restrict__ dw, uint32_t* __restrict__ status) {
    __shared__ float part[kWarps][EP_MAX_TOPK];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kWarps / share) + warp / share;
    const int mine = warp % share;  // of the token's warps
    if (t < T) {
        const int my_row = load_dst_row(dst_row, t, k, rows, mine == 0 ? status : nullptr);
        const float my_w = lane < k ? __ldg(topk_w + t * k + lane) : 0.0f;
        const uint4* src = dout + t * nvec;
        for (int j0 = 0; j0 < k; j0 += kRowBatch) {
            int64_t at[kRowBatch];
            float w[kRowBatch], sum[kRowBatch];
#pragma unroll
            for (int jj = 0; jj < kRowBatch; ++jj) {
                const int r = __shfl_sync(kFullMask, my_row, (j0 + jj) & 31);
                w[jj] = __shfl_sync(kFullMask, my_w, (j0 + jj) & 31);
                at[jj] = j0 + jj < k && r >= 0 ? r * nvec : -1;  // warp-uniform
                sum[jj] = 0.0f;
            }
            for (int64_t v = mine * 32 + lane; v < nvec; v += share * 32) {
                const uint4 d = j0 + kRowBatch < k ? __ldg(src + v) : ld_stream_v4(src + v);
                uint4 q[kRowBatch];
#pragma unroll
                for (int jj = 0; jj < kRowBatch; ++jj) {
                    q[jj] = make_uint4(0, 0, 0, 0);
                    if (at[jj] >= 0 && dw) q[jj] = ld_stream_v4(y + at[jj] + v);
                }
                const uint32_t dd[4] = {d.x, d.y, d.z, d.w};
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = bf16lo_to_f32(dd[i]);
                    f[2 * i + 1] = bf16hi_to_f32(dd[i]);
                }
#pragma unroll
                for (int jj = 0; jj < kRowBatch; ++jj) {
                    if (at[jj] < 0) continue;
                    const uint32_t qq[4] = {q[jj].x, q[jj].y, q[jj].z, q[jj].w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum[jj] = __fmaf_rn(f[2 * i], bf16lo_to_f32(qq[i]), sum[jj]);
                        sum[jj] = __fmaf_rn(f[2 * i + 1], bf16hi_to_f32(qq[i]), sum[jj]);
                        o[i] = pack_bf16x2_rn(__fmul_rn(w[jj], f[2 * i]), __fmul_rn(w[jj], f[2 * i + 1]));
                    }
                    st_v4(dy + at[jj] + v, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
#pragma unroll
            for (int jj = 0; jj < kRowBatch; ++jj) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    sum[jj] = __fadd_rn(sum[jj], __shfl_xor_sync(kFullMask, sum[jj], o));
                if (lane == 0 && j0 + jj < k) part[warp][j0 + jj] = sum[jj];
            }
        }
    }
    __syncthreads();
    if (dw && t < T && mine == 0 && lane < k) {
        float s = 0.0f;
        for (int i = 0; i < share; ++i) s = __fadd_rn(s, part[warp + i][lane]);
        dw[t * k + lane] = s;
    }
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* y, const float* topk_w,
                                    const int32_t* dst_row, int64_t T, int64_t H, int k,
                                    int64_t rows, void* dy, float* dw, uint32_t* status,
                                    cudaStream_t stream) {
    // A warp's step is 32 vectors.  Enough warps to fill the SMs first; beyond that
    // the largest share whose steps are no more than 15 % above one warp's (257
    // vectors: eight warps take two steps each, the second almost empty: 54 us for
    // 6,879 tokens, two pairs each, against 34; 896 vectors: 590 us, four warps 595).
    static std::atomic<int> sm_cache[64];
    const int64_t enough = 16 * (int64_t)cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    const int64_t nvec = H / 8;
    auto steps = [&](int s) { return s * ((nvec + 32 * s - 1) / (32 * s)); };
    int share = kWarps;
    while (share > 1 && (share * 16 >= nvec || (T * share >= 2 * enough && steps(share) * 100 > steps(1) * 115))) share /= 2;
    const int64_t per = kWarps / share;
    return launch_pdl(combine_backward_kernel, dim3((unsigned)((T + per - 1) / per)), dim3(kWarps * 32), 0, stream,
                      static_cast<const uint4*>(dout), static_cast<const uint4*>(y), topk_w, dst_row, T, nvec, k, rows,
                      share, static_cast<uint4*>(dy), dw, status);
}

}  // namespace ep
