// ep_act_backward.cu -- the elementwise half of a dense layer's backward pass:
//     dz[m, n]  = dy[m, n] * act'(z[m, n])        (SwiGLU: both halves)
//     dbias[n]  = sum_m dz[m, n], of the unrounded values
//
// Bound by the bytes of dy, z and dz.  A cluster of up to eight blocks owns a strip of
// columns: a thread has 8 of them (one 16-byte vector) of every so many rows and
// keeps their sums in registers; the block's rows meet by shuffles and in shared memory and
// the blocks' sums in the first block's, all in a fixed order, so that no
// workspace, second launch or atomic is needed.  A strip is 64 columns wide, or
// narrower (down to the 16 of a 32-byte sector) where N has too few strips to
// fill the SMs.
//
// 16,384 x 4,096: ReLU 79 us (5.1 TB/s), SiLU 88, SwiGLU 123 (5.4 TB/s), GELU 129,
// bound by its instructions (75 % of the issue slots when it took 116 with a less exact
// slope).  4,096 x 2,048: 12 to 21 us.  Clusters of four or two: at best 8 % less at one size and more at the
// others; two rows per thread and more blocks: 68 and 116 us, but 142 for
// SwiGLU; GELU two values per instruction: 135 us against 116.
#include "ep_products.cuh"
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256, kMaxCluster = 8;
constexpr int kUnroll = 4;  // rows of a thread whose loads are issued together

template <int ACT>
__global__ void __launch_bounds__(kThreads)
act_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, int64_t M,
                    int64_t N, int vecs, int cluster, uint16_t* __restrict__ dz, float* __restrict__ dbias) {
    constexpr bool kGated = ACT == EP_ACT_SWIGLU;
    constexpr int H = kGated ? 2 : 1;
    __shared__ float sums[kThreads / 32][8][H * 8];
    __shared__ float total[8 * 8 * H];  // of the strip's columns
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int col = threadIdx.x % vecs, lane_row = threadIdx.x / vecs;
    const int per = kThreads / vecs;  // rows of a block's step
    const int64_t n = ((int64_t)(blockIdx.x / cluster) * vecs + col) * 8;
    const int64_t wide = H * N;
    float sum[H * 8];
#pragma unroll
    for (int i = 0; i < H * 8; ++i) sum[i] = 0.0f;
    if (n < N) {
        const int64_t step = (int64_t)cluster * per;
        for (int64_t m0 = (int64_t)rank * per + lane_row; m0 < M; m0 += kUnroll * step) {
            uint4 d[kUnroll], q[kUnroll][H];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t m = m0 + u * step;
                if (m < M) {
                    d[u] = ld_stream_v4(dy + m * N + n);
                    if (ACT != EP_ACT_NONE) {
#pragma unroll
                        for (int h = 0; h < H; ++h) q[u][h] = ld_stream_v4(z + m * wide + h * N + n);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t m = m0 + u * step;
                if (m >= M) break;
                const uint32_t dd[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
                float g[H][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = i & 1 ? bf16hi_to_f32(dd[i / 2]) : bf16lo_to_f32(dd[i / 2]);
                    if constexpr (ACT == EP_ACT_NONE) {
                        g[0][i] = v;
                    } else {
                        float x[H];
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const uint32_t w[4] = {q[u][h].x, q[u][h].y, q[u][h].z, q[u][h].w};
                            x[h] = i & 1 ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
                        }
                        if constexpr (kGated)
                            swiglu_back(x[0], x[H - 1], v, g[0][i], g[H - 1][i]);
                        else
                            g[0][i] = activate_back(x[0], v, ACT);
                    }
                }
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    if (ACT != EP_ACT_NONE)
                        st_v4(dz + m * wide + h * N + n,
                              make_uint4(pack_bf16x2_rn(g[h][0], g[h][1]), pack_bf16x2_rn(g[h][2], g[h][3]),
                                         pack_bf16x2_rn(g[h][4], g[h][5]), pack_bf16x2_rn(g[h][6], g[h][7])));
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[h * 8 + i] += g[h][i];
                }
            }
        }
    }
    if (dbias == nullptr) return;  // for all blocks
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = vecs; o < 32; o *= 2) {
#pragma unroll
        for (int i = 0; i < H * 8; ++i) sum[i] += __shfl_xor_sync(kFullMask, sum[i], o);
    }
    if (lane < vecs) {
#pragma unroll
        for (int i = 0; i < H * 8; ++i) sums[warp][lane][i] = sum[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < vecs * H * 8; i += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += sums[w][i / (H * 8)][i % (H * 8)];
        total[i] = s;
    }
    cluster_sync();
    if (rank == 0) {
        for (int i = threadIdx.x; i < vecs * H * 8; i += kThreads) {
            float s = 0.0f;
            for (int r = 0; r < cluster; ++r) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(v)
                             : "r"(cluster_addr(smem_addr(total + i), r))
                             : "memory");
                s += v;
            }
            const int64_t at = ((int64_t)(blockIdx.x / cluster) * vecs + i / (H * 8)) * 8 + i % 8;
            if (at < N) dbias[(i % (H * 8) / 8) * N + at] = s;
        }
    }
    cluster_sync();  // the other blocks' sums stay until they are read
}

}  // namespace

cudaError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, int64_t M, int64_t N,
                                int activation, uint16_t* dz, float* dbias, cudaStream_t stream) {
    static std::atomic<int> sm_cache[64];
    const int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    // strips of 64 columns, clusters while every thread has four rows, and
    // narrower strips while there are fewer blocks than SMs
    const int64_t all = N / 8;
    int vecs = 8;
    auto blocks_of = [&](int v) {
        const int64_t rows = 4 * (kThreads / v);
        const int64_t c = M <= rows ? 1 : M <= 2 * rows ? 2 : M <= 4 * rows ? 4 : kMaxCluster;
        return std::pair<int64_t, int>((all + v - 1) / v, (int)c);
    };
    while (vecs > 2 && blocks_of(vecs).first * blocks_of(vecs).second < sms) vecs /= 2;
    const auto [strips, cluster] = blocks_of(vecs);
    auto kernel = activation == EP_ACT_NONE   ? act_backward_kernel<EP_ACT_NONE>
                  : activation == EP_ACT_RELU ? act_backward_kernel<EP_ACT_RELU>
                  : activation == EP_ACT_SILU ? act_backward_kernel<EP_ACT_SILU>
                  : activation == EP_ACT_GELU ? act_backward_kernel<EP_ACT_GELU>
                                              : act_backward_kernel<EP_ACT_SWIGLU>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(strips * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;  // an ordinary launch, as the products that follow it
    return cudaLaunchKernelEx(&cfg, kernel, dy, z, M, N, vecs, cluster, dz, dbias);
}

}  // namespace ep
