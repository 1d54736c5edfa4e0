// ep_linear_few.cu -- the dense layer for a few tokens: y[m, n] = sum_k x[m, k]
// w[n, k], where the weights' bytes set the time.
//
// A block has 16 or 32 rows of weights; its eight warps, and where there are few
// rows the blocks of a cluster, split the summed index.  A warp multiplies the
// rows as the 16-row operand of mma.m16n8k16 with the tokens as its columns.
// The order of the summed index inside a product is free as long as both
// operands share it: a lane's operand values are taken from 8 neighbouring ones
// (16 bytes) of a row, so that every load is a whole vector and no shared memory
// or shuffle stands between memory and the product.  The warps' sums meet in
// shared memory and the blocks' over the cluster, in a fixed order.
//
// With SwiGLU rows g and g + 8 of a product are gate and up of one channel.
//
// One token and 256 rows of 7,168: 3.4 us, mostly the launch and the two
// reductions.  Eight tokens and 4,096 rows of 7,168: 10.5 us, 5.6 TB/s; 7,168 rows:
// 17 us, 6.0 TB/s.  The weights are asked for from L2 while the preceding kernel
// ends.  Beyond EP_LINEAR_FEW_TOKENS the tcgen05 kernel takes less (32 tokens, 7,168
// rows of 7,168: 25.9 here, 25.5 us there; 256 rows: 5.5 here, 10.8 us there).
//
// Below it: what follows products whose summed index the tcgen05 kernel split into
// parts, passes over the parts' fp32 sums.
#include "ep_products.cuh"
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kChunk = 32;  // of the summed index: two products
constexpr int kPrefetch = 8192;  // bytes of a row and warp that are asked for from L2 ahead
constexpr int kSumChunks = 16;   // 512 values, after which the products' sums, which truncate, are added up, rounded
// A bf16 output, whose rounding hides more, may have whole sums of 16,384 values per warp.
constexpr int64_t kWholeWidth = 16384 * kWarps;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Up to 8 * NT tokens, RT * 16 rows of weights per block at most: `per` output
// channels.  CUT: a warp's sum ends every kSumChunks.
template <int NT, int RT, bool GATED, bool AHEAD, bool CUT>
__global__ void __launch_bounds__(kThreads, RT == 1 && NT < 4 && !AHEAD ? 3 : 2)
linear_few_kernel(const __grid_constant__ ProductArgs p, int cluster, int per) {
    constexpr int kRows = RT * 16, kTokens = NT * 8;
    constexpr int kUnroll = RT == 1 && NT < 4 ? 4 : 2;
    alignas(16) __shared__ float part[kWarps][kTokens][kRows + 1];
    __shared__ float total[kTokens][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t group = blockIdx.x / cluster;
    const int M = (int)p.rows;
    const int64_t K = p.K, channels = GATED ? p.N / 2 : p.N;
    const int64_t n0 = group * per;  // first output channel
    const uint16_t* w[RT][2];
    bool live[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = GATED ? r * 8 + g : r * 16 + h * 8 + g;
            const int64_t n = n0 + c;
            live[r][h] = c < per && n < channels;
            w[r][h] = p.b + ((GATED && h ? channels : 0) + n) * K + 8 * t;
        }
    const uint16_t* x[NT];
    bool token[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        token[j] = j * 8 + g < M;
        x[j] = p.a + (int64_t)(j * 8 + g) * K + 8 * t;
    }
    const int chunks = (int)((K + kChunk - 1) / kChunk), slices = cluster * kWarps;
    const int share = (chunks + slices - 1) / slices;
    const int c0 = min(chunks, (rank * kWarps + warp) * share), c1 = min(chunks, c0 + share);
    // The weights are asked for from L2 while the preceding kernel ends; nothing
    // is read before the wait.
    if (c0 < c1 && t < 2 * RT) {
        const int64_t first = (int64_t)c0 * kChunk, left = K - first, share_k = (int64_t)(c1 - c0) * kChunk;
        const uint32_t bytes = (uint32_t)min(min(left, share_k) * 2, (int64_t)kPrefetch);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (t == 2 * r + h && live[r][h])
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(w[r][h] - 8 * t + first), "r"(bytes)
                                 : "memory");
    }
    pdl_wait();
    pdl_trigger();
    // The products' sums are added up in registers, or, where four times two products
    // per step leave none (25.9 us would be 31.9), in the warp's share of `part`, a
    // lane's 16 bytes beside the next one's.
    constexpr bool kInRegisters = NT * RT < 8;
    static_assert(kTokens * (kRows + 1) >= RT * NT * 4 * 32 && kTokens * (kRows + 1) % 4 == 0, "");
    float4* kept = reinterpret_cast<float4*>(part[warp][0]) + lane;
    bool any = false;
    float acc[RT][NT][4] = {}, sums[RT][NT][4] = {};
    auto add_up = [&]() {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (!kInRegisters) {
                    float4& at = kept[(r * NT + j) * 32];
                    float4 v = any ? at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v.x += acc[r][j][0], v.y += acc[r][j][1], v.z += acc[r][j][2], v.w += acc[r][j][3];
                    at = v;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kInRegisters) sums[r][j][i] += acc[r][j][i];
                    acc[r][j][i] = 0.0f;
                }
            }
        any = true;
    };
    struct Operands {
        uint4 a[kUnroll][RT][2], b[kUnroll][NT];
    };
    auto load = [&](Operands& o, int c) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t k = (int64_t)(c + u) * kChunk;
            const bool in = c + u < c1 && k + 8 * t < K;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    o.a[u][r][h] = in && live[r][h] ? ld_stream_v4(w[r][h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                o.b[u][j] = in && token[j] ? __ldg(reinterpret_cast<const uint4*>(x[j] + k)) : make_uint4(0, 0, 0, 0);
        }
    };
    auto multiply = [&](const Operands& o) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 &lo = o.a[u][r][0], &hi = o.a[u][r][1], &v = o.b[u][j];
                    mma_bf16(acc[r][j], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
                    mma_bf16(acc[r][j], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
                }
    };
    if (AHEAD) {  // the next step's operands are on their way while one is multiplied
        Operands even, odd;
        load(even, c0);
        for (int c = c0; c < c1; c += 2 * kUnroll) {
            load(odd, c + kUnroll);
            multiply(even);
            load(even, c + 2 * kUnroll);
            multiply(odd);
            if ((c - c0) % kSumChunks == kSumChunks - 2 * kUnroll) add_up();
        }
    } else {
        const int every = CUT ? kSumChunks : chunks;
        for (int first = c0; first < c1; first += every) {
            if (CUT && first > c0) add_up();
            const int end = CUT ? min(c1, first + every) : c1;
            for (int c = first; c < end; c += kUnroll) {
                Operands o;
                load(o, c);
                multiply(o);
            }
        }
    }
    if (CUT && !kInRegisters && any) {
        add_up();
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float4 v = kept[(r * NT + j) * 32];
                acc[r][j][0] = v.x, acc[r][j][1] = v.y, acc[r][j][2] = v.z, acc[r][j][3] = v.w;
            }
        __syncwarp();  // the same places get the sums by token and row
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][j * 8 + 2 * t + (i & 1)][r * 16 + g + (i >> 1) * 8] = sums[r][j][i] + acc[r][j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kTokens; i += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += part[k][i / kRows][i % kRows];
        total[i / kRows][i % kRows] = s;
    }
    if (cluster > 1)
        cluster_sync();
    else
        __syncthreads();
    // the blocks take the tokens in turn
    auto sum = [&](int m, int row) {
        if (cluster == 1) return total[m][row];
        float s = 0.0f;
        for (int r = 0; r < cluster; ++r) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v)
                         : "r"(cluster_addr(smem_addr(&total[m][row]), r))
                         : "memory");
            s += v;
        }
        return s;
    };
    constexpr int kOut = GATED ? RT * 8 : kRows;
    for (int i = threadIdx.x; i < kOut * kTokens; i += kThreads) {
        const int m = i / kOut, c = i % kOut;
        const int64_t n = n0 + c;
        if (m >= M || c >= per || n >= channels || m % cluster != rank) continue;
        const int row = GATED ? (c >> 3) * 16 + (c & 7) : c;
        float v = sum(m, row);
        if (p.bias) v += load_typed(p.bias, p.bias_type, n);
        if (GATED) {
            float u = sum(m, row + 8);
            if (p.bias) u += load_typed(p.bias, p.bias_type, channels + n);
            if (p.z) {
                p.z[(int64_t)m * p.N + n] = bf16_bits(v);
                p.z[(int64_t)m * p.N + channels + n] = bf16_bits(u);
            }
            v = swiglu(v, u);
        } else {
            if (p.z) p.z[(int64_t)m * p.N + n] = bf16_bits(v);
            v = activate(v, p.activation);
        }
        const int64_t at = (int64_t)m * channels + n;
        if (p.out_type == EP_TYPE_F32) {
            if (p.residual) v += static_cast<const float*>(p.residual)[at];
            static_cast<float*>(p.out)[at] = v;
        } else {
            if (p.residual) v += bf16_value(static_cast<const uint16_t*>(p.residual)[at]);
            static_cast<uint16_t*>(p.out)[at] = bf16_bits(v);
        }
    }
    if (cluster > 1) cluster_sync();  // the other blocks' sums stay until they are read
}

// Four elements of a weight gradient whose rows were summed in parts.
__global__ void __launch_bounds__(256)
weight_finish_kernel(const float4* __restrict__ parts, int splits, int64_t vecs, const void* add, void* out, int type) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= vecs) return;
    float4 s = parts[i];
    for (int k = 1; k < splits; ++k) {
        const float4 v = parts[k * vecs + i];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    if (type == EP_TYPE_F32) {
        if (add) {
            const float4 a = static_cast<const float4*>(add)[i];
            s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
        }
        static_cast<float4*>(out)[i] = s;
    } else {
        if (add) {
            const uint2 a = static_cast<const uint2*>(add)[i];
            s.x += bf16lo_to_f32(a.x), s.y += bf16hi_to_f32(a.x);
            s.z += bf16lo_to_f32(a.y), s.w += bf16hi_to_f32(a.y);
        }
        static_cast<uint2*>(out)[i] = make_uint2(pack_bf16x2_rn(s.x, s.y), pack_bf16x2_rn(s.z, s.w));
    }
}

template <int NT, int RT, bool AHEAD>
cudaError_t launch(const ProductArgs& p, int sms, cudaStream_t stream) {
    const bool gated = p.activation == EP_ACT_SWIGLU;
    const int64_t channels = gated ? p.N / 2 : p.N, most = gated ? RT * 8 : RT * 16;
    // As few rounds over the SMs as `most` channels per block allow, and then as
    // many channels per block as the rounds need: equal shares.  Where one
    // round is not full, clusters, while a warp's share of the summed index is
    // four steps.
    const int64_t rounds = (channels + most * sms - 1) / (most * sms);
    const int64_t per = (channels + rounds * sms - 1) / (rounds * sms);
    const int64_t blocks = (channels + (rounds > 1 ? per : most) - 1) / (rounds > 1 ? per : most);
    int cluster = 1;
    while (cluster < 8 && blocks * cluster <= sms && p.K >= kChunk * kWarps * cluster * 4) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    // Adding up costs time where it goes through shared memory (32 tokens, 6,000 rows of
    // 16,384: 50 us, with it 52; 7,168 of 2,048: 10.9 and 11.3), and nothing elsewhere.
    constexpr bool kAlways = NT * RT < 8;
    const bool cut = kAlways || p.out_type == EP_TYPE_F32 || p.K > kWholeWidth;
    auto kernel = gated ? (cut ? linear_few_kernel<NT, RT, true, AHEAD, true> : linear_few_kernel<NT, RT, true, AHEAD, kAlways>)
                        : (cut ? linear_few_kernel<NT, RT, false, AHEAD, true> : linear_few_kernel<NT, RT, false, AHEAD, kAlways>);
    return cudaLaunchKernelEx(&cfg, kernel, p, cluster, (int)(rounds > 1 ? per : most));
}

// A thread's four channels of a token.
template <bool GATED>
__global__ void __launch_bounds__(256)
linear_finish_kernel(const __grid_constant__ ProductArgs p, const float* __restrict__ parts, int splits) {
    pdl_wait();
    pdl_trigger();
    const int64_t channels = GATED ? p.N / 2 : p.N, vecs = channels / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.rows * vecs) return;
    const int64_t m = i / vecs, n = (i - m * vecs) * 4;
    constexpr int H = GATED ? 2 : 1;
    float f[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const float4* src = reinterpret_cast<const float4*>(parts + m * p.N + h * channels + n);
        const int64_t step = p.rows * p.N / 4;
        float4 s = src[0];
        for (int k = 1; k < splits; ++k) {
            const float4 v = src[k * step];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        f[h][0] = s.x, f[h][1] = s.y, f[h][2] = s.z, f[h][3] = s.w;
        if (p.bias) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[h][j] += load_typed(p.bias, p.bias_type, h * channels + n + j);
        }
        if (p.z)
            *reinterpret_cast<uint2*>(p.z + m * p.N + h * channels + n) =
                make_uint2(pack_bf16x2_rn(f[h][0], f[h][1]), pack_bf16x2_rn(f[h][2], f[h][3]));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[0][j] = GATED ? swiglu(f[0][j], f[H - 1][j]) : activate(f[0][j], p.activation);
    const int64_t at = m * channels + n;
    if (p.out_type == EP_TYPE_F32) {
        if (p.residual) {
            const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + at);
            f[0][0] += r.x, f[0][1] += r.y, f[0][2] += r.z, f[0][3] += r.w;
        }
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(f[0][0], f[0][1], f[0][2], f[0][3]);
    } else {
        if (p.residual) {
            const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) + at);
            f[0][0] += bf16lo_to_f32(r.x), f[0][1] += bf16hi_to_f32(r.x);
            f[0][2] += bf16lo_to_f32(r.y), f[0][3] += bf16hi_to_f32(r.y);
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16x2_rn(f[0][0], f[0][1]), pack_bf16x2_rn(f[0][2], f[0][3]));
    }
}

}  // namespace

cudaError_t launch_linear_few(const ProductArgs& p, cudaStream_t stream) {
    static std::atomic<int> sm_cache[64];
    int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    if (sms < 1) sms = 1;
    // More tokens than the 8 columns of a product: their loads weigh as much as the
    // weights', and 32 rows per block share them.  With up to 32 tokens 16 rows
    // are better as long as they come in two rounds (256 rows of 7,168: 5.5
    // against 6.7 us; 7,168 rows of 2,048: 13.1 against 10.7).
    if (p.rows > 16)
        return p.N <= 2 * 16 * (int64_t)sms ? launch<4, 1, false>(p, sms, stream) : launch<4, 2, false>(p, sms, stream);
    if (p.rows > 8) return launch<2, 2, false>(p, sms, stream);
    // A warp with four steps or more of the summed index loads a step ahead (two
    // blocks per SM): 4,096 rows of 7,168: 10.5 against 12.3 us; with less to do
    // the third block per SM gives more (7,168 rows of 2,048: 5.8 against 8.3 us).
    if (p.K < 4 * 4 * kChunk * kWarps) return launch<1, 1, false>(p, sms, stream);
    return p.N <= 2 * 16 * (int64_t)sms ? launch<1, 1, true>(p, sms, stream) : launch<1, 2, true>(p, sms, stream);
}

cudaError_t launch_weight_finish(const float* parts, int splits, int64_t count, const void* add, void* out, int type,
                                 cudaStream_t stream) {
    return launch_pdl(weight_finish_kernel, dim3((unsigned)((count / 4 + 255) / 256)), dim3(256), 0, stream,
                      reinterpret_cast<const float4*>(parts), splits, count / 4, add, out, type);
}

cudaError_t launch_linear_finish(const ProductArgs& p, const float* parts, int splits, cudaStream_t stream) {
    const bool gated = p.activation == EP_ACT_SWIGLU;
    const int64_t threads = p.rows * (gated ? p.N / 2 : p.N) / 4;
    auto kernel = gated ? linear_finish_kernel<true> : linear_finish_kernel<false>;
    return launch_pdl(kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, p, parts, splits);
}

}  // namespace ep
