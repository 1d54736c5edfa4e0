// ep_moe_few.cu -- the whole expert layer for a few tokens in two kernels:
//   up    x's FP8 cast, the gate and up products of every routed expert,
//         SwiGLU and the FP8 cast of h, per (expert, 128 columns of I)
//   down  the second products and the weighted sum over a token's experts
// for tokens whose experts' weights are nearly all read for one to eight rows
// each, so that the time is that of streaming the weights once.
//
// Mathematics: each weight tile of 16 rows is the A operand of an e4m3
// mma.m16n8k32 and up to 8 of the expert's tokens are its 8 columns (a "group":
// an expert with more tokens is several groups, whose later readings of the
// weights come from L2).  Four MMAs make one 128-channel block, whose sum is
// then scaled by a_scale * w_scale and added in fp32.  The order of k inside
// a block is free as long as both operands agree on it, so that each lane
// loads 32 consecutive bytes of two weight rows straight into its A
// registers, and the same 32 bytes of its token into B.
//
// up: a tile holds 8 gate rows and the 8 up rows of the same columns, so that
// a lane's accumulators are the gate and up values of the same h.  A block's
// 16 warps take the 16 tiles of 128 columns; the FP8 cast of h needs only the
// warps' maxima.  With few items the 128 columns are shared by a cluster of C
// blocks, each splitting K over C warps per tile; the maxima meet in
// distributed shared memory.
// down: a block owns 16 output channels for all groups; its warps take equal
// shares of the (group, 128-channel block) sequence, add weighted results per
// token in shared memory of their own and the block adds the warps' sums in
// order, so that the result never depends on timing.
#include <cooperative_groups.h>
#include <stddef.h>

#include "ep_internal.cuh"

namespace ep {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 8;    // tokens per group: columns of one MMA
constexpr int kDepth = 4;   // 128-channel blocks of weights that a warp has in flight
constexpr int kMaxPairs = EP_MOE_FEW_MAX_TOKENS * EP_MAX_TOPK;

// The groups of a route, built by every block for itself.
struct Groups {
    int count;
    uint16_t expert[kMaxPairs];  // per group
    uint16_t first[kMaxPairs];   // its first entry of `pair`, and their number
    uint8_t size[kMaxPairs];
    uint16_t pair[kMaxPairs];    // pairs t * k + j ordered by expert, then by pair
    uint16_t start[EP_MAX_EXPERTS];
    uint16_t seen[EP_MAX_EXPERTS];
};

// Fills `g` (shared); all threads of the block call it.  One warp does the
// work: at most 2,048 ids, 32 at a time.
__device__ void build_groups(Groups& g, const int32_t* __restrict__ topk_idx, int P, int E,
                             uint32_t* status, bool report) {
    for (int e = threadIdx.x; e < E; e += kThreads) g.start[e] = g.seen[e] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        bool bad = false;
        for (int p0 = 0; p0 < P; p0 += 32) {  // pairs per expert
            const int e = p0 + lane < P ? __ldg(topk_idx + p0 + lane) : -1;
            const bool live = e >= 0 && e < E;
            bad |= !live && e != -1;
            const unsigned peers = __match_any_sync(kFullMask, live ? e : -1);
            if (live && (peers & lanemask_lt()) == 0) g.start[e] += (uint16_t)__popc(peers);
            __syncwarp();
        }
        if (report) warp_flag(status, bad, EP_FLAG_BAD_EXPERT);
        int pairs = 0, groups = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {  // scans over the experts
            const int e = e0 + lane;
            const int n = e < E ? g.start[e] : 0;
            const int m = (n + kCols - 1) / kCols;
            int ps = n, gs = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(kFullMask, ps, o), b = __shfl_up_sync(kFullMask, gs, o);
                if (lane >= o) {
                    ps += a;
                    gs += b;
                }
            }
            const int first = pairs + ps - n;
            for (int i = 0; i < m; ++i) {
                const int at = groups + gs - m + i;
                g.expert[at] = (uint16_t)e;
                g.first[at] = (uint16_t)(first + i * kCols);
                g.size[at] = (uint8_t)min(kCols, n - i * kCols);
            }
            if (e < E) g.start[e] = (uint16_t)first;
            pairs += __shfl_sync(kFullMask, ps, 31);
            groups += __shfl_sync(kFullMask, gs, 31);
        }
        if (lane == 0) g.count = groups;
        __syncwarp();
        for (int p0 = 0; p0 < P; p0 += 32) {  // the pairs in expert order
            const int e = p0 + lane < P ? __ldg(topk_idx + p0 + lane) : -1;
            const bool live = e >= 0 && e < E;
            const unsigned peers = __match_any_sync(kFullMask, live ? e : -1);
            const int before = __popc(peers & lanemask_lt());
            int at = 0;
            if (live) at = g.start[e] + g.seen[e] + before;
            __syncwarp();
            if (live) {
                g.pair[at] = (uint16_t)(p0 + lane);
                if (before == 0) g.seen[e] += (uint16_t)__popc(peers);
            }
            __syncwarp();
        }
    }
    __syncthreads();
}

// p += A (16 x 32, e4m3, row) * B (32 x 8, e4m3, column), fp32.
__device__ __forceinline__ void mma_e4m3(float (&p)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(p[0]), "+f"(p[1]), "+f"(p[2]), "+f"(p[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One 128-channel block: lo / hi are a lane's 32 bytes of weight rows g and
// g + 8, b those of its column.
__device__ __forceinline__ void block_product(float (&p)[4], const Vec32& lo, const Vec32& hi,
                                              const uint4& b0, const uint4& b1) {
    p[0] = p[1] = p[2] = p[3] = 0.0f;
    mma_e4m3(p, lo.lo.x, hi.lo.x, lo.lo.y, hi.lo.y, b0.x, b0.y);
    mma_e4m3(p, lo.lo.z, hi.lo.z, lo.lo.w, hi.lo.w, b0.z, b0.w);
    mma_e4m3(p, lo.hi.x, hi.hi.x, lo.hi.y, hi.hi.y, b1.x, b1.y);
    mma_e4m3(p, lo.hi.z, hi.hi.z, lo.hi.w, hi.hi.w, b1.z, b1.w);
}

struct Stage {  // one block of weights in flight
    Vec32 lo, hi;
    float s_lo, s_hi;
};

// ---- up -------------------------------------------------------------------

struct UpShared {
    Groups g;
    float amax[2][kWarps][kCols];     // [item parity][rank * tiles + tile][column]
    alignas(16) float part[kWarps][32][4];  // partial sums of the warps that share a tile
};

static_assert(offsetof(UpShared, part) % 16 == 0 && offsetof(UpShared, amax) % 4 == 0, "");

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
few_up_kernel(const uint16_t* __restrict__ x, int T, int H, int k,
              const int32_t* __restrict__ topk_idx, const uint8_t* __restrict__ w13,
              const float* __restrict__ s13, int I, int E, uint8_t* __restrict__ hq,
              float* __restrict__ hs, uint32_t* __restrict__ status) {
    namespace cg = cooperative_groups;
    constexpr int kTiles = kWarps / C;  // M tiles of a block: 8 columns of I each
    extern __shared__ __align__(16) uint8_t smem[];
    UpShared& sh = *reinterpret_cast<UpShared*>(smem);
    const int stride = H + 16;  // 16 bytes of padding: a quarter-warp's rows meet all banks
    uint8_t* xq = smem + (sizeof(UpShared) + 15) / 16 * 16;
    float* xs = reinterpret_cast<float*>(xq + kCols * stride);
    const int nk = H / 128, nb = I / 128;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = lane >> 2, q4 = lane & 3;
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
    const int worker = blockIdx.x / C, workers = gridDim.x / C;
    const int tile = warp % kTiles, ks = warp / kTiles;

    pdl_wait();
    pdl_trigger();
    build_groups(sh.g, topk_idx, T * k, E, status, blockIdx.x == 0);
    const int items = sh.g.count * nb;  // (group, block of 128 columns)
    const int mine = worker < items ? (items - worker + workers - 1) / workers : 0;
    const int steps = (nk + C - 1) / C;  // blocks of K per warp and item
    const int total = mine * steps;

    // load side
    int l_item = worker, l_step = 0;
    const uint8_t* l_w = nullptr;
    const float* l_s = nullptr;
    auto load = [&](Stage& st, int s) {
        if (s >= total) return;
        if (l_step == 0) {
            const int e = sh.g.expert[l_item / nb], b = l_item % nb;
            l_w = w13 + ((int64_t)e * 2 * I + b * 128 + (rank * kTiles + tile) * 8 + row) * H + q4 * 32;
            l_s = s13 + ((int64_t)e * 2 * nb + b) * nk;
        }
        const int kb = ks * steps + l_step;
        if (kb < nk) {
            st.lo = ld_stream_v8(l_w + kb * 128);
            st.hi = ld_stream_v8(l_w + (int64_t)I * H + kb * 128);
            st.s_lo = __ldg(l_s + kb);
            st.s_hi = __ldg(l_s + (int64_t)nb * nk + kb);
        }
        if (++l_step == steps) {
            l_step = 0;
            l_item += workers;
        }
    };
    Stage st[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(st[d], d);

    int item = worker, step = 0, have = -1;  // `have`: the group whose x is in shared memory
    int parity = 0;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < total; s0 += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (s0 + d >= total) break;  // block-uniform
            const int grp = item / nb, n = sh.g.size[grp];
            if (step == 0 && grp != have) {
                __syncthreads();  // the previous group's reads are done
                // one warp per token: the cast of ep_dispatch_fp8; unused columns are zero
                if (warp < kCols) {
                    const int t = warp < n ? sh.g.pair[sh.g.first[grp] + warp] / k : 0;
                    const uint16_t* src = x + (int64_t)t * H;
                    for (int c0 = 0; c0 < H; c0 += 1024) {
                        uint4 a[2], b[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int c = c0 + u * 512 + lane * 16;
                            a[u] = b[u] = make_uint4(0, 0, 0, 0);
                            if (warp < n && c < H) {
                                a[u] = __ldg(reinterpret_cast<const uint4*>(src + c));
                                b[u] = __ldg(reinterpret_cast<const uint4*>(src + c + 8));
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int c = c0 + u * 512 + lane * 16;
                            const Fp8Group f = quantize16(a[u], b[u]);
                            if (c < H) {
                                *reinterpret_cast<uint4*>(xq + warp * stride + c) = f.q;
                                if ((lane & 7) == 0) xs[warp * nk + (c >> 7)] = f.sf;
                            }
                        }
                    }
                }
                have = grp;
                __syncthreads();
            }
            const int kb = ks * steps + step;
            if (kb < nk) {
                const uint4* bp = reinterpret_cast<const uint4*>(xq + row * stride + kb * 128 + q4 * 32);
                float p[4];
                block_product(p, st[d].lo, st[d].hi, bp[0], bp[1]);
                const float x0 = xs[(2 * q4) * nk + kb], x1 = xs[(2 * q4 + 1) * nk + kb];
                acc[0] = __fmaf_rn(p[0], __fmul_rn(x0, st[d].s_lo), acc[0]);
                acc[1] = __fmaf_rn(p[1], __fmul_rn(x1, st[d].s_lo), acc[1]);
                acc[2] = __fmaf_rn(p[2], __fmul_rn(x0, st[d].s_hi), acc[2]);
                acc[3] = __fmaf_rn(p[3], __fmul_rn(x1, st[d].s_hi), acc[3]);
            }
            load(st[d], s0 + d + kDepth);
            if (++step < steps) continue;
            // the item is done
            if (C > 1) {
                *reinterpret_cast<float4*>(sh.part[warp][lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                __syncthreads();
                if (ks == 0) {
#pragma unroll
                    for (int i = 1; i < C; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(sh.part[i * kTiles + tile][lane]);
                        acc[0] = __fadd_rn(acc[0], v.x);
                        acc[1] = __fadd_rn(acc[1], v.y);
                        acc[2] = __fadd_rn(acc[2], v.z);
                        acc[3] = __fadd_rn(acc[3], v.w);
                    }
                }
            }
            float h[2], m[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                h[i] = swiglu(acc[i], acc[2 + i]);
                m[i] = fabsf(h[i]);
                m[i] = fmaxf(m[i], __shfl_xor_sync(kFullMask, m[i], 4));
                m[i] = fmaxf(m[i], __shfl_xor_sync(kFullMask, m[i], 8));
                m[i] = fmaxf(m[i], __shfl_xor_sync(kFullMask, m[i], 16));
            }
            const int slot = rank * kTiles + tile;
            if (ks == 0 && lane < 4) {
                if (C == 1) {
                    sh.amax[parity][slot][2 * lane] = m[0];
                    sh.amax[parity][slot][2 * lane + 1] = m[1];
                } else {
                    for (int r = 0; r < C; ++r) {
                        float* to = cg::this_cluster().map_shared_rank(&sh.amax[parity][slot][2 * lane], r);
                        to[0] = m[0];
                        to[1] = m[1];
                    }
                }
            }
            if (C == 1) __syncthreads();
            else cg::this_cluster().sync();
            if (ks == 0) {
                const int b = item % nb;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 2 * q4 + i;
                    float a = 1e-4f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) a = fmaxf(a, sh.amax[parity][w][col]);
                    if (col < n) {
                        const int pair = sh.g.pair[sh.g.first[grp] + col];
                        const float inv = __fdiv_rn(448.0f, a);
                        hq[(int64_t)pair * I + b * 128 + slot * 8 + row] =
                            (uint8_t)cvt_e4m3x2_rn_sat(__fmul_rn(h[i], inv), 0.0f);
                        if (slot == 0 && row == 0) hs[(int64_t)pair * nb + b] = __fdiv_rn(a, 448.0f);
                    }
                }
            }
            parity ^= 1;  // the next item's maxima go to the other buffer
            acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
            step = 0;
            item += workers;
        }
    }
    // a block of a cluster must not exit while another still writes its maxima:
    // the last item's cluster barrier came after those writes
}

// ---- down -----------------------------------------------------------------

__global__ void __launch_bounds__(kThreads, 1)
few_down_kernel(const uint8_t* __restrict__ hq, const float* __restrict__ hs, int T, int H, int k,
                const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w,
                const uint8_t* __restrict__ w2, const float* __restrict__ s2, int I, int E,
                uint16_t* __restrict__ out) {
    extern __shared__ __align__(16) uint8_t smem[];
    Groups& g = *reinterpret_cast<Groups*>(smem);
    // [parity][warp][token][16 channels]
    float* slabs = reinterpret_cast<float*>(smem + (sizeof(Groups) + 15) / 16 * 16);
    const int nk = I / 128;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = lane >> 2, q4 = lane & 3;
    // The route and the weights are older than the up kernel, which let this
    // one start only after all earlier work had completed.
    build_groups(g, topk_idx, T * k, E, nullptr, false);
    const int tiles = H / 16;
    const int mine = (int)blockIdx.x < tiles ? (tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const int units = g.count * nk;  // (group, block of K), the same for every tile
    const int u0 = (int)((int64_t)units * warp / kWarps), u1 = (int)((int64_t)units * (warp + 1) / kWarps);
    const int per = u1 - u0;
    const int total = mine * per;

    int l_tile = blockIdx.x, l_u = u0, l_grp = u0 / nk, l_kb = u0 % nk;
    auto load = [&](Stage& st, int s) {
        if (s >= total) return;
        const int e = g.expert[l_grp];
        const uint8_t* w = w2 + ((int64_t)e * H + l_tile * 16 + row) * I + l_kb * 128 + q4 * 32;
        st.lo = ld_stream_v8(w);
        st.hi = ld_stream_v8(w + 8 * (int64_t)I);
        st.s_lo = __ldg(s2 + ((int64_t)e * (H / 128) + l_tile / 8) * nk + l_kb);
        ++l_u;
        if (++l_kb == nk) {
            l_kb = 0;
            ++l_grp;
        }
        if (l_u == u1) {
            l_u = u0;
            l_grp = u0 / nk;
            l_kb = u0 % nk;
            l_tile += gridDim.x;
        }
    };
    Stage st[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(st[d], d);
    const int slab_n = T * 16;
    for (int i = threadIdx.x; i < 2 * kWarps * slab_n; i += kThreads) slabs[i] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int s = 0;
    for (int i = 0; i < mine; ++i) {
        const int tile = blockIdx.x + i * gridDim.x;
        float* slab = slabs + ((i & 1) * kWarps + warp) * slab_n;
        int grp = u0 / nk, kb = u0 % nk;
        for (int u = u0; u < u1; u += 1, ++s) {
            const int n = g.size[grp], first = g.first[grp];
            uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
            if (row < n) {
                const uint4* bp = reinterpret_cast<const uint4*>(
                    hq + (int64_t)g.pair[first + row] * I + kb * 128 + q4 * 32);
                b0 = bp[0];
                b1 = bp[1];
            }
            float x0 = 0.0f, x1 = 0.0f;
            if (2 * q4 < n) x0 = hs[(int64_t)g.pair[first + 2 * q4] * nk + kb];
            if (2 * q4 + 1 < n) x1 = hs[(int64_t)g.pair[first + 2 * q4 + 1] * nk + kb];
            Stage cur;
#pragma unroll
            for (int d = 0; d < kDepth; ++d)
                if (s % kDepth == d) {
                    cur = st[d];
                    load(st[d], s + kDepth);
                }
            float p[4];
            block_product(p, cur.lo, cur.hi, b0, b1);
            acc[0] = __fmaf_rn(p[0], __fmul_rn(x0, cur.s_lo), acc[0]);
            acc[1] = __fmaf_rn(p[1], __fmul_rn(x1, cur.s_lo), acc[1]);
            acc[2] = __fmaf_rn(p[2], __fmul_rn(x0, cur.s_lo), acc[2]);
            acc[3] = __fmaf_rn(p[3], __fmul_rn(x1, cur.s_lo), acc[3]);
            if (++kb == nk || u + 1 == u1) {
                // this warp's share of the group: weight it into its tokens, one
                // column after another (a token may hold an expert twice)
                for (int c = 0; c < n; ++c) {
                    if (c / 2 == q4) {
                        const int pair = g.pair[first + c];
                        const float wt = __ldg(topk_w + pair);
                        float* o = slab + pair / k * 16 + row;
                        o[0] = __fmaf_rn(wt, acc[c & 1], o[0]);
                        o[8] = __fmaf_rn(wt, acc[2 + (c & 1)], o[8]);
                    }
                    __syncwarp();
                }
                acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
                kb = 0;
                ++grp;
            }
        }
        __syncthreads();
        // add the warps' sums in order, clear them for the tile after the next
        float* all = slabs + (i & 1) * kWarps * slab_n;
        for (int v = threadIdx.x; v < slab_n / 2; v += kThreads) {
            float a = 0.0f, b = 0.0f;
            for (int w = 0; w < kWarps; ++w) {
                float2* p2 = reinterpret_cast<float2*>(all + w * slab_n) + v;
                const float2 f = *p2;
                a = __fadd_rn(a, f.x);
                b = __fadd_rn(b, f.y);
                *p2 = make_float2(0.0f, 0.0f);
            }
            const int t = v / 8, c = v % 8 * 2;
            *reinterpret_cast<uint32_t*>(out + (int64_t)t * H + tile * 16 + c) = pack_bf16x2_rn(a, b);
        }
        // the slabs of this parity are next touched two tiles on, after another barrier
    }
}

size_t up_smem(int H) {
    return (sizeof(UpShared) + 15) / 16 * 16 + (size_t)kCols * (H + 16) + (size_t)kCols * (H / 128) * 4;
}
size_t down_smem(int T) { return (sizeof(Groups) + 15) / 16 * 16 + (size_t)2 * kWarps * T * 16 * 4; }

template <int C>
cudaError_t launch_up(int blocks, const void* x, int T, int H, int k, const int32_t* topk_idx,
                      const uint8_t* w13, const float* s13, int I, int E, uint8_t* hq, float* hs,
                      uint32_t* status, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    cudaError_t err = raise_smem_limit(few_up_kernel<C>, up_smem(EP_MOE_FEW_MAX_WIDTH), configured);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = up_smem(H);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {C, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, few_up_kernel<C>, static_cast<const uint16_t*>(x), T, H, k,
                              topk_idx, w13, s13, I, E, hq, hs, status);
}

}  // namespace

size_t moe_few_h_bytes(int64_t T, int k, int I) { return ((size_t)T * k * I + 255) / 256 * 256; }

cudaError_t launch_moe_few(const void* x, int T, int H, int k, const int32_t* topk_idx,
                           const float* topk_w, const uint8_t* w13, const float* s13,
                           const uint8_t* w2, const float* s2, int I, int E, void* out,
                           uint32_t* status, void* workspace, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    static std::atomic<int> sm_cache[64];
    int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    if (sms <= 0) sms = 1;
    uint8_t* hq = static_cast<uint8_t*>(workspace);
    float* hs = reinterpret_cast<float*>(hq + moe_few_h_bytes(T, k, I));
    // Blocks per 128 columns: the C that leaves the fewest idle blocks in the
    // last round of items (at most one expert per pair), 1 where equal.
    const int64_t items = (int64_t)(T * k < E ? T * k : E) * (I / 128);
    int C = 1;
    double best = 1e30;
    for (int c = 1; c <= 4; c *= 2) {
        const double rounds = (double)((items * c + sms - 1) / sms) / c;
        if (rounds < best * 0.999) {
            best = rounds;
            C = c;
        }
    }
    const int blocks = (int)(items * C < sms ? items * C : sms / C * C);
    cudaError_t err =
        C == 1   ? launch_up<1>(blocks, x, T, H, k, topk_idx, w13, s13, I, E, hq, hs, status, stream)
        : C == 2 ? launch_up<2>(blocks, x, T, H, k, topk_idx, w13, s13, I, E, hq, hs, status, stream)
                 : launch_up<4>(blocks, x, T, H, k, topk_idx, w13, s13, I, E, hq, hs, status, stream);
    if (err != cudaSuccess) return err;
    static std::atomic<uint64_t> configured{0};
    err = raise_smem_limit(few_down_kernel, down_smem(EP_MOE_FEW_MAX_TOKENS), configured);
    if (err != cudaSuccess) return err;
    const int tiles = H / 16;
    return launch_pdl(few_down_kernel, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kThreads),
                      down_smem(T), stream, hq, hs, T, H, k, topk_idx, topk_w, w2, s2, I, E,
                      static_cast<uint16_t*>(out));
}

}  // namespace ep
