// ep_group_gemm.cu -- the experts' products over a dispatched FP8 buffer.
// Row r of expert e, with K channels in blocks of 128 (b = k / 128):
//     y[r, n] = sum_b a_scale[r, b] * w_scale[e, n/128, b]
//                     * sum_{k in b} a[r, k] * w[e, n, k]
// e4m3 codes, the block's sum and the sum over blocks in fp32.  Two forms:
//   plain   out[r, n] = bf16_rne(y[r, n])
//   swiglu  the expert's rows n < I are the gate, I <= n < 2I the up
//           projection: h = gate / (1 + exp(-gate)) * up in fp32, then the
//           e4m3 cast of ep_dispatch_fp8 per row and 128 channels of h.
//
// A tile is 128 rows of one expert by 256 weight rows (swiglu: 128 gate rows
// and the 128 up rows of the same channels).  The scales are fp32 and differ
// per row and block of 128, so that the tensor core cannot apply them: it
// makes each block's sum (four tcgen05.mma of K = 32 into one of two TMEM
// buffers), and eight warps read that sum back, scale it and add it into
// fp32 registers while the next block's MMAs run.  A TMEM lane is a row, so
// the row's scale is one value per thread.
//
// One persistent block per SM: warp 0 issues the TMA loads (128-byte swizzle,
// four stages), warp 1 the MMAs, warps 4-11 scale, add and write the output.
// The block is launched with 168 registers a thread; the first warpgroup
// leaves 112 of them to the other two, which need 128 for the sums alone.
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = 128;
constexpr int kStages = 4;
constexpr int kABytes = kTileM * kBlockK, kBBytes = kTileN * kBlockK;
constexpr int kARows = 32;  // rows per TMA box of A: rows past the segment's end are not read
constexpr int kThreads = 384;
constexpr int kIssueRegs = 56, kAddRegs = 224;  // 128 * 56 + 256 * 224 = 384 * 168
constexpr int kAddThreads = 256;

struct Shared {
    alignas(8) uint64_t full[kStages], empty[kStages], sum_full[2], sum_empty[2], swap, drain;
    uint32_t tmem;
    int gave_up;
    float amax[2][kTileM];  // swiglu: the two halves' row maxima
    int first[EP_MAX_EXPERTS], count[EP_MAX_EXPERTS];
    int tiles[EP_MAX_EXPERTS + 1];  // exclusive scan of the experts' row tiles
};

struct Tile {
    int e, n0;     // expert, first output channel
    int row, rows;  // first row, valid rows (1..128)
};

// Tile `i` of the sequence: a row tile's column tiles follow one another.
__device__ __forceinline__ Tile find_tile(const Shared& sh, int E, int64_t i, int ntiles, int width) {
    const int m = (int)(i / ntiles);
    int lo = 0, hi = E;  // the last expert with tiles[e] <= m
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.tiles[mid] <= m) lo = mid;
        else hi = mid;
    }
    const int r0 = (m - sh.tiles[lo]) * kTileM;
    Tile t;
    t.e = lo;
    t.n0 = (int)(i % ntiles) * width;
    t.row = sh.first[lo] + r0;
    t.rows = min(kTileM, sh.count[lo] - r0);
    return t;
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
group_gemm_kernel(const __grid_constant__ CUtensorMap a_map,
                  const __grid_constant__ CUtensorMap w_map, const float* __restrict__ a_scale,
                  const float* __restrict__ w_scale, int64_t rows, int nk, int N, int E,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                  int kind, int capacity, uint16_t* __restrict__ out, uint8_t* __restrict__ out_q,
                  float* __restrict__ out_scale, uint32_t* __restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Shared& sh = *reinterpret_cast<Shared*>(stages + kStages * (kABytes + kBBytes));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t sum_full = smem_addr(sh.sum_full), sum_empty = smem_addr(sh.sum_empty);
    const uint32_t swap = smem_addr(&sh.swap), drain = smem_addr(&sh.drain);
    volatile int* gave_up = &sh.gave_up;

    if (warp == 0) tmem_alloc(smem_addr(&sh.tmem), 512);
    if (tid == 32) {
        tma_prefetch_map(&a_map);
        tma_prefetch_map(&w_map);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sum_full + 8 * i, 1);
            mbar_init(sum_empty + 8 * i, kAddThreads / 32);
        }
        mbar_init(swap, kAddThreads);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.gave_up = 0;
    }
    pdl_wait();
    pdl_trigger();
    for (int e = tid; e < E; e += kThreads) {
        const Segment s = expert_segment(e, counts, offsets, kind, capacity, rows);
        if (s.bad && blockIdx.x == 0 && status) atomicOr(status, EP_FLAG_BAD_ROW);
        sh.first[e] = (int)s.first;
        sh.count[e] = (int)s.count;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        int base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int n = e0 + lane < E ? (sh.count[e0 + lane] + kTileM - 1) / kTileM : 0;
            int s = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, s, o);
                if (lane >= o) s += v;
            }
            if (e0 + lane < E) sh.tiles[e0 + lane] = base + s - n;
            base += __shfl_sync(kFullMask, s, 31);
        }
        if (lane == 0) sh.tiles[E] = base;
    }
    __syncthreads();

    const uint32_t tmem = sh.tmem;
    const int width = SWIGLU ? 128 : kTileN;  // output channels per tile
    const int ntiles = (N + width - 1) / width;
    const int64_t total = (int64_t)sh.tiles[E] * ntiles;
    const int wrows = SWIGLU ? 2 * N : N;  // weight rows per expert

    if (warp < 4) {
      registers_down<kIssueRegs>();
      if (warp == 0 && lane == 0) {
        // ---- loads
        uint32_t it = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
            const Tile t = find_tile(sh, E, i, ntiles, width);
            const int boxes = (t.rows + kARows - 1) / kARows;
            const bool second = SWIGLU || t.n0 + 128 < N;
            const uint32_t bytes = boxes * kARows * kBlockK + (second ? kBBytes : kBBytes / 2);
            const int w0 = t.e * wrows + t.n0, w1 = SWIGLU ? w0 + N : w0 + 128;
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t s = it % kStages;
                if (!mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, gave_up)) {
                    ok = false;
                    break;
                }
                const uint32_t a = smem_addr(stages) + s * (kABytes + kBBytes), b = a + kABytes;
                mbar_expect_tx(full + 8 * s, bytes);
                for (int j = 0; j < boxes; ++j)
                    tma_load_2d(a + j * kARows * kBlockK, &a_map, kb * kBlockK, t.row + j * kARows, full + 8 * s);
                tma_load_2d(b, &w_map, kb * kBlockK, w0, full + 8 * s);
                if (second) tma_load_2d(b + kBBytes / 2, &w_map, kb * kBlockK, w1, full + 8 * s);
            }
        }
        if (!ok) {  // given up: this block's copies in flight end before it does
            const uint64_t start = global_ns();
            for (uint32_t j = it < kStages ? 0 : it - kStages; j < it; ++j)
                while (!mbar_try_wait(full + 8 * (j % kStages), (j / kStages) & 1) &&
                       global_ns() - start < 1000000000ull) {
                }
        }
      } else if (warp == 1 && lane == 0) {
        // ---- MMAs
        uint32_t it = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
            const Tile t = find_tile(sh, E, i, ntiles, width);
            const uint32_t instr = SWIGLU || t.n0 + 128 < N ? e4m3_instr_desc(kTileM, kTileN)
                                                            : e4m3_instr_desc(kTileM, kTileN / 2);
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t s = it % kStages, b = it & 1;
                if (!mbar_wait(sum_empty + 8 * b, ((it >> 1) & 1) ^ 1, gave_up) ||
                    !mbar_wait(full + 8 * s, (it / kStages) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_addr(stages) + s * (kABytes + kBBytes);
                const uint64_t da = operand_desc(a), db = operand_desc(a + kABytes);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_f8(tmem + b * kTileN, da + 2 * j, db + 2 * j, instr, j > 0);
                mma_commit(empty + 8 * s);
                mma_commit(sum_full + 8 * b);
            }
        }
        if (!ok) {  // given up: the MMAs in flight end before the TMEM is freed
            mma_commit(drain);
            const uint64_t start = global_ns();
            while (!mbar_try_wait(drain, 0) && global_ns() - start < 1000000000ull) {
            }
        }
      }
    } else {
        registers_up<kAddRegs>();
        // ---- scale, add, write
        const int half = (warp - 4) >> 2;         // columns [128 half, +128), swiglu: 64 gate and 64 up
        const int quarter = warp & 3;             // the TMEM lanes that this warp may read
        const int r = quarter * 32 + lane;        // row of the tile
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const int wblocks = (wrows + 127) / 128;  // blocks of 128 weight rows per expert
        uint32_t it = 0, swaps = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
            const Tile t = find_tile(sh, E, i, ntiles, width);
            const bool live = r < t.rows;
            // warps whose rows or columns all lie outside only pass the buffers on
            const bool work = quarter * 32 < t.rows && (SWIGLU || half == 0 || t.n0 + 128 < N);
            const int64_t row = t.row + r;
            const float* sa = a_scale + (live ? row * nk : (int64_t)t.row * nk);
            const int nb = t.n0 / 128;
            const float* sb0 = w_scale + ((int64_t)t.e * wblocks + (SWIGLU ? nb : min(nb + half, wblocks - 1))) * nk;
            const float* sb1 = SWIGLU ? sb0 + (int64_t)(N / 128) * nk : sb0;
            uint64_t acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = 0;
            float va = __ldg(sa), v0 = __ldg(sb0), v1 = __ldg(sb1);
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const float s0 = __fmul_rn(va, v0), s1 = SWIGLU ? __fmul_rn(va, v1) : s0;
                if (kb + 1 < nk) {  // the next block's scales, loaded behind this one's sum
                    va = __ldg(sa + kb + 1);
                    v0 = __ldg(sb0 + kb + 1);
                    if (SWIGLU) v1 = __ldg(sb1 + kb + 1);
                }
                const uint32_t b = it & 1;
                if (!mbar_wait(sum_full + 8 * b, (it >> 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                if (work) {
                    tc_fence_after();
                    const uint32_t from = lanes + b * kTileN;
                    const uint64_t p0 = pack2(__float_as_uint(s0), __float_as_uint(s0));
                    const uint64_t p1 = pack2(__float_as_uint(s1), __float_as_uint(s1));
                    auto column = [&](int c) {
                        return from + (SWIGLU ? (c < 4 ? half * 64 + c * 16 : 128 + half * 64 + (c - 4) * 16)
                                              : half * 128 + c * 16);
                    };
                    uint32_t v[2][16];
                    tmem_load16(v[0], column(0));
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        tmem_wait16(v[c & 1]);
                        if (c < 7) tmem_load16(v[(c + 1) & 1], column(c + 1));
                        else tc_fence_before();
                        if (c == 7) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(sum_empty + 8 * b);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            fma2(acc[c * 8 + j], pack2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), c < 4 ? p0 : p1);
                    }
                } else if (lane == 0) {
                    mbar_arrive(sum_empty + 8 * b);
                }
            }
            if (!ok) break;
            if (!SWIGLU) {
                if (work && live) {
                    uint16_t* o = out + row * N + t.n0 + half * 128;
                    const int left = N - t.n0 - half * 128;  // a multiple of 8
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (c * 8 < left) {
                            const uint4 q = make_uint4(pack_bf16x2_rn(lo2(acc[4 * c]), hi2(acc[4 * c])),
                                                       pack_bf16x2_rn(lo2(acc[4 * c + 1]), hi2(acc[4 * c + 1])),
                                                       pack_bf16x2_rn(lo2(acc[4 * c + 2]), hi2(acc[4 * c + 2])),
                                                       pack_bf16x2_rn(lo2(acc[4 * c + 3]), hi2(acc[4 * c + 3])));
                            st_v4(o + c * 8, q);
                        }
                    }
                }
            } else {
                float h[64], amax = 0.0f;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    h[2 * c] = swiglu(lo2(acc[c]), lo2(acc[32 + c]));
                    h[2 * c + 1] = swiglu(hi2(acc[c]), hi2(acc[32 + c]));
                    amax = fmaxf(amax, fmaxf(fabsf(h[2 * c]), fabsf(h[2 * c + 1])));
                }
                sh.amax[half][r] = amax;
                mbar_arrive(swap);
                if (!mbar_wait(swap, swaps & 1, gave_up)) break;
                ++swaps;
                const float a = fmaxf(fmaxf(sh.amax[0][r], sh.amax[1][r]), 1e-4f);
                // both halves have read the maxima before either writes the next tile's
                mbar_arrive(swap);
                if (!mbar_wait(swap, swaps & 1, gave_up)) break;
                ++swaps;
                if (live) {
                    const float inv = __fdiv_rn(448.0f, a);
                    uint8_t* o = out_q + row * N + t.n0 + half * 64;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* f = h + c * 16 + j * 4;
                            q[j] = cvt_e4m3x2_rn_sat(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv)) |
                                   (cvt_e4m3x2_rn_sat(__fmul_rn(f[2], inv), __fmul_rn(f[3], inv)) << 16);
                        }
                        st_v4(o + c * 16, make_uint4(q[0], q[1], q[2], q[3]));
                    }
                    if (half == 0) out_scale[row * (N / 128) + nb] = __fdiv_rn(a, 448.0f);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && sh.gave_up && status) atomicOr(status, EP_FLAG_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr size_t kSmem = 1024 + kStages * (kABytes + kBBytes) + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "");

}  // namespace

cudaError_t launch_group_gemm(const uint8_t* a_q, const float* a_scale, int64_t rows, int64_t K,
                              const uint8_t* w_q, const float* w_scale, int64_t N, int E,
                              const int32_t* counts, const int32_t* offsets, int kind,
                              int capacity, void* out, uint8_t* out_q, float* out_scale,
                              uint32_t* status, cudaStream_t stream) {
    const bool swiglu = out == nullptr;
    CUtensorMap a_map, w_map;
    cudaError_t err = byte_matrix_map(&a_map, a_q, rows, K, kARows);
    if (err != cudaSuccess) return err;
    err = byte_matrix_map(&w_map, w_q, (int64_t)E * (swiglu ? 2 * N : N), K, 128);
    if (err != cudaSuccess) return err;
    static std::atomic<int> sm_cache[64];
    int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    if (sms <= 0) sms = 1;
    static std::atomic<uint64_t> configured[2];
    auto kernel = swiglu ? group_gemm_kernel<true> : group_gemm_kernel<false>;
    err = raise_smem_limit(kernel, kSmem, configured[swiglu]);
    if (err != cudaSuccess) return err;
    return launch_pdl(kernel, dim3((unsigned)sms), dim3(kThreads), kSmem, stream, a_map, w_map,
                      a_scale, w_scale, rows, (int)(K / 128), (int)N, E, counts, offsets, kind,
                      capacity, static_cast<uint16_t*>(out), out_q, out_scale, status);
}

}  // namespace ep
