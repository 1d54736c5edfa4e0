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
// per row and block of 128, so that the tensor core cannot apply them: it makes
// each block's sum (four tcgen05.mma of K = 32 into one of two TMEM buffers),
// and eight warps read that sum back, scale it and add it into fp32 registers
// while the next block's MMAs run.  A TMEM lane is a row, so the row's scale is
// one value per thread.
//
// One persistent block per SM: warp 0 issues the TMA loads (128-byte swizzle,
// four stages), warp 1 the MMAs, warps 2 and 3 bring the scales into shared
// memory, and warps 4-11 scale, add and write the output.  The block is
// launched with 168 registers a thread; the first warpgroup keeps 72 and leaves
// the rest to the other two, 216 each, which need 128 for the sums alone.
//
// Few rows per expert: bound by the weights' bytes (64 rows each, 256 experts:
// 575 us and 1.09 ms, 7.0 TB/s; a plain copy, half of it writes, makes 6.7).
// Many rows: the tensor pipe is busy 58 % of the cycles (16,384 rows, 32 experts,
// K = 7168: 430 us, 2.2 PFLOP/s).  The adding warps' chain sets the pace, about
// 880 cycles per block of K: some 150 to learn that a sum is there, 450 to read and add it, the rest the
// scales, the loop and the share of the tile's epilogue; 512 cycles of MMAs and
// the loads run beside it.  Long calls also meet the power limit
// (1.45 GHz after some milliseconds, 1.7 GHz at first).  Measured and not
// taken: a pair of SMs per 256 x 256 tile (464 against 444 us; half of the
// weight traffic, but rows are padded to 256 and each hand-over crosses the
// SMs), 16 adding warps (476), the two halves of N as separate MMAs (538: A is
// read twice from shared memory), 32 columns per TMEM load (461).
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kRowsM = 128;                     // rows of a tile
constexpr int kTileN = 256, kBlockK = 128;
constexpr int kStages = 4;
constexpr int kABytes = kRowsM * kBlockK, kBBytes = kTileN * kBlockK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kARows = 32;                      // rows per TMA box of A: at most 31 past the segment's end are read
constexpr int kAddWarps = 8;                    // warps that scale and add
constexpr int kAddThreads = kAddWarps * 32;
constexpr int kThreads = 128 + kAddThreads;
constexpr int kIssueRegs = 72, kAddRegs = 216;  // 128 * 72 + 256 * 216 = 384 * 168
constexpr int kShares = kAddWarps / 4;          // column shares of a tile
constexpr int kCols = kTileN / kShares;         // columns of a share
constexpr int kChunk = 16;                      // columns per TMEM load
constexpr int kAhead = 16;                      // blocks whose scales are brought together

struct Shared {
    alignas(8) uint64_t full[kStages], empty[kStages], sum_full[2], sum_empty[2];
    uint64_t scale_full[2], scale_empty[2], swap, drain;
    uint32_t tmem;
    int gave_up;
    // weight scales of the tile's two blocks of 128 weight rows and row scales;
    // a row past the last lets the reader run one block ahead
    alignas(8) float2 sw[2][kAhead + 1];
    float sa[2][kAhead + 1][kRowsM + 1];
    int4 tile[2];                     // the tile that each scale buffer belongs to
    float amax[2][kShares][kRowsM];   // swiglu: the shares' row maxima
    int first[EP_MAX_EXPERTS], count[EP_MAX_EXPERTS];
    int tiles[EP_MAX_EXPERTS + 1];    // exclusive scan of the experts' row tiles
};

struct Tile {
    int e, n0;      // expert, first output channel
    int row, rows;  // first row, valid rows (1..128)
};

// The tiles of a block, one after another, as a whole warp walks them: a row
// tile's column tiles follow one another, and the block takes every step-th.
struct Walk {
    uint32_t m, n;    // row tile and column tile
    uint32_t dm, dn;  // a step, split in the same way
    int e;            // an expert at or before the row tile's
    __device__ Walk(uint32_t first, uint32_t step, uint32_t ntiles)
        : m(first / ntiles), n(first % ntiles), dm(step / ntiles), dn(step % ntiles), e(0) {}
    __device__ __forceinline__ void next(uint32_t ntiles) {
        m += dm;
        n += dn;
        if (n >= ntiles) {
            n -= ntiles;
            ++m;
        }
    }
    // Expert e has the row tiles [tiles[e], tiles[e + 1]): 32 experts at a look.
    __device__ __forceinline__ Tile tile(const Shared& sh, int E, int width) {
        const int lane = threadIdx.x & 31;
        unsigned past;
        while ((past = __ballot_sync(kFullMask, sh.tiles[min(e + 1 + lane, E)] > (int)m)) == 0) e += 32;
        e += __ffs(past) - 1;
        const int r0 = ((int)m - sh.tiles[e]) * kRowsM;
        Tile t;
        t.e = e;
        t.n0 = (int)n * width;
        t.row = sh.first[e] + r0;
        t.rows = min(kRowsM, sh.count[e] - r0);
        return t;
    }
};

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
    Shared& sh = *reinterpret_cast<Shared*>(stages + kStages * kStageBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t sum_full = smem_addr(sh.sum_full), sum_empty = smem_addr(sh.sum_empty);
    const uint32_t scale_full = smem_addr(sh.scale_full), scale_empty = smem_addr(sh.scale_empty);
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
            mbar_init(sum_empty + 8 * i, kAddWarps);
            mbar_init(scale_full + 8 * i, 2);
            mbar_init(scale_empty + 8 * i, kAddWarps);
        }
        mbar_init(swap, kAddWarps);
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
            const int n = e0 + lane < E ? (sh.count[e0 + lane] + kRowsM - 1) / kRowsM : 0;
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
    const uint32_t total = (uint32_t)sh.tiles[E] * ntiles;  // at most an output row's tiles each
    const int wrows = SWIGLU ? 2 * N : N;     // weight rows per expert
    const int wblocks = (wrows + 127) / 128;  // and blocks of 128 of them
    // rows of output that allow 32-byte stores
    const bool wide = SWIGLU ? (uintptr_t)out_q % 32 == 0 : (uintptr_t)out % 32 == 0 && N % 16 == 0;
    const uint32_t step = gridDim.x;

    if (warp < 4) {
        registers_down<kIssueRegs>();
        if (warp == 0) {
            // ---- loads
            uint32_t it = 0;
            bool ok = true;
            Walk walk(blockIdx.x, step, ntiles);
            for (uint32_t i = blockIdx.x; i < total && ok; i += step, walk.next(ntiles)) {
                const Tile t = walk.tile(sh, E, width);
                const bool second = SWIGLU || t.n0 + 128 < N;  // the tile has a second 128 weight rows
                const int boxes = (t.rows + kARows - 1) / kARows;
                const uint32_t bytes = boxes * kARows * kBlockK + (second ? kBBytes : kBBytes / 2);
                const int w0 = t.e * wrows + t.n0, w1 = w0 + (SWIGLU ? N : 128);
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_addr(stages) + s * kStageBytes;
                    if (elect_one()) {
                        mbar_expect_tx(full + 8 * s, bytes);
                        for (int j = 0; j < boxes; ++j)
                            tma_load_2d(a + j * kARows * kBlockK, &a_map, kb * kBlockK, t.row + j * kARows,
                                        full + 8 * s);
                        tma_load_2d(a + kABytes, &w_map, kb * kBlockK, w0, full + 8 * s);
                        if (second)
                            tma_load_2d(a + kABytes + kBBytes / 2, &w_map, kb * kBlockK, w1, full + 8 * s);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // given up: the copies in flight end before the block does
                const uint64_t start = global_ns();
                for (uint32_t j = it < kStages ? 0 : it - kStages; j < it; ++j)
                    while (!mbar_try_wait(full + 8 * (j % kStages), (j / kStages) & 1) &&
                           global_ns() - start < 1000000000ull) {
                    }
            }
        } else if (warp == 1) {
            // ---- MMAs
            uint32_t it = 0;
            bool ok = true;
            const uint32_t instr = e4m3_instr_desc(kRowsM, kTileN);
            for (uint32_t i = blockIdx.x; i < total && ok; i += step) {
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t s = it % kStages, b = it & 1;
                    // the operands are there long before the sums have room
                    if (!mbar_wait(full + 8 * s, (it / kStages) & 1, gave_up) ||
                        !mbar_wait(sum_empty + 8 * b, ((it >> 1) & 1) ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_addr(stages) + s * kStageBytes;
                    const uint64_t da = operand_desc(a), db = operand_desc(a + kABytes);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f8(tmem + b * kTileN, da + 2 * j, db + 2 * j, instr, j > 0);
                        mma_commit(sum_full + 8 * b);
                        mma_commit(empty + 8 * s);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // given up: the MMAs in flight end before the TMEM is freed
                if (elect_one()) mma_commit(drain);
                __syncwarp();
                const uint64_t start = global_ns();
                while (!mbar_try_wait(drain, 0) && global_ns() - start < 1000000000ull) {
                }
            }
        } else if (warp >= 2) {
            // ---- scales: 16 blocks of K at a time, whole lines of each row
            uint32_t c = 0;
            bool ok = true;
            const int kl = lane & 15, side = lane >> 4;
            Walk walk(blockIdx.x, step, ntiles);
            for (uint32_t i = blockIdx.x; i < total && ok; i += step, walk.next(ntiles)) {
                const Tile t = walk.tile(sh, E, width);
                const int live = t.rows;
                const float* src = a_scale + (int64_t)(t.row) * nk;
                const int nb = t.n0 / 128 + (side == 0 ? 0 : SWIGLU ? N / 128 : 1);
                const float* wsrc = w_scale + ((int64_t)t.e * wblocks + min(nb, wblocks - 1)) * nk;
                for (int k0 = 0; k0 < nk; k0 += kAhead, ++c) {
                    const uint32_t b = c & 1;
                    if (!mbar_wait(scale_empty + 8 * b, ((c >> 1) & 1) ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    if (warp == 2 && lane == 0) sh.tile[b] = make_int4(t.e, t.n0, t.row, t.rows);
                    const bool in = k0 + kl < nk;
                    if (warp == 2) (side ? sh.sw[b][kl].y : sh.sw[b][kl].x) = in ? __ldg(wsrc + k0 + kl) : 0.0f;
                    for (int r0 = 0; r0 < kRowsM && r0 < live; r0 += 32) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int r = r0 + j * 4 + (warp - 2) * 2 + side;
                            v[j] = in && r < live ? __ldg(src + (int64_t)r * nk + k0 + kl) : 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) sh.sa[b][kl][r0 + j * 4 + (warp - 2) * 2 + side] = v[j];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(scale_full + 8 * b);
                }
            }
        }
    } else {
        registers_up<kAddRegs>();
        // ---- scale, add, write
        const int share = (warp - 4) >> 2;        // columns [kCols * share, +kCols), swiglu: half of them up
        const int quarter = warp & 3;             // the TMEM lanes that this warp may read
        const int r = quarter * 32 + lane;        // row of the block
        // this warp's lanes, at its share's first column
        const uint32_t lanes =
            tmem + ((uint32_t)(quarter * 32) << 16) + share * (SWIGLU ? kCols / 2 : kCols);
        constexpr int kChunks = kCols / kChunk;
        // chunk c of the share: the up half of a swiglu share lies 128 columns after its gate half
        auto column = [](int c) { return c * kChunk + (SWIGLU && c >= kChunks / 2 ? 128 - kCols / 2 : 0); };
        uint32_t buf = 0, parity = 0;  // the sum at hand: 8 x buffer, and its barrier's phase
        uint32_t c16 = 0, swaps = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < total && ok; i += step) {
            if (!mbar_wait(scale_full + 8 * (c16 & 1), (c16 >> 1) & 1, gave_up)) break;
            const int4 info = sh.tile[c16 & 1];
            const Tile t{info.x, info.y, info.z, info.w};
            const bool live = r < t.rows;
            // warps whose rows or columns all lie outside only pass the buffers on
            const bool work = quarter * 32 < t.rows && (SWIGLU || t.n0 + share * kCols < N);
            const int64_t row = t.row + r;
            uint64_t acc[kCols / 2];  // pairs of columns
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) acc[c] = 0;
            for (int k0 = 0; k0 < nk && ok; k0 += kAhead, ++c16) {
                const uint32_t sbuf = c16 & 1;
                if (k0 > 0 && !mbar_wait(scale_full + 8 * sbuf, (c16 >> 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                const float* pa = &sh.sa[sbuf][0][r];
                const float2* pw = sh.sw[sbuf];
                float va = *pa;
                float2 w = *pw;
                const int n = min(kAhead, nk - k0);
#pragma unroll 1
                for (int kc = 0; kc < n; ++kc) {
                    const float s0 = __fmul_rn(va, SWIGLU || share * kCols < 128 ? w.x : w.y);
                    const float s1 = SWIGLU ? __fmul_rn(va, w.y) : s0;
                    const uint64_t p0 = pack2(s0, s0), p1 = SWIGLU ? pack2(s1, s1) : p0;
                    pa += kRowsM + 1;
                    ++pw;
                    va = *pa;  // the next block's, read behind this one's sum
                    w = *pw;
                    if (!mbar_wait(sum_full + buf, parity, gave_up)) {
                        ok = false;
                        break;
                    }
                    if (work) {
                        tc_fence_after();
                        const uint32_t from = lanes + buf * (kTileN / 8);
                        uint32_t v[2][kChunk];
                        tmem_load(v[0], from);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            tmem_wait();
                            if (c + 1 < kChunks) {
                                tmem_load(v[(c + 1) & 1], from + column(c + 1));
                            } else {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(sum_empty + buf);
                            }
#pragma unroll
                            for (int j = 0; j < kChunk / 2; ++j)
                                fma2(acc[c * kChunk / 2 + j], v[c & 1][2 * j], v[c & 1][2 * j + 1],
                                     c < kChunks / 2 ? p0 : p1);
                        }
                    } else if (lane == 0) {
                        mbar_arrive(sum_empty + buf);
                    }
                    parity ^= buf >> 3;
                    buf ^= 8;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(scale_empty + 8 * sbuf);
            }
            if (!ok) break;
            if (!SWIGLU) {
                if (work && live) {
                    uint16_t* o = out + row * N + t.n0 + share * kCols;
                    const int cols = N - t.n0 - share * kCols;  // a multiple of 8
                    auto pack8 = [&](int c) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) q[j] = pack_bf16x2_rn(lo2(acc[4 * c + j]), hi2(acc[4 * c + j]));
                        return make_uint4(q[0], q[1], q[2], q[3]);
                    };
                    if (wide) {  // whole sectors
#pragma unroll
                        for (int c = 0; c < kCols / 8; c += 2)
                            if (c * 8 < cols) st_v8(o + c * 8, Vec32{pack8(c), pack8(c + 1)});
                    } else {
#pragma unroll
                        for (int c = 0; c < kCols / 8; ++c)
                            if (c * 8 < cols) st_v4(o + c * 8, pack8(c));
                    }
                }
            } else {
                constexpr int kH = kCols / 2;
                float h[kH], amax = 0.0f;
#pragma unroll
                for (int c = 0; c < kH / 2; ++c) {
                    h[2 * c] = swiglu(lo2(acc[c]), lo2(acc[kH / 2 + c]));
                    h[2 * c + 1] = swiglu(hi2(acc[c]), hi2(acc[kH / 2 + c]));
                    amax = fmaxf(amax, fmaxf(fabsf(h[2 * c]), fabsf(h[2 * c + 1])));
                }
                // the shares' maxima meet in shared memory, every other tile's in
                // the other place: who writes there again has passed a barrier
                // that all reach after reading
                sh.amax[swaps & 1][share][r] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(swap);
                if (!mbar_wait(swap, swaps & 1, gave_up)) break;
                float a = 1e-4f;
#pragma unroll
                for (int j = 0; j < kShares; ++j) a = fmaxf(a, sh.amax[swaps & 1][j][r]);
                ++swaps;
                if (live) {
                    const float inv = __fdiv_rn(448.0f, a);
                    uint8_t* o = out_q + row * N + t.n0 + share * kH;
                    auto codes16 = [&](int c) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* f = h + c * 16 + j * 4;
                            q[j] = cvt_e4m3x2_rn_sat(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv)) |
                                   (cvt_e4m3x2_rn_sat(__fmul_rn(f[2], inv), __fmul_rn(f[3], inv)) << 16);
                        }
                        return make_uint4(q[0], q[1], q[2], q[3]);
                    };
                    if (wide) {
#pragma unroll
                        for (int c = 0; c < kH / 16; c += 2) st_v8(o + c * 16, Vec32{codes16(c), codes16(c + 1)});
                    } else {
#pragma unroll
                        for (int c = 0; c < kH / 16; ++c) st_v4(o + c * 16, codes16(c));
                    }
                    if (share == 0) out_scale[row * (N / 128) + t.n0 / 128] = __fdiv_rn(a, 448.0f);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && sh.gave_up && status) atomicOr(status, EP_FLAG_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr size_t kSmem = 1024 + kStages * kStageBytes + sizeof(Shared);
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
    const int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    static std::atomic<uint64_t> configured[2];
    auto kernel = swiglu ? group_gemm_kernel<true> : group_gemm_kernel<false>;
    err = raise_smem_limit(kernel, kSmem, configured[swiglu]);
    if (err != cudaSuccess) return err;
    return launch_pdl(kernel, dim3((unsigned)(sms > 0 ? sms : 1)), dim3(kThreads), kSmem, stream,
                      a_map, w_map, a_scale, w_scale, rows, (int)(K / 128), (int)N, E, counts,
                      offsets, kind, capacity, static_cast<uint16_t*>(out), out_q, out_scale,
                      status);
}

}  // namespace ep
