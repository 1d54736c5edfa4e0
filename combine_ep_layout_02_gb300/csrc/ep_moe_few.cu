// ep_moe_few.cu -- the whole expert layer for a few tokens in two kernels:
//   up    x's FP8 cast, the gate and up products of every routed expert,
//         SwiGLU and the FP8 cast of h, per (expert, 128 channels of I)
//   down  the second products and the weighted sum over a token's experts
// for tokens whose experts' weights are nearly all read for one to eight rows
// each, so that the time is that of streaming the weights once.
//
// Mathematics: a tile of 16 weight rows is the A operand of an e4m3
// mma.m16n8k32 and up to 8 of the expert's (token, place) pairs are its 8
// columns (a "group", of no more pairs than the call has tokens: an expert with
// more is several groups, whose later readings of the weights come from L2).  Four MMAs make the sum of one block of 128 channels,
// which is then scaled by a_scale * w_scale and added in fp32.  Tensor cores
// of the fifth generation would need 128 rows by at least 8 columns per
// instruction and a trip through TMEM per block; the work here is 2 % of what
// mma.sync delivers, and the memory is what has to be kept busy.
//
// Both kernels are a ring of TMA stages in shared memory, filled by one warp
// as far ahead as the ring reaches, across items, and emptied by the others.
//   up: a stage is one block of K of 128 gate and 128 up rows (32 KB).  Each
//   of 8 warps owns 16 channels as two tiles of 8 gate and the same 8 up rows,
//   so that a lane's accumulators are the gate and up values of the same h,
//   and the FP8 cast of the 128 channels needs only the warps' maxima.  Where
//   the tokens leave room two blocks share an SM, and one streams while the
//   other casts x or writes h.
//   down: a block owns 16 output channels for all groups; a stage is eight
//   blocks of K of one group's 16 weight rows (16 KB) with its tokens' codes
//   and scales.  The warps take the stages in turn, each adds its weighted
//   results per token in shared memory of its own, and the block adds the
//   warps' sums in order: the result never depends on timing.
// Measured (three sets of weights in turn; the rate is the weights' bytes over
// the time): 8 tokens, H = 7168, I = 2048, 256 experts: 380-390 us, 6.5-6.7 TB/s,
// bound by DRAM; 45 tokens, H = 2048, I = 1024, 128 experts: 140-146 us, 5.3 TB/s,
// bound by the last round of up items and by the down warps' 1,930 cycles per
// stage; one token there: 17-20 us, 2.7 TB/s, bound by the two kernels' start-up
// and hand-over (about 10 us) beside 7.5 us of weights: an up block and a down
// block ask for more shared memory than one SM has, so that the down blocks of
// the SMs with an up block begin to read when that one ends.
//
// An SM can draw more than twice its share of the memory's bandwidth, so that
// neither kernel needs its items to divide evenly over the SMs.  Only where
// there are fewer items than half the SMs do clusters of blocks share one.
#include <stddef.h>

#include "ep_few_plan.h"
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kMaxPairs = EP_MOE_FEW_MAX_TOKENS * EP_MAX_TOPK;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSmemHalf = 113 * 1024;  // of two blocks on an SM

// h between the kernels: per pair and eight blocks of 128 channels a record of
// their codes and their scales, one copy for a stage of the down kernel.
constexpr int kRecordBlocks = 8;
constexpr int kRecordScales = kRecordBlocks * 128;            // bytes before the scales
constexpr int kRecord = kRecordScales + kRecordBlocks * 4;

// The groups of a route, built by every block for itself.
struct Groups {
    int count;
    uint16_t expert[kMaxPairs];  // per group
    uint16_t first[kMaxPairs];   // its first entry of `pair`, and their number
    uint16_t pair[kMaxPairs];    // pairs t * k + j ordered by expert, then by pair
    union {
        struct {
            uint8_t size[kMaxPairs];
            uint8_t twice[kMaxPairs];  // whether two of its pairs belong to one token
        };
        uint16_t id[kMaxPairs];  // until the pairs are in order: each one's expert
    };
    uint16_t start[EP_MAX_EXPERTS];
    uint16_t seen[EP_MAX_EXPERTS];
};

// An id of the route.  The down kernel reads them before it waits for the up
// kernel, when only that one's own wait has seen the route complete: the load
// takes the value from L2, past any line that this SM holds from a call before.
__device__ __forceinline__ int route_id(const int32_t* p) { return __ldcg(p); }

// Up to 32 pairs: one per lane, ranked by (expert, pair).
__device__ void build_groups_warp(Groups& g, const int32_t* topk_idx, int P, int E,
                                  int limit, uint32_t* status, bool report) {
    const int lane = threadIdx.x & 31;
    const int e = lane < P ? route_id(topk_idx + lane) : -1;
    const bool live = e >= 0 && e < E;
    if (report) warp_flag(status, !live && e != -1, EP_FLAG_BAD_EXPERT);
    const int key = live ? e : EP_MAX_EXPERTS;
    int at = 0;
    for (int q = 0; q < P; ++q) {
        const int other = __shfl_sync(kFullMask, key, q);
        at += other < key || (other == key && q < lane);
    }
    if (live) {
        g.pair[at] = (uint16_t)lane;
        g.seen[at] = (uint16_t)e;
    }
    const int n = __popc(__ballot_sync(kFullMask, live));
    __syncwarp();
    const int se = lane < n ? g.seen[lane] : -1;  // the lane-th pair in that order
    const unsigned peers = __match_any_sync(kFullMask, se);
    const int in = __popc(peers & lanemask_lt());
    const bool head = lane < n && in % limit == 0;
    const unsigned heads = __ballot_sync(kFullMask, head);
    if (head) {
        const int grp = __popc(heads & lanemask_lt());
        g.expert[grp] = (uint16_t)se;
        g.first[grp] = (uint16_t)lane;
        g.size[grp] = (uint8_t)group_size(__popc(peers), in / limit, limit);
    }
    if (lane == 0) g.count = __popc(heads);
}

// Marks the groups that hold a token twice: its pairs follow one another.
__device__ void mark_twice(Groups& g, int k) {
    for (int i = threadIdx.x & 31; i < g.count; i += 32) {
        bool twice = false;
        for (int j = 1; j < g.size[i]; ++j)
            twice |= g.pair[g.first[i] + j - 1] / k == g.pair[g.first[i] + j] / k;
        g.twice[i] = twice;
    }
}

// Fills `g` (shared); all threads of the block call it.  All read the ids, at
// most 2,048; one warp orders them, 32 at a time.
__device__ void build_groups(Groups& g, const int32_t* topk_idx, int P, int k, int E,
                             uint32_t* status, bool report) {
    const int limit = group_limit(P / k);
    if (P <= 32) {
        if (threadIdx.x < 32) {
            build_groups_warp(g, topk_idx, P, E, limit, status, report);
            __syncwarp();
            mark_twice(g, k);
        }
        __syncthreads();
        return;
    }
    constexpr int kNone = 0xffff;
    for (int e = threadIdx.x; e < E; e += blockDim.x) g.start[e] = g.seen[e] = 0;
    bool bad = false;
    for (int p = threadIdx.x; p < P; p += blockDim.x) {
        const int e = route_id(topk_idx + p);
        const bool live = e >= 0 && e < E;
        bad |= !live && e != -1;
        g.id[p] = (uint16_t)(live ? e : kNone);
    }
    if (report) warp_flag(status, bad, EP_FLAG_BAD_EXPERT);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        auto inclusive = [lane](int v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(kFullMask, v, o);
                if (lane >= o) v += a;
            }
            return v;
        };
        for (int p0 = 0; p0 < P; p0 += 32) {  // pairs per expert
            const int e = p0 + lane < P ? g.id[p0 + lane] : kNone;
            const unsigned peers = __match_any_sync(kFullMask, e);
            if (e != kNone && (peers & lanemask_lt()) == 0) g.start[e] += (uint16_t)__popc(peers);
            __syncwarp();
        }
        int pairs = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {  // their exclusive scan
            const int e = e0 + lane, n = e < E ? g.start[e] : 0, sum = inclusive(n);
            if (e < E) g.start[e] = (uint16_t)(pairs + sum - n);
            pairs += __shfl_sync(kFullMask, sum, 31);
        }
        __syncwarp();
        for (int p0 = 0; p0 < P; p0 += 32) {  // the pairs in expert order
            const int e = p0 + lane < P ? g.id[p0 + lane] : kNone;
            const unsigned peers = __match_any_sync(kFullMask, e);
            const int before = __popc(peers & lanemask_lt());
            int at = 0;
            if (e != kNone) at = g.start[e] + g.seen[e] + before;
            __syncwarp();
            if (e != kNone) {
                g.pair[at] = (uint16_t)(p0 + lane);
                if (before == 0) g.seen[e] += (uint16_t)__popc(peers);
            }
            __syncwarp();
        }
        int groups = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {  // the groups; `id` is no longer needed
            const int e = e0 + lane, n = e < E ? g.seen[e] : 0;
            const int m = group_count(n, limit), sum = inclusive(m);
            for (int i = 0; i < m; ++i) {
                const int at = groups + sum - m + i;
                g.expert[at] = (uint16_t)e;
                g.first[at] = (uint16_t)(g.start[e] + i * limit);
                g.size[at] = (uint8_t)group_size(n, i, limit);
            }
            groups += __shfl_sync(kFullMask, sum, 31);
        }
        if (lane == 0) g.count = groups;
        __syncwarp();
        mark_twice(g, k);
    }
    __syncthreads();
}

// p += A (16 x 32, e4m3, row) * B (32 x 8, e4m3, column), fp32.
__device__ __forceinline__ void mma_e4m3(float (&p)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(p[0]), "+f"(p[1]), "+f"(p[2]), "+f"(p[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 16-byte matrices, one row address per lane.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The sum of one block of 128 channels.  a_row: this lane's weight row (of
// matrix lane / 8: rows 0-7, 8-15, and the same again), 128 bytes with TMA's
// 128-byte swizzle (16-byte chunk c of row r at c ^ (r % 8)); b_row: the 128
// bytes of token lane % 8.
struct Operands {
    uint32_t a[4][4], b[8];
};
__device__ __forceinline__ void load_tokens(Operands& o, uint32_t b_row) {
    const uint32_t quad = (threadIdx.x & 31) >> 3;
    load_matrices(*reinterpret_cast<uint32_t(*)[4]>(o.b), b_row + quad * 16);
    load_matrices(*reinterpret_cast<uint32_t(*)[4]>(o.b + 4), b_row + 64 + quad * 16);
}
__device__ __forceinline__ void load_weights(Operands& o, uint32_t a_row) {
    const uint32_t lane = threadIdx.x & 31, r = lane & 7, hi = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) load_matrices(o.a[j], a_row + (((2 * j + hi) ^ r) << 4));
}
// Two chains of two MMAs, added at the end: half the latency of one of four.
__device__ __forceinline__ void block_product(float (&p)[4], const Operands& o) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = q[i] = 0.0f;
    mma_e4m3(p, o.a[0], o.b[0], o.b[1]);
    mma_e4m3(q, o.a[1], o.b[2], o.b[3]);
    mma_e4m3(p, o.a[2], o.b[4], o.b[5]);
    mma_e4m3(q, o.a[3], o.b[6], o.b[7]);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __fadd_rn(p[i], q[i]);
}

// Ring of TMA stages: the filling warp's side.
struct Fill {
    uint32_t full, empty, stages;  // barrier addresses, their number
    uint32_t s = 0, phase = 1;     // phase: of `empty`, passed at once in the first round
    uint32_t issued = 0;
    __device__ __forceinline__ bool wait(volatile int* gave_up) { return mbar_wait(empty + 8 * s, phase, gave_up); }
    __device__ __forceinline__ void next() {
        ++issued;
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    // Given up: wait, for at most a second, for the copies still in flight.
    __device__ void drain() {
        const uint64_t start = global_ns();
        const uint32_t n = issued < stages ? issued : stages;
        for (uint32_t i = issued - n; i < issued; ++i)
            while (!mbar_try_wait(full + 8 * (i % stages), (i / stages) & 1) &&
                   global_ns() - start < 1000000000ull) {
            }
    }
};

// A barrier of the consuming warps that gives up like every other wait.
struct WarpsBarrier {
    uint32_t bar, phase = 0;
    __device__ __forceinline__ bool sync(volatile int* gave_up) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
        const bool ok = mbar_wait(bar, phase, gave_up);
        phase ^= 1;
        return ok;
    }
};

// ---- up -------------------------------------------------------------------

// The FP8 cast of 16 channels of x, 8 lanes to a block of 128, as in
// quantize16 but for the quotient 448 / a', which is one reciprocal times 448:
// x is bf16, whose few values often lie on the midpoint of two codes, and
// there the second rounding decides.
__device__ __forceinline__ Fp8Group cast16(const uint4& lo, const uint4& hi) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float f[16], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[2 * i] = bf16lo_to_f32(w[i]);
        f[2 * i + 1] = bf16hi_to_f32(w[i]);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    const float a = fmaxf(amax, 1e-4f), inv = __fmul_rn(__frcp_rn(a), 448.0f);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = cvt_e4m3x2_rn_sat(__fmul_rn(f[4 * i], inv), __fmul_rn(f[4 * i + 1], inv)) |
               (cvt_e4m3x2_rn_sat(__fmul_rn(f[4 * i + 2], inv), __fmul_rn(f[4 * i + 3], inv)) << 16);
    return Fp8Group{make_uint4(q[0], q[1], q[2], q[3]), __fdiv_rn(a, 448.0f)};
}

constexpr int kUpStage = 2 * 128 * 128;  // one block of K of 128 gate and 128 up rows
constexpr int kUpMaxStages = 6;

struct UpShared {
    uint64_t full[kUpMaxStages], empty[kUpMaxStages], sync;
    int gave_up;
    uint64_t part_full;
    float amax[2][kCols][kUpWarps];  // [item parity][column][warp]
    Groups g;
};

// C > 1: the C blocks of a cluster share each item's channels of K and the
// first adds the others' sums in order; every cluster has at most one item.
template <int C>
__global__ void __launch_bounds__((kUpWarps + 1) * 32, 2)
few_up_kernel(const __grid_constant__ CUtensorMap w_map, const uint16_t* __restrict__ x, int T,
              int H, int k, const int32_t* topk_idx, const float* __restrict__ s13,
              int I, int E, int stages, uint8_t* __restrict__ h8, uint32_t* __restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* xq = ring + stages * kUpStage;
    const UpPlan plan = up_plan(T, H, C, sizeof(UpShared));
    const int stride = plan.stride, held = plan.rows;
    UpShared& sh = *reinterpret_cast<UpShared*>(xq + plan.shared);
    float* xs = reinterpret_cast<float*>(xq + plan.scales);
    float4* part = reinterpret_cast<float4*>(xq + plan.part);  // C > 1
    const int nk = H / 128, nb = I / 128;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    volatile int* gave_up = &sh.gave_up;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kUpWarps);
        }
        mbar_init(smem_addr(&sh.sync), kUpWarps);
        mbar_init(smem_addr(&sh.part_full), (C - 1) * kUpWarps + (C == 1));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.gave_up = 0;
        tma_prefetch_map(&w_map);
    }
    pdl_wait();
    pdl_trigger();
    build_groups(sh.g, topk_idx, T * k, k, E, status, blockIdx.x == 0);
    if (C > 1) cluster_sync();  // the first block's barrier is ready for the others
    const int items = sh.g.count * nb;  // (group, block of 128 channels)
    const int worker = blockIdx.x / C, workers = gridDim.x / C;
    // this block's blocks of K
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
    const int k0 = nk * rank / C, k1 = nk * (rank + 1) / C;

    if (warp == kUpWarps) {
        Fill fill{full, empty, (uint32_t)stages};
        bool ok = true;
        for (int item = worker; item < items && ok; item += workers) {
            const int gate = sh.g.expert[item / nb] * 2 * I + item % nb * 128;
            for (int kb = k0; kb < k1; ++kb) {
                if (!(ok = fill.wait(gave_up))) break;
                if (elect_one()) {
                    const uint32_t bar = full + 8 * fill.s, to = smem_addr(ring) + fill.s * kUpStage;
                    mbar_expect_tx(bar, kUpStage);
                    tma_load_2d(to, &w_map, kb * 128, gate, bar);
                    tma_load_2d(to + kUpStage / 2, &w_map, kb * 128, gate + I, bar);
                }
                __syncwarp();
                fill.next();
            }
        }
        if (!ok) fill.drain();
    } else {
        WarpsBarrier barrier{smem_addr(&sh.sync)};
        const int row = lane >> 2, q4 = lane & 3;
        // matrices 0 and 2: this warp's gate rows, 1 and 3: its up rows
        const uint32_t a_lane = smem_addr(ring) + ((lane >> 3) & 1) * (kUpStage / 2) + (warp * 8 * kUpTiles + (lane & 7)) * 128;
        const uint32_t b_lane = smem_addr(xq) + min(lane & 7, held - 1) * stride;
        const float* x0 = xs + min(2 * q4, held - 1) * nk;  // the scales of this lane's two tokens
        const float* x1 = xs + min(2 * q4 + 1, held - 1) * nk;
        uint32_t s = 0, phase = 0, parity = 0;
        int have = -1;  // the group whose x is in shared memory
        bool ok = true;
        for (int item = worker; item < items && ok; item += workers) {
            const int grp = item / nb, b = item % nb, n = sh.g.size[grp], first = sh.g.first[grp];
            const float* sg = s13 + ((int64_t)sh.g.expert[grp] * 2 * nb + b) * nk;
            const float* su = sg + (int64_t)nb * nk;
            // the weights' scales, a block per lane: the first 32, read behind the cast
            float vg = __ldg(sg + min(k0 + lane, nk - 1)), vu = __ldg(su + min(k0 + lane, nk - 1));
            if (grp != have) {
                // The previous group's reads are done: all warps met at the maxima
                // since.  Pieces of 512 channels, two per warp at a time.
                const int per = (k1 - k0 + 3) / 4, pieces = n * per;
                for (int p0 = warp; p0 < pieces; p0 += 2 * kUpWarps) {
                    uint4 a[2], q[2];
                    int tok[2], c[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int piece = p0 + u * kUpWarps;
                        tok[u] = piece / per;
                        c[u] = k0 * 128 + (piece - tok[u] * per) * 512 + lane * 16;
                        if (piece >= pieces) c[u] = k1 * 128;  // no such piece
                        a[u] = q[u] = make_uint4(0, 0, 0, 0);
                        if (c[u] < k1 * 128) {
                            const uint16_t* src = x + (int64_t)(sh.g.pair[first + tok[u]] / k) * H + c[u];
                            a[u] = __ldg(reinterpret_cast<const uint4*>(src));
                            q[u] = __ldg(reinterpret_cast<const uint4*>(src + 8));
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const Fp8Group f = cast16(a[u], q[u]);
                        if (c[u] < k1 * 128) {
                            *reinterpret_cast<uint4*>(xq + tok[u] * stride + c[u]) = f.q;
                            if ((lane & 7) == 0) xs[tok[u] * nk + (c[u] >> 7)] = f.sf;
                        }
                    }
                }
                have = grp;
                if (!(ok = barrier.sync(gave_up))) break;
            }
            float acc[kUpTiles][4] = {};
            for (int kb = k0; kb < k1; ++kb) {
                if (kb > k0 && (kb - k0) % 32 == 0) {
                    const int to = min(kb + lane, nk - 1);
                    vg = __ldg(sg + to);
                    vu = __ldg(su + to);
                }
                if (!(ok = mbar_wait(full + 8 * s, phase, gave_up))) break;
                Operands o[kUpTiles];
                float p[kUpTiles][4];
                load_tokens(o[0], b_lane + kb * 128);
#pragma unroll
                for (int j = 0; j < kUpTiles; ++j) {
                    if (j > 0)
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[j].b[i] = o[0].b[i];
                    load_weights(o[j], a_lane + s * kUpStage + j * 8 * 128);
                }
#pragma unroll
                for (int j = 0; j < kUpTiles; ++j) block_product(p[j], o[j]);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * s);
                if (++s == (uint32_t)stages) {
                    s = 0;
                    phase ^= 1;
                }
                const float wg = __shfl_sync(kFullMask, vg, (kb - k0) % 32);
                const float wu = __shfl_sync(kFullMask, vu, (kb - k0) % 32);
                const float c0 = x0[kb], c1 = x1[kb];
#pragma unroll
                for (int j = 0; j < kUpTiles; ++j) {
                    acc[j][0] = __fmaf_rn(p[j][0], __fmul_rn(c0, wg), acc[j][0]);
                    acc[j][1] = __fmaf_rn(p[j][1], __fmul_rn(c1, wg), acc[j][1]);
                    acc[j][2] = __fmaf_rn(p[j][2], __fmul_rn(c0, wu), acc[j][2]);
                    acc[j][3] = __fmaf_rn(p[j][3], __fmul_rn(c1, wu), acc[j][3]);
                }
            }
            if (!ok) break;
            if (C > 1) {
                if (rank > 0) {  // hand the sums to the cluster's first block: nothing else to do
#pragma unroll
                    for (int j = 0; j < kUpTiles; ++j) {
                        const uint32_t to = cluster_addr(
                            smem_addr(part + (((rank - 1) * kUpWarps + warp) * kUpTiles + j) * 32 + lane), 0);
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(acc[j][0]),
                                     "f"(acc[j][1]), "f"(acc[j][2]), "f"(acc[j][3])
                                     : "memory");
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&sh.part_full), 0));
                    break;
                }
                if (!(ok = mbar_wait_cluster(smem_addr(&sh.part_full), 0, gave_up))) break;
#pragma unroll
                for (int r = 0; r < C - 1; ++r) {
#pragma unroll
                    for (int j = 0; j < kUpTiles; ++j) {
                        const float4 v = part[((r * kUpWarps + warp) * kUpTiles + j) * 32 + lane];
                        acc[j][0] = __fadd_rn(acc[j][0], v.x);
                        acc[j][1] = __fadd_rn(acc[j][1], v.y);
                        acc[j][2] = __fadd_rn(acc[j][2], v.z);
                        acc[j][3] = __fadd_rn(acc[j][3], v.w);
                    }
                }
            }
            float h[kUpTiles][2], m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < kUpTiles; ++j) {
                    h[j][i] = swiglu(acc[j][i], acc[j][2 + i]);
                    m[i] = fmaxf(m[i], fabsf(h[j][i]));
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(kFullMask, m[i], o));
            }
            if (lane < 4) {
                sh.amax[parity][2 * lane][warp] = m[0];
                sh.amax[parity][2 * lane + 1][warp] = m[1];
            }
            if (!(ok = barrier.sync(gave_up))) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 2 * q4 + i;
                float a = 1e-4f;
#pragma unroll
                for (int w = 0; w < kUpWarps; ++w) a = fmaxf(a, sh.amax[parity][col][w]);
                if (col < n) {
                    const int pair = sh.g.pair[first + col];
                    const float inv = __fdiv_rn(448.0f, a);
                    uint8_t* record = h8 + ((int64_t)pair * ((nb + kRecordBlocks - 1) / kRecordBlocks) +
                                            b / kRecordBlocks) * kRecord;
                    uint8_t* to = record + b % kRecordBlocks * 128 + warp * 8 * kUpTiles + row;
#pragma unroll
                    for (int j = 0; j < kUpTiles; ++j)
                        to[j * 8] = (uint8_t)cvt_e4m3x2_rn_sat(__fmul_rn(h[j][i], inv), 0.0f);
                    if (warp == 0 && row == 0)
                        reinterpret_cast<float*>(record + kRecordScales)[b % kRecordBlocks] = __fdiv_rn(a, 448.0f);
                }
            }
            parity ^= 1;  // the next item's maxima go to the other buffer
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && sh.gave_up && status) atomicOr(status, EP_FLAG_TIMEOUT);
    if (C > 1) cluster_sync();  // no block leaves while another may still write to it
}

template <int C>
cudaError_t launch_up(int blocks, size_t smem, cudaStream_t stream, const CUtensorMap& w_map, const void* x,
                      int T, int H, int k, const int32_t* topk_idx, const float* s13, int I, int E, int stages,
                      uint8_t* h8, uint32_t* status) {
    static std::atomic<uint64_t> configured{0};
    const cudaError_t err = raise_smem_limit(few_up_kernel<C>, kSmemLimit, configured);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((kUpWarps + 1) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {C, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, few_up_kernel<C>, w_map, static_cast<const uint16_t*>(x), T, H, k,
                              topk_idx, s13, I, E, stages, h8, status);
}


// ---- down -----------------------------------------------------------------

// Multiplying warps, and as many stages: a warp's stages always lie in the same
// place.  Eight where the tokens' sums leave room for them, else six (8 tokens
// at H = 7168: 383 us against 395 us with six; one at 2048: 19.5 against 20.2).
constexpr int kDownMaxWarps = 8, kDownMinWarps = 6;
constexpr int kDownRows = 16;                     // output channels of a block
constexpr int kDownBlocks = kRecordBlocks;        // blocks of K of a stage
constexpr int kDownW = kDownRows * kDownBlocks * 128;
constexpr int kTokenRow = kRecord + 16;           // an odd number of 16 bytes: eight rows' chunks meet all banks
constexpr int kDownStage = (kDownW + kCols * kTokenRow + 1023) / 1024 * 1024;
static_assert(kTokenRow / 16 % 2 == 1 && kRecord % 16 == 0, "");

struct DownShared {
    uint64_t full[kDownMaxWarps], empty[kDownMaxWarps], sync;
    int gave_up;
    Groups g;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

template <int kDownWarps>
__global__ void __launch_bounds__((kDownWarps + 2) * 32, 1)
few_down_kernel(const __grid_constant__ CUtensorMap w_map, const uint8_t* __restrict__ h8, int T, int H, int k,
                const int32_t* topk_idx, const float* __restrict__ topk_w,
                const float* __restrict__ s2, int I, int E, uint16_t* __restrict__ out,
                uint32_t* __restrict__ status) {
    constexpr int kDownStages = kDownWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float* slabs = reinterpret_cast<float*>(ring + kDownStages * kDownStage);  // [warp][token][16 channels]
    DownShared& sh = *reinterpret_cast<DownShared*>(slabs + kDownWarps * T * kDownRows);
    const int nk = I / 128;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    volatile int* gave_up = &sh.gave_up;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDownStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(smem_addr(&sh.sync), kDownWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.gave_up = 0;
        tma_prefetch_map(&w_map);
    }
    // The route and the weights are older than the up kernel, which let this
    // one start only after all earlier work had completed.
    build_groups(sh.g, topk_idx, T * k, k, E, nullptr, false);
    const int tiles = H / kDownRows;
    const int groups = sh.g.count;

    if (warp == kDownWarps) {
        // ---- weights, from before the up kernel has finished on the SMs that
        // its blocks have left
        Fill fill{full, empty, (uint32_t)kDownStages};
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            int n = 0, e = 0;
            if (groups > 0) n = sh.g.size[0], e = sh.g.expert[0];
            for (int grp = 0; grp < groups && ok; ++grp) {
                const int tokens = n, wrow = e * H + tile * kDownRows;
                if (grp + 1 < groups) n = sh.g.size[grp + 1], e = sh.g.expert[grp + 1];
                for (int b0 = 0; b0 < nk; b0 += kDownBlocks) {
                    if (!(ok = fill.wait(gave_up))) break;
                    if (elect_one()) {
                        const uint32_t bar = full + 8 * fill.s;
                        mbar_expect_tx(bar, kDownW + tokens * kRecord);
                        tma_load_3d(smem_addr(ring) + fill.s * kDownStage, &w_map, 0, wrow, b0, bar);
                    }
                    __syncwarp();
                    fill.next();
                }
            }
        }
        if (!ok) fill.drain();
    } else if (warp == kDownWarps + 1) {
        // ---- h: a stage's tokens' records, one lane each
        pdl_wait();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        Fill fill{full, empty, (uint32_t)kDownStages};
        bool ok = true;
        const int records = (nk + kRecordBlocks - 1) / kRecordBlocks;
        // four groups at a look: lane 8 g + c has the records of column c of group g
        const uint32_t to = smem_addr(ring) + kDownW + (lane & 7) * kTokenRow;
        auto look = [&](int grp) -> const uint8_t* {
            grp += lane >> 3;
            return grp < groups && (lane & 7) < sh.g.size[grp]
                       ? h8 + (int64_t)sh.g.pair[sh.g.first[grp] + (lane & 7)] * records * kRecord
                       : nullptr;
        };
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const uint8_t* next = look(0);
            for (int grp0 = 0; grp0 < groups && ok; grp0 += 4) {
                const uint8_t* src = next;
                next = look(grp0 + 4);
                const int n = min(4, groups - grp0) * records;
                for (int i = 0, g = 0, r = 0; i < n; ++i) {
                    if (!(ok = fill.wait(gave_up))) break;
                    if (src && (lane >> 3) == g)
                        bulk_load(to + fill.s * kDownStage, src + r * kRecord, kRecord, full + 8 * fill.s);
                    __syncwarp();
                    fill.next();
                    if (++r == records) {
                        r = 0;
                        ++g;
                    }
                }
            }
        }
        if (!ok) fill.drain();
    } else {
        const int slab_n = T * kDownRows;
        for (int i = threadIdx.x; i < kDownWarps * slab_n; i += kDownWarps * 32) slabs[i] = 0.0f;
        pdl_wait();
        WarpsBarrier barrier{smem_addr(&sh.sync)};
        const int row = lane >> 2, q4 = lane & 3;
        const uint32_t a_lane = smem_addr(ring) + (lane & 15) * 128;
        const uint32_t b_lane = smem_addr(ring) + kDownW + (lane & 7) * kTokenRow;
        const uint8_t* c_lane = ring + kDownW + 2 * q4 * kTokenRow + kRecordScales;  // the first of two tokens' scales
        float* slab = slabs + warp * slab_n;
        const int per_group = (nk + kDownBlocks - 1) / kDownBlocks;  // stages
        const uint32_t per_tile = groups * per_group;
        const uint32_t s = warp;
        uint32_t base = 0, at = warp, phase = 0;  // stages before this tile; this warp's next
        // What a stage needs besides its bytes: its first block of K, the
        // weights' scales (block b0 + lane % 8), and this lane's two columns'
        // tokens and weights.
        struct Next {
            int b0, n, t0, t1;
            bool twice;
            float scale, wt0, wt1;
        };
        auto look = [&](uint32_t u, const float* ws) {
            Next x{};
            if (u < per_tile) {
                const int grp = u / per_group, first = sh.g.first[grp];
                x.b0 = u % per_group * kDownBlocks;
                x.n = sh.g.size[grp];
                x.twice = sh.g.twice[grp];
                x.scale = __ldg(ws + (int64_t)sh.g.expert[grp] * (H / 128) * nk + min(x.b0 + (lane & 7), nk - 1));
                const int pair0 = sh.g.pair[first + min(2 * q4, x.n - 1)];
                const int pair1 = sh.g.pair[first + min(2 * q4 + 1, x.n - 1)];
                x.wt0 = __ldg(topk_w + pair0);
                x.wt1 = __ldg(topk_w + pair1);
                x.t0 = pair0 / k;
                x.t1 = pair1 / k;
            }
            return x;
        };
        bool ok = barrier.sync(gave_up);
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, base += per_tile) {
            const float* ws = s2 + (int64_t)(tile * kDownRows / 128) * nk;  // of expert 0
            // this warp's stages: every kDownWarps-th of the block's sequence; the next
            // one's scalars are read behind the wait for this one
            Next next = look(at - base, ws);
            for (; at < base + per_tile; at += kDownWarps) {
                const Next now = next;
                next = look(at + kDownWarps - base, ws);
                if (!(ok = mbar_wait(full + 8 * s, phase, gave_up))) break;
                phase ^= 1;
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const uint32_t a = a_lane + s * kDownStage, t = b_lane + s * kDownStage;
                const float* c = reinterpret_cast<const float*>(c_lane + s * kDownStage);
                // two blocks at a time, the next two's operands read behind their
                // MMAs; what lies past the last block is read, not used
                Operands o[4];
                auto operands = [&](int j) {
                    load_tokens(o[j & 3], t + j * 128);
                    load_weights(o[j & 3], a + j * kDownRows * 128);
                };
                operands(0);
                operands(1);
#pragma unroll
                for (int j = 0; j < kDownBlocks; j += 2) {
                    if (now.b0 + j < nk) {  // warp-uniform
                        if (j + 2 < kDownBlocks) {
                            operands(j + 2);
                            operands(j + 3);
                        }
                        float p[2][4];
                        block_product(p[0], o[j & 3]);
                        block_product(p[1], o[(j + 1) & 3]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (now.b0 + j + i < nk) {
                                const float w = __shfl_sync(kFullMask, now.scale, j + i);
                                const float c0 = __fmul_rn(c[j + i], w), c1 = __fmul_rn(c[kTokenRow / 4 + j + i], w);
                                acc[0] = __fmaf_rn(p[i][0], c0, acc[0]);
                                acc[1] = __fmaf_rn(p[i][1], c1, acc[1]);
                                acc[2] = __fmaf_rn(p[i][2], c0, acc[2]);
                                acc[3] = __fmaf_rn(p[i][3], c1, acc[3]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * s);
                float* o0 = slab + now.t0 * kDownRows + row;
                float* o1 = slab + now.t1 * kDownRows + row;
                if (!now.twice) {  // every column has a token of its own
                    if (2 * q4 < now.n) {
                        o0[0] = __fmaf_rn(now.wt0, acc[0], o0[0]);
                        o0[8] = __fmaf_rn(now.wt0, acc[2], o0[8]);
                    }
                    if (2 * q4 + 1 < now.n) {
                        o1[0] = __fmaf_rn(now.wt1, acc[1], o1[0]);
                        o1[8] = __fmaf_rn(now.wt1, acc[3], o1[8]);
                    }
                } else {  // one column after another
                    for (int col = 0; col < now.n; ++col) {
                        if (col / 2 == q4) {
                            float* o = col & 1 ? o1 : o0;
                            const float wt = col & 1 ? now.wt1 : now.wt0;
                            o[0] = __fmaf_rn(wt, col & 1 ? acc[1] : acc[0], o[0]);
                            o[8] = __fmaf_rn(wt, col & 1 ? acc[3] : acc[2], o[8]);
                        }
                        __syncwarp();
                    }
                }
                __syncwarp();
            }
            if (!ok || !(ok = barrier.sync(gave_up))) break;
            // add the warps' sums in order and clear them
            for (int v = threadIdx.x; v < slab_n / 2; v += kDownWarps * 32) {
                float x = 0.0f, y = 0.0f;
#pragma unroll
                for (int w = 0; w < kDownWarps; ++w) {
                    float2* p2 = reinterpret_cast<float2*>(slabs + w * slab_n) + v;
                    x = __fadd_rn(x, p2->x);
                    y = __fadd_rn(y, p2->y);
                    *p2 = make_float2(0.0f, 0.0f);
                }
                *reinterpret_cast<uint32_t*>(out + (int64_t)(v / 8) * H + tile * kDownRows + v % 8 * 2) =
                    pack_bf16x2_rn(x, y);
            }
            ok = barrier.sync(gave_up);
        }
    }
    pdl_trigger();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && sh.gave_up && status) atomicOr(status, EP_FLAG_TIMEOUT);
}

constexpr size_t up_rest(int T, int H, int C) {  // shared memory besides the ring
    return 1024 + up_plan(T, H, C, sizeof(UpShared)).bytes;
}
constexpr size_t down_smem(int warps, int T) {
    return 1024 + (size_t)warps * kDownStage + (size_t)warps * T * kDownRows * 4 + sizeof(DownShared);
}
static_assert(up_rest(EP_MOE_FEW_MAX_TOKENS, EP_MOE_FEW_MAX_WIDTH, 1) + 2 * kUpStage <= kSmemLimit,
              "at least two stages at the widest");
static_assert(down_smem(kDownMinWarps, EP_MOE_FEW_MAX_TOKENS) <= kSmemLimit, "");

}  // namespace

size_t moe_few_bytes(int64_t T, int k, int I) {
    return ((size_t)T * k * ((I / 128 + kRecordBlocks - 1) / kRecordBlocks) * kRecord + 255) / 256 * 256;
}

cudaError_t launch_moe_few(const void* x, int T, int H, int k, const int32_t* topk_idx,
                           const float* topk_w, const uint8_t* w13, const float* s13,
                           const uint8_t* w2, const float* s2, int I, int E, void* out,
                           uint32_t* status, void* workspace, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    static std::atomic<int> sm_cache[64];
    int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    if (sms <= 0) sms = 1;
    uint8_t* h8 = static_cast<uint8_t*>(workspace);

    CUtensorMap w13_map, w2_map;
    cudaError_t err = byte_matrix_map(&w13_map, w13, (int64_t)E * 2 * I, H, 128);
    if (err != cudaSuccess) return err;
    // at most one group per pair and 128 channels
    const int64_t items = (int64_t)T * k * (I / 128);
    // Few items leave SMs without one: then several blocks share an item's K
    // (not at widths where the tokens would leave the ring too few stages).
    // One token, unshared against shared: 8 items at H = 7168 37.5 -> 19.9 us
    // (C = 4), 64 items at 7168 49.5 -> 42.6 us (C = 2), 16 items at 2048 15.9
    // -> 13.2 us (C = 4), 64 items at 2048 the same (19.7 and 20.0 us).
    const int C = H > 8192 || H < 1024 ? 1 : items * 4 <= sms ? 4 : items * 2 <= sms ? 2 : 1;
    const size_t rest = up_rest(T, H, C);
    // Two blocks per SM where each has at least two stages and an item (45
    // tokens, H = 2048: 152 us against 159 us with one).
    const int per_sm = C == 1 && items > sms && rest + 2 * kUpStage <= kSmemHalf ? 2 : 1;
    int stages = (int)(((per_sm == 2 ? kSmemHalf : kSmemLimit) - rest) / kUpStage);
    if (stages > kUpMaxStages) stages = kUpMaxStages;
    const int blocks = C > 1 ? (int)items * C : (int)(items < sms * per_sm ? items : sms * per_sm);
    const auto up = C == 4 ? launch_up<4> : C == 2 ? launch_up<2> : launch_up<1>;
    err = up(blocks, rest + (size_t)stages * kUpStage, stream, w13_map, x, T, H, k, topk_idx, s13, I, E, stages,
             h8, status);
    if (err != cudaSuccess) return err;

    const int tiles = H / kDownRows;
    err = byte_blocks_map(&w2_map, w2, (int64_t)E * H, I, kDownRows, kDownBlocks);
    if (err != cudaSuccess) return err;
    static std::atomic<uint64_t> configured[2];
    const bool most = down_smem(kDownMaxWarps, T) <= kSmemLimit;
    const int warps = most ? kDownMaxWarps : kDownMinWarps;
    const auto down = most ? few_down_kernel<kDownMaxWarps> : few_down_kernel<kDownMinWarps>;
    err = raise_smem_limit(down, kSmemLimit, configured[most]);
    if (err != cudaSuccess) return err;
    return launch_pdl(down, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3((warps + 2) * 32),
                      down_smem(warps, T), stream, w2_map, h8, T, H, k, topk_idx, topk_w, s2, I, E,
                      static_cast<uint16_t*>(out), status);
}

}  // namespace ep
