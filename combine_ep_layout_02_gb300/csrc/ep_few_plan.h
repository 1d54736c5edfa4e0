// ep_few_plan.h -- plain arithmetic of the few-token layer that its kernels,
// their launcher and a host compiler share: how many pairs a group may hold,
// and where things lie in the up kernel's shared memory.
#pragma once

#include <stddef.h>

#ifdef __CUDACC__
#define EP_PLAN __host__ __device__ __forceinline__ constexpr
#else
#define EP_PLAN constexpr
#endif

namespace ep {

constexpr int kCols = 8;           // columns of one MMA
constexpr int kUpWarps = 8;        // multiplying warps of an up block
constexpr int kUpTiles = 16 / kUpWarps;  // of 8 channels, per warp

// Most pairs of a group.  The up kernel keeps a row of x for every pair of the
// group at hand, and a call of T < 8 tokens has T rows of room (one token: 7 KB
// instead of 57 KB at H = 7168, which the ring needs).  A token may name an
// expert several times, so that an expert can have more pairs than there are
// tokens: then it has more groups.
EP_PLAN int group_limit(int T) { return T < kCols ? T : kCols; }
// Groups that n pairs of one expert make, and the size of the i-th of them.
EP_PLAN int group_count(int n, int limit) { return (n + limit - 1) / limit; }
EP_PLAN int group_size(int n, int i, int limit) { return n - i * limit < limit ? n - i * limit : limit; }

// Bytes from the end of the up kernel's ring (a multiple of 1,024).
struct UpPlan {
    int rows;    // of x and of its scales
    int stride;  // bytes of a row of codes: 16 of padding, so that eight rows' chunks meet all banks
    size_t shared;  // the block's barriers and tables, after the rows
    size_t scales;  // [row][H / 128] float
    size_t part;    // clusters of C > 1 blocks: the others' sums [C - 1][warp][tile][lane] float4
    size_t bytes;
};
EP_PLAN UpPlan up_plan(int T, int H, int C, size_t shared_bytes) {
    UpPlan p{};
    p.rows = group_limit(T);
    p.stride = H + 16;
    p.shared = (size_t)p.rows * p.stride;  // H is a multiple of 128: 16-byte aligned
    p.scales = p.shared + shared_bytes;
    p.part = (p.scales + (size_t)p.rows * (H / 128) * 4 + 15) / 16 * 16;
    p.bytes = p.part + (size_t)(C - 1) * kUpWarps * kUpTiles * 32 * 16;
    return p;
}

}  // namespace ep
