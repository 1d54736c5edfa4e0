// ep_products.cu -- BF16 products grouped by expert, and their gradients, on
// tcgen05.  For rows r of expert e:
//   forward  out[r, n] = sum_k x[r, k] w[e, n, k]       (dense: one expert)
//   input    dx[r, k]  = sum_n dy[r, n] w[e, n, k]
//   weight   dw[e, n, k] = sum_r dy[r, n] x[r, k]
// bf16 operands, fp32 sums, and an epilogue on the sums: bias, activation or
// SwiGLU and residual (forward), SwiGLU's derivative (input), an addend
// (weight).
//
// A tile is the product of a pair of SMs: 256 x up to 256 sums, 128 of the rows
// in each block's TMEM, both blocks' halves of the other operand shared.  The
// 256 rows are the weights' output channels (weight: the channels of dy); the
// columns are the expert's tokens (weight: the channels of x).  Tokens are the
// ragged side, and the column count of an MMA goes in steps of 32, so that an
// expert's tokens are split evenly and rounded up to 32, where rows would be
// rounded up to 256 (16,384 rows over 32 experts: 6 % instead of 25 % wasted).
// What a kernel reads as rows or columns may have its summed index or its rows
// contiguous in memory; tcgen05 takes either through the descriptors, so that no
// operand is transposed.
//
// Forward and input: an expert's last columns may hold rows of the next
// segment, which only reach columns that are not written.  Weight: the tokens
// are the summed index, and rows behind the segment may hold anything, so that
// the last block's rows are overwritten with zeros in shared memory before the
// MMAs read them.
//
// One persistent block per SM: warp 0 issues the TMA loads (128-byte swizzle,
// five or six stages of 64 values of the summed index), warp 1 of the even block
// the MMAs, warp 2 clears the tails, the warps from 4 on write the output while
// the next tile's MMAs run into the other half of the TMEM.  Forward and input:
// TMEM lanes are channels, the output's rows tokens; sums are read in an mma
// accumulator's layout and turned by stmatrix, so that the stores run along the
// channels, and what the epilogue reads turns the other way.  Weight: a lane is a
// row of dw; 128 bytes of 32 rows go through shared memory to a TMA store.
//
// The tensor core truncates where it adds to a sum: over n steps of 16 values
// the result shrinks by about n / 3 parts in 2^24 (operands of one sign, spread over
// many binades: n).  fp32 outputs (weight gradients, router logits, the parts of a
// split sum) show it, and in time a bf16 output does (4 million rows: 3 %).  So a sum
// ends after 512 values and eight warps add the sums, rounded, in registers (128 a
// thread: setmaxnreg moves registers from the four issuing warps).  1,024 rows to
// fp32: error 1.1e-6 without, 4.4e-7 with; 1.40 against 1.43-1.48 ms for 3.8 GB of
// gradients.  bf16 outputs keep whole sums up to 16,384 values, where the loss is 2e-5
// (7e-5 at most) and the rounding 2e-3 to 4e-3: reading the TMEM every 512 values, and
// one stage less, cost 2 to 8 % there, through SwiGLU's derivative up to 28 % (8
// experts, 8,192 rows, 4,096 of 7,168: 286 and 299 us; their weights' gradient of
// 1,024 rows each 272 and 282).
//
// Few tokens per expert: bound by the weights' bytes (4 rows each of 128 experts:
// 84 us, 6.3 TB/s).  Many: by the tensor pipe, 95 % of its cycles busy (8 experts
// of 1,024 rows, K 7168: 269 us, 1.79 PFLOP/s; dense 8,192 x 4,096 x 7,168: 247-257
// us, cuBLAS 254), and on long calls by the power limit (1.5-1.6 PFLOP/s).
// Behind it lies the copies' rate: a stage brings 32 KB into an SM in the 512
// cycles of its MMAs, and an SM takes about 60 bytes a cycle.  So narrower tiles
// wait for their weights (stage times in dense_plan()), and weight gradients of
// few rows, whose tiles are stored after 16 stages, reach 67 % (fp32) and 83 %
// (bf16) of the tensor pipe.
//
// Measured and not taken: clusters of two pairs that share the columns' copies
// by multicast (within 2 % everywhere: the bytes into an SM stay the same, and
// clusters of four leave 8 of 152 SMs idle); weight gradients stored from
// registers, a lane a channel (111 -> 175 us at 19 rows: 64-byte pieces); full
// tiles of 256 tokens and a rest (2.79 instead of 2.46 ms); several copies of 16
// rows per stage (each copy costs the stage some 20 cycles); TMEM loads a chunk ahead (no
// change: a load takes 100 cycles of a chunk's 1,000); residuals two chunks ahead
// instead of one (no change); a release at cluster scope
// behind the tails' zeros (3.49 -> 1.49 ms without).
#include "ep_product_wait.h"
#include "ep_products.cuh"
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTileM = 256, kTileN = 256, kBlockK = 64;  // per pair
constexpr int kMaxStages = 6;
constexpr int kABytes = 128 * kBlockK * 2, kBBytes = 128 * kBlockK * 2;  // per block and stage
constexpr int kStageBytes = kABytes + kBBytes;
// Warps that write the output: four, or two column shares of four (`eight`:
// sums in parts).
__host__ __device__ constexpr int epi_warps(bool eight) { return eight ? 8 : 4; }
__host__ __device__ constexpr int threads_of(bool eight) { return 128 + 32 * epi_warps(eight); }
constexpr int kSlot = 32 * 64;   // staging: 32 tokens of 32 channels in bf16
constexpr int kBox = 32 * 128;   // 32 rows of 128 bytes
// per warp: two slots, or a box, at the expense of a stage
__host__ __device__ constexpr int staging(bool eight) { return eight ? kBox : 2 * kSlot; }
__host__ __device__ constexpr int stage_count(bool eight) { return eight ? 5 : kMaxStages; }
// Sums in parts: blocks of the summed index whose sum the tensor core makes, and
// registers of the first warps and of those that add.
constexpr int kSeg = 8;
constexpr int kIssueRegs = 72, kAddRegs = 216;  // 128 * 72 + 256 * 216 = 384 * 168
// The sum of a bf16 output stays whole up to this many blocks, 16,384 values.
constexpr int kWholeBlocks = 256;
// Forward and input products have an instance for either (CUT).  An expert's rows are
// known on the device alone: the one instance for bf16 weight gradients does both.
template <ProductKind KIND, bool F32, bool CUT>
__device__ __forceinline__ bool in_parts(int blocks) {
    return KIND == kWeight && !F32 ? blocks > kWholeBlocks : CUT;
}
constexpr int kBand = 16;        // channel tiles that share the tokens while they are in L2

struct Shared {
    alignas(8) uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int gave_up;
    int first[EP_MAX_EXPERTS], count[EP_MAX_EXPERTS];
    int tiles[EP_MAX_EXPERTS + 1];  // exclusive scan of the experts' token tiles
};

constexpr size_t smem_bytes(bool eight) {
    return 1024 + stage_count(eight) * kStageBytes + epi_warps(eight) * staging(eight) + sizeof(Shared);
}
static_assert(smem_bytes(false) <= 227 * 1024 && smem_bytes(true) <= 227 * 1024, "");

struct Maps {
    CUtensorMap a;     // the 256-row side: weights; dy
    CUtensorMap b[8];  // the other: boxes of 16, 32, .. 128 tokens, one copy per stage and block
                       // (weight: b[0] x, boxes of 64 tokens x 64 channels; b[1] dw, of 32 rows)
};

struct Tile {
    int e;
    int m0;       // first channel of the pair's 256 (SwiGLU forward: of 128)
    int row;      // first token; weight: the segment's first
    int n;        // valid columns
    int width;    // columns of the MMA
    int n0;       // weight: first channel of x
    int blocks;   // of the summed index
    int tail;     // weight: rows of the last block that count, 0: all
    int k0;       // first value of the summed index
    int part;     // of the summed index
};

// Sizes of a call that every role derives its tiles from.
struct Grid {
    int channels;     // output channels on the 256-row side
    int per;          // of them in a tile
    int mtiles;       // tiles of them
    int ntiles;       // weight: tiles of x's channels
    int most;         // columns of a tile at most
    int blocks;       // of the summed index, per part (not weight)
    int splits, last; // parts of it, and the last part's blocks
    uint64_t total;   // tiles
};

template <ProductKind KIND>
struct Walk {
    int e = 0;
    // Tile i, as a whole warp walks them in increasing order.
    __device__ __forceinline__ Tile tile(const Shared& sh, const Grid& g, int E, uint64_t i) {
        Tile t;
        if (KIND == kWeight) {
            const uint32_t per = (uint32_t)g.mtiles * g.ntiles;
            t.e = (int)(i / per);
            const uint32_t r = (uint32_t)(i - (uint64_t)t.e * per);
            t.m0 = (int)(r / g.ntiles) * kTileM;
            t.n0 = (int)(r % g.ntiles) * g.most;
            t.row = sh.first[t.e];
            const int count = sh.count[t.e];
            t.blocks = (count + kBlockK - 1) / kBlockK;
            t.tail = count % kBlockK;
            t.width = g.most;
            t.n = g.most;
            t.k0 = t.part = 0;
            return t;
        }
        t.part = 0;
        if (KIND == kForward && g.splits > 1) {
            t.part = (int)(i % (uint32_t)g.splits);
            i /= (uint32_t)g.splits;
        }
        t.k0 = t.part * g.blocks * kBlockK;
        t.blocks = t.part == g.splits - 1 ? g.last : g.blocks;
        const int lane = threadIdx.x & 31;
        const uint64_t at = i / (uint32_t)g.mtiles;  // the expert's share: mtiles for each of its token tiles
        unsigned past;
        while ((past = __ballot_sync(kFullMask, (uint64_t)sh.tiles[min(e + 1 + lane, E)] > at)) == 0) e += 32;
        e += __ffs(past) - 1;
        const uint32_t tokens = (uint32_t)(sh.tiles[e + 1] - sh.tiles[e]);
        const uint64_t r = i - (uint64_t)sh.tiles[e] * (uint32_t)g.mtiles;
        // bands of channel tiles; within a band all channels of a token tile, then the next token tile
        const uint64_t band_size = (uint64_t)tokens * kBand;
        const uint32_t band = (uint32_t)(r / band_size);
        const uint32_t in = (uint32_t)(r - band * band_size);
        const uint32_t wide = min((uint32_t)kBand, (uint32_t)g.mtiles - band * kBand);
        const uint32_t tt = in / wide;
        const int count = sh.count[e];
        t.e = e;
        t.m0 = (int)(band * kBand + in % wide) * g.per;
        // the tokens in units of 32, split as evenly as they go: two widths that differ by a unit
        const uint32_t units = (uint32_t)(count + 31) / 32, base = units / tokens, more = units - base * tokens;
        const int before = (int)(tt * base + min(tt, more)) * 32;
        t.row = sh.first[e] + before;
        t.width = (int)(base + (tt < more)) * 32;
        t.n = min(t.width, count - before);
        t.n0 = 0;
        t.tail = 0;
        return t;
    }
};

// ---- the epilogue's pieces ---------------------------------------------------

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// The addend of a box of 32 rows x 128 bytes: `rows` and `cols` exist, the
// first of them at element `at`, rows ld apart.  Read box by box, each with its whole
// latency: 64 experts, 65,536 rows, 2,048 x 7,168, fp32 1.48 ms without and 2.8 with an
// addend, bf16 1.24 and 1.43; 2,300 rows of 128 experts, 2,048 x 1,024: 188 and 720 us, 93
// and 327 (3 and 5 times the addend's bytes).
__device__ __forceinline__ void add_to_box(uint32_t box, const void* add, int size, int64_t at, int64_t ld, int rows,
                                           int cols) {
    const int lane = threadIdx.x & 31, piece = lane & 7;
    const uint8_t* base = static_cast<const uint8_t*>(add) + (at + piece * (16 / size)) * size;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (r < rows && piece * (16 / size) < cols)
            st_shared_v4(box + r * 128 + ((piece ^ (r & 7)) << 4), *reinterpret_cast<const uint4*>(base + r * ld * size));
    }
    __syncwarp();
}

// A warp's 32 tokens x 32 channels (SwiGLU forward: 16) of bf16 in shared
// memory, 16-byte pieces exchanged so that neither the fragments' nor the rows'
// accesses share a bank.
template <int PIECES>  // 16-byte pieces per token: 4 or 2
__device__ __forceinline__ uint32_t slot_at(uint32_t slot, int token, int piece) {
    return slot + token * (PIECES * 16) + ((piece ^ ((token >> (PIECES == 4 ? 1 : 2)) & (PIECES - 1))) << 4);
}

// A lane's address for half `h` (channels 16h..) and token groups c, c + 1.
template <int PIECES>
__device__ __forceinline__ uint32_t fragment_at(uint32_t slot, int h, int c) {
    const int lane = threadIdx.x & 31, j = lane >> 3;
    return slot_at<PIECES>(slot, 8 * (c + (j >> 1)) + (lane & 7), 2 * h + (j & 1));
}

template <int PIECES>
__device__ __forceinline__ void put_fragments(uint32_t slot, int h, const float (&v)[16]) {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = pack_bf16x2_rn(v[4 * c + 2 * j], v[4 * c + 2 * j + 1]);
        stmatrix_trans(fragment_at<PIECES>(slot, h, c), q);
    }
}
template <int PIECES>
__device__ __forceinline__ void get_fragments(uint32_t slot, int h, float (&v)[16]) {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
        uint32_t q[4];
        ldmatrix_trans(q, fragment_at<PIECES>(slot, h, c));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[4 * c + 2 * j] = bf16lo_to_f32(q[j]);
            v[4 * c + 2 * j + 1] = bf16hi_to_f32(q[j]);
        }
    }
}

// 32 rows of PIECES * 16 bytes, of which `tokens` and `bytes` exist, `ld` bytes
// apart in memory: a lane has one piece of every 32 / PIECES-th row.
template <int PIECES>
struct Rows {
    uint4 v[PIECES];
    static __device__ __forceinline__ int token(int i) { return i * (32 / PIECES) + (threadIdx.x & 31) / PIECES; }
    static __device__ __forceinline__ int piece() { return (threadIdx.x & 31) % PIECES; }
    __device__ __forceinline__ void load(const void* at, int64_t ld, int tokens, int bytes) {
        const uint8_t* p = static_cast<const uint8_t*>(at) + piece() * 16;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (token(i) < tokens && piece() * 16 < bytes) v[i] = *reinterpret_cast<const uint4*>(p + token(i) * ld);
    }
    __device__ __forceinline__ void store(void* at, int64_t ld, int tokens, int bytes) const {
        uint8_t* p = static_cast<uint8_t*>(at) + piece() * 16;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (token(i) < tokens && piece() * 16 < bytes) st_v4(p + token(i) * ld, v[i]);
    }
    __device__ __forceinline__ void put(uint32_t slot) const {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) st_shared_v4(slot_at<PIECES>(slot, token(i), piece()), v[i]);
        __syncwarp();
    }
    __device__ __forceinline__ void get(uint32_t slot) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PIECES; ++i) v[i] = ld_shared_v4(slot_at<PIECES>(slot, token(i), piece()));
        __syncwarp();
    }
};

// The slot's rows to memory.
template <int PIECES>
__device__ __forceinline__ void write_rows(uint32_t slot, uint16_t* at, int64_t ld, int tokens, int channels) {
    Rows<PIECES> r;
    r.get(slot);
    r.store(at, ld * 2, tokens, channels * 2);
}

__device__ __forceinline__ void as_floats(const uint32_t (&v)[16], float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
}

__device__ __forceinline__ void activate16(float (&f)[16], int act) {
    if (act == EP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = activate(f[i], EP_ACT_RELU);
    } else if (act == EP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = activate(f[i], EP_ACT_SILU);
    } else if (act == EP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = activate(f[i], EP_ACT_GELU);
    }
}

__device__ __forceinline__ void activate4(float (&f)[4], int act) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = activate(f[i], act);
}

// A lane's row and piece of 16 bytes in a box with the TMA's 128-byte swizzle.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int row, int piece) {
    return box + row * 128 + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ void store_box(uint32_t box, const CUtensorMap& map, int x, int y, int z) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tma_store_3d(&map, x, y, z, box);
}

// fp32 gradients of weights: rows n.. of dw (a lane's each), `share` columns from k.
__device__ __forceinline__ void write_weights(const float (&acc)[8][16], const ProductArgs& p, const CUtensorMap& map,
                                              uint32_t box, const Tile& t, int n, int k, int share, int N, int K) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {  // 32 columns
        if (c * 16 >= share || n >= N || k + c * 16 >= K) break;
        if (lane == 0) tma_store_wait<0>();
        __syncwarp();
        if (p.add) add_to_box(box, p.add, 4, ((int64_t)t.e * N + n) * K + k + c * 16, K, N - n, K - k - c * 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t at = box_at(box, lane, j);
            float f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = acc[c + (j >> 2)][(j & 3) * 4 + x];
            if (p.add) {
                const uint4 q = ld_shared_v4(at);
                f[0] += __uint_as_float(q.x), f[1] += __uint_as_float(q.y);
                f[2] += __uint_as_float(q.z), f[3] += __uint_as_float(q.w);
            }
            st_shared_v4(at, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                        __float_as_uint(f[3])));
        }
        store_box(box, map, k + c * 16, n, t.e);
    }
}

// 64 columns of bf16 gradients of weights: rows n.. of dw (a lane's each), columns from k, of which `cols` exist.
__device__ __forceinline__ void write_weights_bf16(const float (&v)[4][16], const ProductArgs& p, const CUtensorMap& map,
                                                   uint32_t box, int e, int n, int k, int cols, int N, int K) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) tma_store_wait<0>();
    __syncwarp();
    if (p.add) add_to_box(box, p.add, 2, ((int64_t)e * N + n) * K + k, K, N - n, cols);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t at = box_at(box, lane, h * 2 + j);
            float q8[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) q8[x] = v[h][8 * j + x];
            if (p.add) {
                const uint4 q = ld_shared_v4(at);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    q8[2 * x] += bf16lo_to_f32(w[x]);
                    q8[2 * x + 1] += bf16hi_to_f32(w[x]);
                }
            }
            st_shared_v4(at, make_uint4(pack_bf16x2_rn(q8[0], q8[1]), pack_bf16x2_rn(q8[2], q8[3]),
                                        pack_bf16x2_rn(q8[4], q8[5]), pack_bf16x2_rn(q8[6], q8[7])));
        }
    }
    store_box(box, map, k, n, e);
}

// fp32 outputs of a dense layer: channels ch.. (a lane's each), `share` columns
// of the tile from c0.  32 tokens of 32 channels turn in shared memory (a lane's
// channel in, four channels of a token out), so that a store is 16 bytes a lane.
__device__ __forceinline__ void write_tokens(const float (&acc)[8][16], const ProductArgs& p, uint32_t slot,
                                             const Tile& t, int ch, int c0, int share, int channels) {
    const int lane = threadIdx.x & 31, piece = lane & 7, n = ch + piece * 4;
    const bool live = n < channels;
    float bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = p.bias && live ? load_typed(p.bias, p.bias_type, n + j) : 0.0f;
    float* out = static_cast<float*>(p.out) + (int64_t)t.part * p.rows * channels;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
        const int left = min(share, t.n - c0) - c * 16;  // tokens from here on
        if (left <= 0 || ch >= channels) break;
        const int tokens = live ? min(32, left) : 0;
        const int64_t at = (int64_t)(t.row + c0 + c * 16) * channels + ch;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + j * 128 + lane * 4), "f"(acc[c + (j >> 4)][j & 15])
                         : "memory");
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 8; h += 4) {  // 16 tokens, their residuals' loads together
            float4 r[4];
            const int64_t mine = at + (int64_t)Rows<8>::token(h) * channels + piece * 4;
            if (p.residual) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (Rows<8>::token(h + j) < tokens)
                        r[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + mine + (int64_t)j * 4 * channels);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int token = Rows<8>::token(h + j);
                if (token >= tokens) continue;
                const int64_t to = mine + (int64_t)j * 4 * channels;
                const uint4 q = ld_shared_v4(slot + token * 128 + piece * 16);
                float f[4] = {__uint_as_float(q.x) + bias[0], __uint_as_float(q.y) + bias[1],
                              __uint_as_float(q.z) + bias[2], __uint_as_float(q.w) + bias[3]};
                if (p.z)
                    *reinterpret_cast<uint2*>(p.z + to) =
                        make_uint2(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]));
                if (p.activation != EP_ACT_NONE) activate4(f, p.activation);
                if (p.residual) f[0] += r[j].x, f[1] += r[j].y, f[2] += r[j].z, f[3] += r[j].w;
                st_v4(out + to, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                           __float_as_uint(f[3])));
            }
        }
    }
}

template <ProductKind KIND, bool SWIGLU, bool F32, bool CUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(CUT), 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ProductArgs p, int most) {
    constexpr bool kGated = SWIGLU && KIND == kForward;  // two rows of weights per output channel
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr bool kEight = CUT;
    static_assert(CUT || (!F32 && KIND != kWeight), "");
    constexpr int kStages = stage_count(kEight), kStaging = staging(kEight);
    constexpr int kEpiWarps = epi_warps(kEight), kThreads = threads_of(kEight);
    uint8_t* slots = stages + kStages * kStageBytes;
    Shared& sh = *reinterpret_cast<Shared*>(slots + kEpiWarps * kStaging);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty), tail = smem_addr(sh.tail);
    const uint32_t acc_full = smem_addr(sh.acc_full), acc_empty = smem_addr(sh.acc_empty);
    const uint32_t drain = smem_addr(&sh.drain);
    volatile int* gave_up = &sh.gave_up;

    if (warp == 0) tmem_alloc_pair(smem_addr(&sh.tmem), 512);
    if (tid == 32) {
        tma_prefetch_map(&maps.a);
        tma_prefetch_map(&maps.b[0]);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, KIND == kWeight ? 2 : 1);
            mbar_init(empty + 8 * i, 1);
            mbar_init(tail + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.gave_up = 0;
    }
    for (int e = tid; e < p.E; e += kThreads) {
        const Segment s = product_segment(p, e);
        if (s.bad && blockIdx.x == 0 && p.status) atomicOr(p.status, EP_FLAG_BAD_ROW);
        sh.first[e] = (int)s.first;
        sh.count[e] = (int)s.count;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (KIND != kWeight && warp == 0 && !scan_tiles(sh.count, p.E, most, sh.tiles) && tid == 0 && blockIdx.x == 0 &&
        p.status)
        atomicOr(p.status, EP_FLAG_BAD_ROW);
    cluster_sync();  // both blocks' barriers are set up

    const uint32_t tmem = sh.tmem;
    const int N = (int)p.N, K = (int)p.K;
    Grid g;
    g.channels = KIND == kForward ? (kGated ? N / 2 : N) : KIND == kInput ? K : N;
    g.per = kGated ? kTileM / 2 : kTileM;
    g.mtiles = (g.channels + g.per - 1) / g.per;
    g.most = most;
    g.ntiles = KIND == kWeight ? (K + most - 1) / most : 1;
    const int blocks = ((KIND == kInput ? N : K) + kBlockK - 1) / kBlockK;
    g.splits = KIND == kForward ? p.splits : 1;
    g.blocks = (blocks + g.splits - 1) / g.splits;
    g.last = blocks - (g.splits - 1) * g.blocks;
    g.total = KIND == kWeight ? (uint64_t)p.E * g.mtiles * g.ntiles : (uint64_t)sh.tiles[p.E] * g.mtiles * g.splits;
    const uint32_t pair = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < 4) {
        if (CUT) registers_down<kIssueRegs>();
        if (warp == 0) {
            // ---- loads: this block's 128 rows of A and its half of B's columns
            const uint32_t bar0 = cluster_addr(full, 0);
            // widths of whole blocks of 64 channels: one copy brings a stage's two blocks
            const bool awhole = KIND != kForward && g.channels % 64 == 0;
            const bool bwhole = KIND == kWeight && K % 64 == 0 && most == kTileN;
            uint32_t it = 0;
            bool ok = true;
            Walk<KIND> walk;
            for (uint64_t i = pair; i < g.total && ok; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                const int half = t.width / 2;
                const uint32_t bytes = kABytes + half * kBlockK * 2;
                const int m = t.m0 + rank * (g.per / 2);          // this block's first channel
                const int brow = t.row + rank * half;             // and token
                for (int kb = 0; kb < t.blocks; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_addr(stages) + s * kStageBytes, b = a + kABytes;
                    const bool last = KIND == kWeight && t.tail != 0 && kb == t.blocks - 1;
                    uint32_t bar = bar0 + 8 * s;
                    if (elect_one()) {
                        if (KIND == kWeight) {
                            if (last) {  // counted here, and passed on by warp 2
                                bar = cluster_addr(tail, rank) + 8 * s;
                                mbar_expect_tx(tail + 8 * s, bytes);
                            } else {
                                mbar_expect_tx_pair(bar, bytes);
                            }
                        } else if (rank == 0) {
                            mbar_expect_tx(full + 8 * s, 2 * bytes);
                        }
                        const int k0 = t.k0 + kb * kBlockK;
                        if (KIND == kWeight) {
                            const int r0 = t.row + k0;
                            if (awhole) {
                                tma_pair_3d(a, &maps.a, 0, r0, m / 64, bar);
                            } else {
                                tma_pair_2d(a, &maps.a, m, r0, bar);
                                tma_pair_2d(a + kABytes / 2, &maps.a, m + 64, r0, bar);
                            }
                            const int n = t.n0 + rank * half;
                            if (bwhole)
                                tma_pair_3d(b, &maps.b[0], 0, r0, n / 64, bar);
                            else
                                for (int j = 0; j < half; j += 64) tma_pair_2d(b + j * 128, &maps.b[0], n + j, r0, bar);
                        } else {
                            if (kGated) {
                                tma_pair_5d(a, &maps.a, k0, 0, 0, m / 16, t.e, bar);
                            } else if (KIND == kForward) {
                                tma_pair_3d(a, &maps.a, k0, m, t.e, bar);
                            } else if (awhole) {
                                tma_pair_4d(a, &maps.a, 0, k0, m / 64, t.e, bar);
                            } else {
                                tma_pair_3d(a, &maps.a, m, k0, t.e, bar);
                                tma_pair_3d(a + kABytes / 2, &maps.a, m + 64, k0, t.e, bar);
                            }
                            tma_pair_2d(b, &maps.b[half / 16 - 1], k0, brow, bar);
                        }
                    }
                    __syncwarp();
                }
            }
            // The MMAs' last arrivals are here before the block ends: they come from the pair's other block.
            for (uint32_t j = it < kStages ? 0 : it - kStages; ok && j < it; ++j)
                ok = mbar_wait(empty + 8 * (j % kStages), (j / kStages) & 1, gave_up);
            if (!ok && rank == 0) {  // given up: the copies in flight end before the block does
                const uint64_t start = global_ns();
                for (uint32_t j = it < kStages ? 0 : it - kStages; j < it; ++j)
                    while (!mbar_try_wait(full + 8 * (j % kStages), (j / kStages) & 1) &&
                           global_ns() - start < 1000000000ull) {
                    }
            }
        } else if (warp == 1 && rank == 0) {
            // ---- MMAs of the pair
            uint32_t it = 0, done = 0;
            bool ok = true;
            Walk<KIND> walk;
            for (uint64_t i = pair; i < g.total && ok; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                if (t.blocks == 0) continue;
                uint32_t buf = 0, d = 0;
                const bool parts = in_parts<KIND, F32, CUT>(t.blocks);
                const uint32_t instr = bf16_instr_desc(kTileM, t.width, KIND != kForward, KIND == kWeight);
                for (int kb = 0; kb < t.blocks; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    // a new sum: the tile's, or a part of it
                    const bool first = kb == 0 || (parts && kb % kSeg == 0);
                    const bool last = kb == t.blocks - 1 || (parts && kb % kSeg == kSeg - 1);
                    if (first) {
                        buf = done & 1;
                        d = tmem + buf * kTileN;
                        if (!mbar_wait(acc_empty + 8 * buf, ((done >> 1) & 1) ^ 1, gave_up)) {
                            ok = false;
                            break;
                        }
                        ++done;
                    }
                    if (!mbar_wait(full + 8 * s, (it / kStages) & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_addr(stages) + s * kStageBytes, b = a + kABytes;
                    // 16 values of the summed index: 32 bytes along a row, or 16 rows of 128 bytes
                    const uint64_t da = KIND == kForward ? operand_desc(a) : operand_desc_mn(a, kABytes / 2);
                    const uint64_t db = KIND != kWeight ? operand_desc(b) : operand_desc_mn(b, 64 * 128);
                    constexpr uint64_t sa = (KIND == kForward ? 32 : 16 * 128) >> 4;
                    constexpr uint64_t sb = (KIND != kWeight ? 32 : 16 * 128) >> 4;
                    // of a tail the 16 values that hold its last row are the last
                    const int steps = KIND == kWeight && t.tail != 0 && kb == t.blocks - 1 ? (t.tail + 15) / 16 : kBlockK / 16;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < kBlockK / 16; ++j)
                            if (KIND != kWeight || j < steps)
                                mma_pair_bf16(d, da + j * sa, db + j * sb, instr, !first || j > 0);
                        mma_commit_pair(empty + 8 * s);
                        if (last) mma_commit_pair(acc_full + 8 * buf);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // given up: the MMAs in flight end before the TMEM is freed
                if (elect_one()) mma_commit_pair(drain);
                __syncwarp();
                const uint64_t start = global_ns();
                while (!mbar_try_wait(drain, 0) && global_ns() - start < 1000000000ull) {
                }
            }
        } else if (warp == 2 && KIND == kWeight) {
            // ---- tails: zeros in the rows behind the segment
            const uint32_t bar0 = cluster_addr(full, 0);
            uint32_t it = 0, phases = 0;  // a stage's bit: the parity of its tail barrier
            TileWait since;
            Walk<KIND> walk;
            for (uint64_t i = pair; i < g.total; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                it += t.blocks;
                since.enter(t.blocks);
                if (t.blocks == 0 || t.tail == 0) continue;
                const uint32_t s = (it - 1) % kStages;
                if (!mbar_wait(tail + 8 * s, (phases >> s) & 1, gave_up, since.limit())) break;
                since.waited();
                phases ^= 1u << s;
                uint8_t* a = stages + s * kStageBytes;
                const int boxes = 2 + t.width / 128;  // of 64 rows x 128 bytes, A's and B's
                const int end = (t.tail + 15) / 16 * 16 * 8;  // the MMAs stop there
                for (int q = t.tail * 8 + lane; q < end; q += 32)
                    for (int j = 0; j < boxes; ++j)
                        reinterpret_cast<uint4*>(a + j * 8192)[q] = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                // the zeros are in this block's shared memory, where its tensor core
                // reads them: a release at cluster scope took 2,000 cycles per tail
                if (lane == 0) mbar_arrive_pair(bar0 + 8 * s);
            }
        }
    } else {
        if (CUT) registers_up<kAddRegs>();
        // ---- output
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t slot = smem_addr(slots) + (warp - 4) * kStaging;
        const uint32_t bar0 = cluster_addr(acc_empty, 0);
        constexpr int kReads = KIND == kInput && SWIGLU ? 2 : 1, kReadPieces = kGated ? 2 : 4;
        uint32_t done = 0;
        Walk<KIND> walk;
        if constexpr (F32) {
            bool ok = true;
            for (uint64_t i = pair; i < g.total && ok; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                const int share = t.width / 2, c0 = ((warp >> 2) - 1) * share;  // this warp's columns
                float acc[8][16];
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c][j] = 0.0f;
                for (int kb = 0; kb < t.blocks; kb += kSeg, ++done) {
                    const uint32_t buf = done & 1, src = lanes + buf * kTileN + c0;
                    if (!mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        if (c * 16 >= share) break;
                        uint32_t v[2][16];
                        tmem_load(v[0], src + c * 16);
                        tmem_load(v[1], src + c * 16 + 16);  // of an odd share: columns past it, not used
                        tmem_wait_for(v[0]);
                        tmem_wait_for(v[1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            acc[c][j] += __uint_as_float(v[0][j]);
                            acc[c + 1][j] += __uint_as_float(v[1][j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(bar0 + 8 * buf);
                }
                if (!ok) break;
                if (KIND == kWeight)
                    write_weights(acc, p, maps.b[1], slot, t, t.m0 + (int)rank * 128 + quarter * 32, t.n0 + c0, share, N, K);
                else
                    write_tokens(acc, p, slot, t, t.m0 + (int)rank * 128 + quarter * 32, c0, share, g.channels);
            }
            if (KIND == kWeight && lane == 0) tma_store_wait<0>();
        } else if constexpr (KIND == kWeight) {
            // bf16: a lane is a row of dw; 128 bytes of each row go through a box in shared memory to a TMA store
            bool ok = true;
            for (uint64_t i = pair; i < g.total && ok; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                const int n = t.m0 + (int)rank * 128 + quarter * 32;              // the warp's first row
                const int cols = min(t.width, K - t.n0);                          // a multiple of 8
                const int share = t.width / 2, c0 = ((warp >> 2) - 1) * share;    // this warp's columns
                if (!in_parts<KIND, F32, CUT>(t.blocks)) {
                    const uint32_t buf = done & 1, src = lanes + buf * kTileN;
                    if (t.blocks > 0) {
                        if (!mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, gave_up, tile_limit(t.blocks))) break;
                        tc_fence_after();
                        ++done;
                    }
                    for (int c = c0; c < c0 + share; c += 64) {
                        uint32_t v[4][16] = {};
                        if (t.blocks > 0) {
                            __syncwarp();
#pragma unroll
                            for (int h = 0; h < 4; ++h) tmem_load(v[h], src + c + h * 16);
#pragma unroll
                            for (int h = 0; h < 4; ++h) tmem_wait_for(v[h]);
                            if (c + 64 >= c0 + share) {  // the buffer's last sums are in registers
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive_pair(bar0 + 8 * buf);
                            }
                        }
                        float f[4][16];
#pragma unroll
                        for (int h = 0; h < 4; ++h) as_floats(v[h], f[h]);
                        if (n < N && c < cols)
                            write_weights_bf16(f, p, maps.b[1], slot, t.e, n, t.n0 + c, cols - c, N, K);
                    }
                    continue;
                }
                float acc[8][16];
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c][j] = 0.0f;
                for (int kb = 0; kb < t.blocks; kb += kSeg, ++done) {
                    const uint32_t buf = done & 1, src = lanes + buf * kTileN + c0;
                    if (!mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        if (c * 16 >= share) break;
                        uint32_t v[2][16];
                        tmem_load(v[0], src + c * 16);
                        tmem_load(v[1], src + c * 16 + 16);  // of an odd share: columns past it, not used
                        tmem_wait_for(v[0]);
                        tmem_wait_for(v[1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            acc[c][j] += __uint_as_float(v[0][j]);
                            acc[c + 1][j] += __uint_as_float(v[1][j]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(bar0 + 8 * buf);
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < 8; c += 4) {
                    if (c * 16 >= share) break;
                    float f[4][16];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[h][j] = acc[c + h][j];
                    const int at = c0 + c * 16;
                    if (n < N && at < cols)
                        write_weights_bf16(f, p, maps.b[1], slot, t.e, n, t.n0 + at, cols - at, N, K);
                }
            }
            if (lane == 0) tma_store_wait<0>();
        } else {
            // Lanes are channels, columns tokens, read in an mma accumulator's layout.  A whole sum goes from TMEM through
            // four warps; sums in parts are added here, rounded, by eight, and each four have half of the tile's chunks
            // of 32 tokens.
            bool ok = true;
            for (uint64_t i = pair; i < g.total && ok; i += step) {
                const Tile t = walk.tile(sh, g, p.E, i);
                const int span = kGated ? 16 : 32;  // output channels of this warp
                const int ch = t.m0 + (int)rank * (g.per / 2) + quarter * span;
                const int chans = min(span, g.channels - ch);
                const int first = CUT ? (t.width + 32) / 64 * 32 : t.width;  // columns of the first four warps
                const int c0 = warp < 8 ? 0 : first, end = warp < 8 ? min(t.n, first) : t.n;
                // What the epilogue reads (a residual, or the pre-activations of gate and up) is asked for a chunk of 32
                // tokens ahead, the first one before the sums are there.
                Rows<kReadPieces> ahead[kReads];
                auto ask = [&](int c) {
                    if (c >= end || chans <= 0) return;
                    const int tokens = min(32, end - c);
                    const int64_t row = t.row + c;
                    if (KIND == kInput && SWIGLU) {
                        const uint16_t* z = p.z + row * 2 * K + ch;
                        ahead[0].load(z, (int64_t)K * 4, tokens, chans * 2);
                        ahead[kReads - 1].load(z + K, (int64_t)K * 4, tokens, chans * 2);
                    } else if (KIND == kForward && p.residual) {
                        ahead[0].load(static_cast<const uint16_t*>(p.residual) + row * g.channels + ch,
                                      (int64_t)g.channels * 2, tokens, chans * 2);
                    }
                };
                float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // biases of this lane's channels
                if (KIND == kForward && p.bias) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = 8 * j + lane / 4;  // TMEM lane of the warp
                        const int n = kGated ? ch + k % 16 + (j >= 2 ? g.channels : 0) : ch + k;
                        if (kGated || n < g.channels) b[j] = load_typed(p.bias, p.bias_type, n);
                    }
                }
                auto finish = [&](float (&f)[2][16], int c) {  // the sums of tokens c..
                    const int tokens = min(32, end - c);
                    const int64_t row = t.row + c;
                    if (KIND == kForward && p.bias) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            f[0][j] += b[(j >> 1) & 1];
                            f[1][j] += b[2 + ((j >> 1) & 1)];
                        }
                    }
                    uint16_t* out = static_cast<uint16_t*>(p.out);
                    if (kGated) {
                        if (p.z) {
                            uint16_t* z = p.z + row * N + ch;
                            put_fragments<2>(slot, 0, f[0]);
                            put_fragments<2>(slot + kSlot / 2, 0, f[1]);
                            write_rows<2>(slot, z, N, tokens, 16);
                            write_rows<2>(slot + kSlot / 2, z + g.channels, N, tokens, 16);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[0][j] = swiglu(f[0][j], f[1][j]);
                        if (p.residual) {
                            ahead[0].put(slot + 3 * kSlot / 2);
                            ask(c + 32);
                            get_fragments<2>(slot + 3 * kSlot / 2, 0, f[1]);
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[0][j] += f[1][j];
                        }
                        put_fragments<2>(slot + kSlot, 0, f[0]);
                        write_rows<2>(slot + kSlot, out + row * g.channels + ch, g.channels, tokens, 16);
                    } else if (KIND == kInput && SWIGLU) {
                        ahead[0].put(slot);
                        ahead[kReads - 1].put(slot + kSlot);
                        ask(c + 32);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float gate[16], up[16];
                            get_fragments<4>(slot, h, gate);
                            get_fragments<4>(slot + kSlot, h, up);
#pragma unroll
                            for (int j = 0; j < 16; ++j) swiglu_back(gate[j], up[j], f[h][j], gate[j], up[j]);
                            // a lane's fragments of one half are its own to overwrite once all lanes have read theirs
                            __syncwarp();
                            put_fragments<4>(slot, h, gate);
                            put_fragments<4>(slot + kSlot, h, up);
                        }
                        uint16_t* dz = out + row * 2 * K + ch;
                        write_rows<4>(slot, dz, 2 * K, tokens, chans);
                        write_rows<4>(slot + kSlot, dz + K, 2 * K, tokens, chans);
                    } else {
                        const int64_t at = row * g.channels + ch;
                        if (KIND == kForward) {
                            if (p.z) {
                                put_fragments<4>(slot, 0, f[0]);
                                put_fragments<4>(slot, 1, f[1]);
                                write_rows<4>(slot, p.z + at, g.channels, tokens, chans);
                            }
                            activate16(f[0], p.activation);
                            activate16(f[1], p.activation);
                            if (p.residual) {
                                ahead[0].put(slot + kSlot);
                                ask(c + 32);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float r[16];
                                    get_fragments<4>(slot + kSlot, h, r);
#pragma unroll
                                    for (int j = 0; j < 16; ++j) f[h][j] += r[j];
                                }
                            }
                        }
                        __syncwarp();
                        put_fragments<4>(slot, 0, f[0]);
                        put_fragments<4>(slot, 1, f[1]);
                        write_rows<4>(slot, out + at, g.channels, tokens, chans);
                    }
                };
                if constexpr (CUT) {
                    float acc[4][2][16];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c][0][j] = acc[c][1][j] = 0.0f;
                    for (int kb = 0; kb < t.blocks; kb += kSeg, ++done) {
                        const uint32_t buf = done & 1, src = lanes + buf * kTileN + c0;
                        if (kb + kSeg >= t.blocks) ask(c0);
                        if (!mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, gave_up)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c0 + c * 32 >= end || chans <= 0) break;
                            uint32_t v[2][16];
                            tmem_load_16x256(v[0], src + c * 32);
                            tmem_load_16x256(v[1], src + c * 32 + (16u << 16));
                            tmem_wait_for(v[0]);
                            tmem_wait_for(v[1]);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                acc[c][0][j] += __uint_as_float(v[0][j]);
                                acc[c][1][j] += __uint_as_float(v[1][j]);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(bar0 + 8 * buf);
                    }
                    if (!ok) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c0 + c * 32 >= end || chans <= 0) break;
                        finish(acc[c], c0 + c * 32);
                    }
                } else {
                    const uint32_t buf = done & 1, src = lanes + buf * kTileN;
                    ask(0);
                    if (!mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, gave_up, tile_limit(t.blocks))) break;
                    tc_fence_after();
                    auto release = [&]() {  // the buffer's last sums are in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(bar0 + 8 * buf);
                    };
                    if (chans <= 0) release();
                    for (int c = 0; c < end && chans > 0; c += 32) {
                        uint32_t v[2][16];
                        __syncwarp();
                        tmem_load_16x256(v[0], src + c);
                        tmem_load_16x256(v[1], src + c + (16u << 16));
                        tmem_wait_for(v[0]);
                        tmem_wait_for(v[1]);
                        if (c + 32 >= end) release();
                        float f[2][16];
                        as_floats(v[0], f[0]);
                        as_floats(v[1], f[1]);
                        finish(f, c);
                    }
                    ++done;
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && sh.gave_up && p.status) atomicOr(p.status, EP_FLAG_TIMEOUT);
    cluster_sync();  // no copy, arrival or MMA of the other block reaches this one any more
    if (warp == 0) tmem_dealloc_pair(tmem, 512);
    cluster_sync();  // the release is a pair's: neither block leaves its SM to another kernel before both are through
}

}  // namespace

DensePlan dense_plan(int64_t M, int64_t K, int64_t channels, bool gated, bool split) {
    static std::atomic<int> sm_cache[64];
    const int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    const int64_t pairs = sms >= 2 ? sms / 2 : 1;
    // The search takes some 5 us, and a layer asks for the same sizes again and again.
    struct Known {
        int64_t M, K, channels, rest;
        DensePlan plan;
    };
    static thread_local Known known[16];
    const int64_t rest = pairs * 4 + gated * 2 + split;
    Known& at = known[(uint64_t)(M * 31 + K * 7 + channels * 3 + rest) % 16];
    if (at.M == M && at.K == K && at.channels == channels && at.rest == rest) return at.plan;
    // Cycles of a stage for 32, 64, .. 256 columns, measured on a dense layer of
    // 4,096 channels: the narrow ones wait for the weights from L2.  Input products, whose
    // weights lie the other way, are planned by the same figures.
    static const int stage[8] = {276, 285, 311, 330, 357, 421, 458, 512};
    // the second pass: its launch behind the first (some 3 us), and as much again on the host
    constexpr double kFinishCycles = 9000.0;
    const int64_t blocks = (K + kBlockK - 1) / kBlockK;
    // parts are products with all rows of w alike, written and read again in fp32
    const int64_t rows = gated ? 2 * channels : channels, mtiles = (rows + kTileM - 1) / kTileM;
    struct Parts {
        int64_t count, per, mtiles;
        double more;
    } parts[16];
    int kinds = 0;
    for (int64_t want = 1; want <= (split ? 16 : 1) && (want == 1 || want * 4 <= blocks); ++want) {
        const int64_t per = (blocks + want - 1) / want;
        if ((blocks + per - 1) / per != want) continue;
        if (want == 1)
            parts[kinds++] = {1, per, gated ? (channels + kTileM / 2 - 1) / (kTileM / 2) : mtiles, 0.0};
        else
            parts[kinds++] = {want, per, mtiles, kFinishCycles + (double)(want * M) * (double)rows * 8.0 / 4000.0};
    }
    DensePlan best = {kTileN, 1};
    double least = 0.0;
    for (int u = 8; u >= 1; --u) {
        const int64_t tokens = (M + 32 * u - 1) / (32 * u);
        for (int i = 0; i < kinds; ++i) {
            const int64_t rounds = (parts[i].mtiles * tokens * parts[i].count + pairs - 1) / pairs;
            const double cost = (double)rounds * (double)(parts[i].per * stage[u - 1] + 400) + 2000.0 + 400.0 * u + parts[i].more;
            if (least == 0.0 || cost < least * 0.98) {
                least = cost;
                best = {32 * u, (int)parts[i].count};
            }
        }
    }
    at = {M, K, channels, rest, best};
    return best;
}

// Blocks of 64 tokens x 64 channels of a row-major matrix; `two`: a copy is two
// such blocks, side by side in the matrix and one after the other in shared memory.
static cudaError_t token_blocks_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t width, bool two) {
    if (two) {
        const uint64_t d[3] = {64, rows, width / 64}, s[2] = {width * 2, 128};
        const uint32_t box[3] = {64, 64, 2};
        return typed_map(map, EP_TYPE_BF16, base, 3, d, s, box);
    }
    const uint64_t d[2] = {width, rows}, s[1] = {width * 2};
    const uint32_t box[2] = {64, 64};
    return typed_map(map, EP_TYPE_BF16, base, 2, d, s, box);
}

// Tiles of 256 columns, or of 128 (a block of the summed index then takes 420 cycles
// instead of 530, for half of the columns), and parts of the rows where the tiles
// alone leave pairs without work.  The costs are fitted to 18 sizes by up to 12
// numbers of parts; of these the rule takes the fastest, or at most 12 % more.
// One part of the rows and what the rule takes, in us: 65,536 rows to 256 x 7,168 (28
// tiles of 1,024 blocks) 274 and 172; 32,768 to 512 x 2,048 136 and 53; 4,096 to
// 1,024 x 1,024 22.8 and 16.3; 9,000 to 8 x 8 39.3 and 9.9.  4,096 to 2,816 x 2,048
// stays whole: 45.0, and 46.1 in two parts.
DensePlan weight_plan(int64_t M, int64_t N, int64_t K, bool split) {
    static std::atomic<int> sm_cache[64];
    const int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    const int64_t pairs = sms >= 2 ? sms / 2 : 1, blocks = (M + kBlockK - 1) / kBlockK;
    const int64_t mtiles = (N + kTileM - 1) / kTileM;
    DensePlan best = {K <= 128 ? 128 : kTileN, 1};
    double least = 0.0;
    for (int columns = best.most; columns >= 128; columns -= 128) {
        const int64_t tiles = mtiles * ((K + columns - 1) / columns);
        for (int64_t want = 1; want <= (split ? 16 : 1) && (want == 1 || want * 4 <= blocks); ++want) {
            const int64_t per = (blocks + want - 1) / want;
            if (want > 1 && (blocks + per - 1) / per != want) continue;
            const int64_t rounds = (tiles * want + pairs - 1) / pairs;
            double cost = (double)rounds * (double)(per * (columns == 128 ? 420 : 530) + 2500);
            if (want > 1) cost += 1500.0 + (double)want * (double)N * (double)K * 8.0 / 6000.0;
            if (least == 0.0 || cost < least * 0.95) {
                least = cost;
                best = {columns, (int)want};
            }
        }
    }
    return best;
}

cudaError_t launch_product(const ProductArgs& p, ProductKind kind, cudaStream_t stream) {
    const bool swiglu = p.activation == EP_ACT_SWIGLU;
    const int most = p.most ? p.most : kind == kWeight && p.K <= 128 ? 128 : kTileN;
    Maps maps;
    const uint64_t N = (uint64_t)p.N, K = (uint64_t)p.K, E = (uint64_t)p.E, rows = (uint64_t)p.rows;
    cudaError_t err = cudaSuccess;
    if (kind == kWeight) {
        // no rows at all: nothing is loaded, and any address will do
        const void* dy = rows ? static_cast<const void*>(p.a) : p.out;
        const void* x = rows ? static_cast<const void*>(p.b) : p.out;
        err = token_blocks_map(&maps.a, dy, rows ? rows : 1, N, N % 64 == 0);
        if (err == cudaSuccess) err = token_blocks_map(&maps.b[0], x, rows ? rows : 1, K, K % 64 == 0 && most == kTileN);
        const bool f32 = p.out_type == EP_TYPE_F32;
        const uint64_t size = f32 ? 4 : 2;
        const uint64_t dc[3] = {K, N, E}, sc[2] = {K * size, N * K * size};
        const uint32_t cbox[3] = {f32 ? 32u : 64u, 32, 1};
        if (err == cudaSuccess) err = typed_map(&maps.b[1], p.out_type, p.out, 3, dc, sc, cbox);
    } else {
        if (kind == kForward && swiglu) {
            const uint64_t I = N / 2;
            const uint64_t d[5] = {K, 16, 2, I / 16, E}, s[4] = {K * 2, I * K * 2, 16 * K * 2, N * K * 2};
            const uint32_t box[5] = {64, 16, 2, 4, 1};
            err = typed_map(&maps.a, EP_TYPE_BF16, p.b, 5, d, s, box);
        } else if (kind == kInput && K % 64 == 0) {
            const uint64_t d[4] = {64, N, K / 64, E}, s[3] = {K * 2, 128, N * K * 2};
            const uint32_t box[4] = {64, 64, 2, 1};
            err = typed_map(&maps.a, EP_TYPE_BF16, p.b, 4, d, s, box);
        } else {
            const uint64_t d[3] = {K, N, E}, s[2] = {K * 2, N * K * 2};
            const uint32_t box[3] = {64, kind == kForward ? 128u : 64u, 1};
            err = typed_map(&maps.a, EP_TYPE_BF16, p.b, 3, d, s, box);
        }
        const uint64_t width = kind == kForward ? K : N;
        const uint64_t d[2] = {width, rows}, s[1] = {width * 2};
        // the boxes that a tile of these rows can ask for
        const uint32_t widest = (uint32_t)((rows < (uint64_t)most ? rows + 31 : (uint64_t)most) / 32);
        for (uint32_t j = 0; j < widest && err == cudaSuccess; ++j) {
            const uint32_t box[2] = {64, 16 * (j + 1)};
            err = typed_map(&maps.b[j], EP_TYPE_BF16, p.a, 2, d, s, box);
        }
    }
    if (err != cudaSuccess) return err;
    static std::atomic<int> sm_cache[64];
    const int sms = cached_device_attribute(cudaDevAttrMultiProcessorCount, sm_cache);
    const bool f32 = p.out_type == EP_TYPE_F32;
    const bool cut = f32 || kind == kWeight || (kind == kForward ? p.K : p.N) > kBlockK * kWholeBlocks;
    static std::atomic<uint64_t> configured[11];
    const int which = kind == kWeight ? f32 : f32 ? 2 : 3 + (kind == kInput) * 4 + swiglu * 2 + cut;
    auto kernel = which == 0   ? product_kernel<kWeight, false, false, true>
                  : which == 1 ? product_kernel<kWeight, false, true, true>
                  : which == 2 ? product_kernel<kForward, false, true, true>
                  : which == 3 ? product_kernel<kForward, false, false, false>
                  : which == 4 ? product_kernel<kForward, false, false, true>
                  : which == 5 ? product_kernel<kForward, true, false, false>
                  : which == 6 ? product_kernel<kForward, true, false, true>
                  : which == 7 ? product_kernel<kInput, false, false, false>
                  : which == 8 ? product_kernel<kInput, false, false, true>
                  : which == 9 ? product_kernel<kInput, true, false, false>
                               : product_kernel<kInput, true, false, true>;
    const size_t smem = smem_bytes(cut);
    err = raise_smem_limit(kernel, smem, configured[which]);
    if (err != cudaSuccess) return err;
    const unsigned grid = sms >= 2 ? (unsigned)(sms & ~1) : 2u;
    // An ordinary launch, and no early one of what follows.  As programmatic launches a
    // chain elementwise pass, input product, weight product came to a stop.  By reading:
    // blocks of another kernel were started on one SM of a pair while the other still
    // released its TMEM.  Mended together, and not told apart: this, the barrier after the
    // release, the loading warp's wait for the MMAs' last arrivals in the other block, and
    // a warp's reconvergence before a cluster barrier.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads_of(cut));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, most);
}

}  // namespace ep
