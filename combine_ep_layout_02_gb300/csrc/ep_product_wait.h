// ep_product_wait.h -- how long the product kernel's waits may last: plain
// arithmetic that the kernel and a host compiler share.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EP_WAIT __host__ __device__ __forceinline__ constexpr
#else
#define EP_WAIT constexpr
#endif

namespace ep {

// A wait that spans whole tiles: a second, 2 us per block of the summed index (0.25
// to 0.4 us measured) and 100 us per tile for its output (5 us, with an addend 20).
EP_WAIT uint64_t tile_limit(uint64_t blocks, uint64_t tiles = 0) {
    return 1000000000ull + 2000ull * blocks + 100000ull * tiles;
}

// The same for a warp that waits in some of its tiles only: a wait spans the tiles
// since the last one.
struct TileWait {
    uint64_t blocks = 0, tiles = 0;
    EP_WAIT void enter(int blocks_of_tile) {
        blocks += (uint64_t)blocks_of_tile;
        ++tiles;
    }
    EP_WAIT uint64_t limit() const { return tile_limit(blocks, tiles); }
    EP_WAIT void waited() { blocks = tiles = 0; }
};

}  // namespace ep
