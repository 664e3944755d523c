// moe_tiles.h -- which tiles of rows and outputs the grouped products on the tensor cores have
// (moe_gemm_tc.cu); plain arithmetic, for the host as well.
//
// Expert e has ceil(rows / columns) tiles of rows, cum[e] tiles lie before its own, cum[n_experts] is their number.
// A plan may come from elsewhere and its offsets may overlap, which would ask for more tiles than the workspace
// has cells: every entry of cum is cut to that, so that a tile of any item is a cell of the workspace.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define RZ_TILES_FN __host__ __device__ __forceinline__
#else
#define RZ_TILES_FN inline
#endif

namespace rz {

// The most tiles that so many rows of so many experts can have.
RZ_TILES_FN int64_t moe_most_tiles(int64_t n_pairs, int n_experts, int columns) { return n_pairs / columns + (n_pairs < n_experts ? n_pairs : n_experts); }

// Tiles of the expert whose rows are lo .. hi; none where those are not rows.  At most moe_most_tiles.
RZ_TILES_FN int moe_expert_tiles(int lo, int hi, int n_pairs, int columns)
{
    return lo >= 0 && hi > lo && hi <= n_pairs ? (hi - lo - 1) / columns + 1 : 0;
}

// `before` cut to `most`.  Sums of 32 experts stay below 2^31 when they start from such a value: 33 (2^27 / 16 + 512).
RZ_TILES_FN int moe_cut(int before, int most) { return before < most ? before : most; }

// The expert of tile i < cum[n_experts].
RZ_TILES_FN int moe_expert_of(int i, const int *cum, int n_experts)
{
    int lo = 0, hi = n_experts;  // cum[lo] <= i < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Item `it` of cum[n_experts] * row_tiles: tiles of outputs after one another, the expert's tiles of rows within.
struct MoeItem {
    int expert, row_tile, tile;  // tile: among the expert's, cell cum[expert] + tile of the workspace
};
RZ_TILES_FN MoeItem moe_item(int64_t it, int row_tiles, const int *cum, int n_experts)
{
    MoeItem m;
    m.expert = moe_expert_of(static_cast<int>(it / row_tiles), cum, n_experts);
    const int tiles = cum[m.expert + 1] - cum[m.expert];
    const int64_t at = it - static_cast<int64_t>(cum[m.expert]) * row_tiles;
    m.row_tile = static_cast<int>(at / tiles);
    m.tile = static_cast<int>(at - static_cast<int64_t>(m.row_tile) * tiles);
    return m;
}

}  // namespace rz
