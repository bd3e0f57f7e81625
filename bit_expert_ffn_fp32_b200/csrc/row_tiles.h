// How an expert's rows are spread over tiles (plain C++, so that it is tested on
// the host at row counts no test can run).
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// Tiles of at most tn rows that `rows` (up to 2^31 - 4096) take.
MOE_HD int row_tiles(int rows, int tn) { return (rows + tn - 1) / tn; }

// Rows of a tile: spread evenly over the tiles, in multiples of 16. Nothing here
// passes 32 bits: rows is not rounded up before the division.
MOE_HD int rows_per_tile(int rows, int tiles, int tn) {
    return tiles == 1 ? tn : ((rows - 1) / tiles + 16) & ~15;
}

// Columns of the products of n columns by cg CTAs together: an M = 128 product
// takes multiples of 16, one of M = 256 by a pair of CTAs multiples of 32.
MOE_HD int padded_columns(int n, int cg) { return (n + 16 * cg - 1) & ~(16 * cg - 1); }

}  // namespace moe
