// row_blocks.h -- how the bias gradient's kernel deals rows over its blocks.  Host and device code; plain C++.
#pragma once
#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define MLPL_HD __host__ __device__
#else
#define MLPL_HD
#endif

namespace mlpl {

constexpr int kStrip = 256;    // columns per CTA: 32 lanes x 8

// Rows per block: about four CTAs per SM, at least 16 rows (two per warp).
inline int32_t grad_block_rows(int64_t N, int num_sms, int64_t rows)
{
    auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t blocks = std::max<int64_t>(1, cdiv(4 * num_sms, cdiv(N, kStrip)));
    return static_cast<int32_t>(std::max<int64_t>(16, cdiv(cdiv(rows, blocks), 8) * 8));
}

// End of the block that starts at row lo < rows.  (lo + block_rows could wrap.)
MLPL_HD inline int32_t block_end(int32_t lo, int32_t block_rows, int32_t rows)
{
    return block_rows < rows - lo ? lo + block_rows : rows;
}

}  // namespace mlpl
