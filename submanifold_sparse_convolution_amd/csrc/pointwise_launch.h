// Tile choice of the product kernel (included by the files that instantiate it).
#pragma once

#include "pointwise_gemm.h"

namespace smc {

// One per operand layout and epilogue family (their own files: they compile
// in parallel).
hipError_t launch_store_16(const ProductArgs& p, int dt, hipStream_t s);
hipError_t launch_gated_16(const ProductArgs& p, int dt, hipStream_t s);
hipError_t launch_slope_16(const ProductArgs& p, int dt, hipStream_t s);
hipError_t launch_gated_slope_16(const ProductArgs& p, int dt, hipStream_t s);
hipError_t launch_store_e4m3(const ProductArgs& p, int dt, bool along, hipStream_t s);
hipError_t launch_gated_e4m3(const ProductArgs& p, int dt, bool along, hipStream_t s);
// Up to kFewRows rows, aligned gated layers 4 (kEpiStore, kEpiGated; 16-bit operands).
hipError_t launch_few_rows(const ProductArgs& p, Epilogue epi, int dt, hipStream_t s);

namespace {

// Tile by the number of tiles (bf16, us on the GPU, silu unless noted).
// Small (32 x 64, six steps ahead) while two of them a CU are enough: one round
// of blocks, each with little work, and the latency of its loads well covered.
//   c_in -> 512, rows        Small   Rows   Mid
//   128   1,024                4.5    4.9   6.0
//   512   1,024 / 2,048    6.5/7.9 7.2/7.3 9.1/9.3
//   2048  2,048 / 3,000  15.9/26.0 19.1/19.6 22.4/22.7
//   gated 512 -> 1024, 512 / 768 rows: Small 7.7 / 10.8, Wide 8.3 / 8.4
//   unaligned 141 -> 141, 4,000 rows: Small 16.4, Rows 18.1; 20,000 x 141 -> 525: 89.6, 59.3
// Rows (64 x 128, three blocks a CU) or Mid (128 x 128, two), Rows / Mid in us:
// - up to one Mid tile a CU, Rows: Mid would leave CUs idle. 512 -> 512, 3,000 / 6,000
//   rows 8.3 / 9.8, 9.5 / 10.4; 512 -> 256, 15,000 rows 8.9 / 10.1.
// - up to one round of Mid, Rows if it takes one too: 40,000 x 64 -> 128 7.2 / 7.6,
//   200 -> 64 9.0 / 9.4, with a residual 9.9 / 11.1; but where Rows needs a second round:
//   50,000 x 128 -> 64 8.9 / 8.2, 512 -> 128 17.0 / 15.3; 512 -> 512, 15,000 rows 15.5 / 13.5.
// - beyond, Mid, whose waves read less from LDS for a product: 512 -> 512, 30,000 rows
//   25.2 / 23.7; 91,000 x 128 -> 64 13.2 / 12.2, -> 256 21.0 / 20.7 - except with a residual (or dy) and contractions of up to 256, where a
//   tile is mostly epilogue and three blocks overlap it: 91,000 x 128 -> 64 / 128 / 256 /
//   384 / 512 15.2 / 16.5, 16.9 / 17.6, 25.6 / 25.9, 33.3 / 36.0, 42.1 / 46.3, 192 -> 512 50.0 /
//   55.3, 256 -> 256 32.8 / 32.8; and one column tile of a longer contraction or with a
//   residual: 91,000 x 512 -> 64 20.8 / 23.2, with it 23.8 / 26.5.
// (With three steps in flight and two blocks a CU: 2048 -> 512, 3,000 rows 18.0, but
// 512 -> 512, 6,000 and 8,000 rows 10.2 and 10.8 against 9.5 and 9.7.)
// Unaligned operands, which go through registers, leave Mid too few of them.
// Gated: Wide, 32 x 64 a wave, twice the waves to overlap the epilogues of both
// halves; long 16-bit contractions in Mid, whose waves read less from LDS for a
// product. 91,000 x 128 -> 344: Wide 35.4, Mid 36.9; e4m3 15,000 x 512 -> 2048:
// 50.6, 53.5; bf16 4,096 x 512 -> 1024 and 15,000 x 512 -> 2048: 13.9 and 74.3,
// 12.5 and 69.0. (Slopes only in Wide.)
template <int DT, bool E4M3, int LA, int LB, int EPI>
hipError_t launch_tiled(const ProductArgs& p, hipStream_t s) {
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    const int64_t cus = device_cus();
    const int64_t small = ((p.m + 31) / 32) * (int64_t)((p.n + 63) / 64);
    const int64_t mid = ((p.m + 127) / 128) * (int64_t)((p.n + 127) / 128);
    if (small <= 2 * cus) return launch_product<DT, E4M3, LA, LB, EPI, TileSmall>(p, s);
    if constexpr (kGated) {
        if constexpr (EPI == kEpiGated && !E4M3)
            if (p.k >= 256 && p.vec_a && p.vec_b) return launch_product<DT, E4M3, LA, LB, EPI, TileMid>(p, s);
        return launch_product<DT, E4M3, LA, LB, EPI, TileWide>(p, s);
    } else {
        const int64_t rows = ((p.m + 63) / 64) * (int64_t)((p.n + 127) / 128);
        const bool one_round = mid <= 2 * cus;
        const bool narrow = p.n <= 128 && p.k > 256, epilogue = p.extra && (p.k <= 256 || p.n <= 128);
        if (mid <= cus || (one_round ? rows <= 3 * cus : narrow || epilogue) || !p.vec_a || !p.vec_b)
            return launch_product<DT, E4M3, LA, LB, EPI, TileRows>(p, s);
        return launch_product<DT, E4M3, LA, LB, EPI, TileMid>(p, s);
    }
}

}  // namespace
}  // namespace smc
