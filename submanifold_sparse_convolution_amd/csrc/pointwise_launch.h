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
// Up to kFewRows rows (kEpiStore, kEpiGated; 16-bit operands).
constexpr int kFewRows = 8;
hipError_t launch_few_rows(const ProductArgs& p, Epilogue epi, int dt, hipStream_t s);

namespace {

template <int DT, bool E4M3, int LA, int LB, int EPI>
hipError_t launch_tiled(const ProductArgs& p, hipStream_t s) {
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    const bool words = p.vec_a && p.vec_b;
    const int rows = words ? 128 : 64;          // of the tile that would be taken
    const int64_t tiles = ((p.m + rows - 1) / rows) * (int64_t)((p.n + 127) / 128);
    if (tiles < device_cus() / 2) return launch_product<DT, E4M3, LA, LB, EPI, TileSmall>(p, s);
    if constexpr (kGated) {
        return launch_product<DT, E4M3, LA, LB, EPI, TileWide>(p, s);
    } else {
        if (p.n <= 128 || !words) return launch_product<DT, E4M3, LA, LB, EPI, TileRows>(p, s);
        return launch_product<DT, E4M3, LA, LB, EPI, TileMid>(p, s);
    }
}

}  // namespace
}  // namespace smc
