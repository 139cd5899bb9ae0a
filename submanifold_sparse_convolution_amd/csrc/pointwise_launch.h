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

namespace {

template <int DT, bool E4M3, int LA, int LB, int EPI>
hipError_t launch_tiled(const ProductArgs& p, hipStream_t s) {
    const int64_t cus = device_cus();
    const int64_t mid = ((p.m + 127) / 128) * ((p.n + 127) / 128) * p.splits;
    if (mid >= cus) return launch_product<DT, E4M3, LA, LB, EPI, TileMid>(p, s);
    return launch_product<DT, E4M3, LA, LB, EPI, TileSmall>(p, s);
}

}  // namespace
}  // namespace smc
