// Forward products of the linear and gated layers on 16-bit operands:
// x [m, k] rows along the contraction, W [k, n] across it.
#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {

hipError_t launch_store_16(const ProductArgs& p, int dt, hipStream_t s) {
    return dt == kF16 ? launch_tiled<kF16, false, kAlongK, kAcrossK, kEpiStore>(p, s)
                      : launch_tiled<kBF16, false, kAlongK, kAcrossK, kEpiStore>(p, s);
}

hipError_t launch_gated_16(const ProductArgs& p, int dt, hipStream_t s) {
    return dt == kF16 ? launch_tiled<kF16, false, kAlongK, kAcrossK, kEpiGated>(p, s)
                      : launch_tiled<kBF16, false, kAlongK, kAcrossK, kEpiGated>(p, s);
}

}  // namespace smc
