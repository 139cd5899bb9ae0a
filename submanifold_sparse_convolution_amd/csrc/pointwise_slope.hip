// The first kernel of the backward passes: the forward product again, its
// pre-activations turned into the gradient that reaches them.
#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {

hipError_t launch_slope_16(const ProductArgs& p, int dt, hipStream_t s) {
    return dt == kF16 ? launch_tiled<kF16, false, kAlongK, kAcrossK, kEpiSlope>(p, s)
                      : launch_tiled<kBF16, false, kAlongK, kAcrossK, kEpiSlope>(p, s);
}

hipError_t launch_gated_slope_16(const ProductArgs& p, int dt, hipStream_t s) {
    return dt == kF16 ? launch_tiled<kF16, false, kAlongK, kAcrossK, kEpiGatedSlope>(p, s)
                      : launch_tiled<kBF16, false, kAlongK, kAcrossK, kEpiGatedSlope>(p, s);
}

}  // namespace smc
