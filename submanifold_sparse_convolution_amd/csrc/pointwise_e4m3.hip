// Forward products on e4m3 operands with float32 scales: x along the
// contraction, the weights either way.
#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {
namespace {

template <int DT, int EPI>
hipError_t launch_e4m3(const ProductArgs& p, bool along, hipStream_t s) {
    return along ? launch_tiled<DT, true, kAlongK, kAlongK, EPI>(p, s)
                 : launch_tiled<DT, true, kAlongK, kAcrossK, EPI>(p, s);
}

}  // namespace

hipError_t launch_store_e4m3(const ProductArgs& p, int dt, bool along, hipStream_t s) {
    return dt == kF16 ? launch_e4m3<kF16, kEpiStore>(p, along, s) : launch_e4m3<kBF16, kEpiStore>(p, along, s);
}

hipError_t launch_gated_e4m3(const ProductArgs& p, int dt, bool along, hipStream_t s) {
    return dt == kF16 ? launch_e4m3<kF16, kEpiGated>(p, along, s) : launch_e4m3<kBF16, kEpiGated>(p, along, s);
}

}  // namespace smc
