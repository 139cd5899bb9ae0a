// Words of 8 elements of 16-bit rows as float32, for the kernels that read and
// write rows through registers.
#pragma once

#include "pointwise_gemm.h"

namespace smc {
namespace {

constexpr int W = 8;        // elements of a word

// A word of a row: elements i .. i + 7, of which `left` exist (all of them where
// ALIGNED, which also means that the address is a multiple of 16).
template <bool ALIGNED>
__device__ __forceinline__ u32x4 load_word(const void* p, int64_t i, int left) {
    const uint16_t* e0 = static_cast<const uint16_t*>(p) + i;
    return ALIGNED ? *reinterpret_cast<const u32x4*>(e0) : left >= W ? load_unaligned(e0) : load_tail(e0, left);
}

template <int DT>
__device__ __forceinline__ void unpack(u32x4 u, float (&v)[W]) {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = to_f32<DT>((u[e >> 1] >> ((e & 1) * 16)) & 0xffffu);
}

template <int DT, bool ALIGNED>
__device__ __forceinline__ void load_f32(const void* p, int64_t i, int left, float (&v)[W]) {
    unpack<DT>(load_word<ALIGNED>(p, i, left), v);
}

template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_16(void* p, int64_t i, int left, const float (&v)[W]) {
    uint16_t* e0 = static_cast<uint16_t*>(p) + i;
    const u32x4 u = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    if (ALIGNED) {
        *reinterpret_cast<u32x4*>(e0) = u;
    } else if (left >= W) {
        __builtin_memcpy(e0, &u, 16);
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < left) e0[e] = (uint16_t)(u[e >> 1] >> ((e & 1) * 16));
    }
}

// 1 / sqrt(v); a row of zeros without an epsilon stays zeros.
__device__ __forceinline__ float inverse_root(float v) { return v == 0.f ? 0.f : 1.f / sqrtf(v); }

}  // namespace
}  // namespace smc
