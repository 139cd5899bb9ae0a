// Gradients of the linear and gated layers: dx = dz W^T, dW = x^T dz and
// db = column sums of dz.
#include <algorithm>
#include <mutex>

#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {

int device_cus() {
    static std::mutex mu;
    static int known[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        int v = 0;
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) v = 256;
        known[dev] = v;
    }
    return known[dev];
}

hipError_t launch_forward(ProductArgs p, Epilogue epi, int dt, bool e4m3, bool w_along, hipStream_t s) {
    p.k_split = p.k;
    p.splits = 1;
    if (e4m3)
        return epi == kEpiGated ? launch_gated_e4m3(p, dt, w_along, s) : launch_store_e4m3(p, dt, w_along, s);
    // (unaligned rows of which no copies were made cost the product kernel far more)
    if ((epi == kEpiStore || epi == kEpiGated) &&
        (p.vec_a && p.vec_b ? few_rows_pay(p, epi) : p.m <= kFewRows))
        return launch_few_rows(p, epi, dt, s);
    switch (epi) {
        case kEpiGated: return launch_gated_16(p, dt, s);
        case kEpiSlope: return launch_slope_16(p, dt, s);
        case kEpiGatedSlope: return launch_gated_slope_16(p, dt, s);
        default: return launch_store_16(p, dt, s);
    }
}

hipError_t launch_input_gradient(ProductArgs p, int dt, hipStream_t s) {
    p.k_split = p.k;
    p.splits = 1;
    return dt == kF16 ? launch_tiled<kF16, false, kAlongK, kAlongK, kEpiStore>(p, s)
                      : launch_tiled<kBF16, false, kAlongK, kAlongK, kEpiStore>(p, s);
}

// Ranges of the rows: as many as give every CU at most two 128 x 128 tiles, what
// is resident at once (rounded up, a few blocks took a second tile: dW of 84,276 x
// 144 -> 832 61.7 us, 40.5 so; 5,172 x 336 -> 1824 20.7, 16.7), none shorter than 256
// rows (4 steps), so that a tile's sums (64 KiB to memory and back) stay small
// beside the rows it reads.
// A range is whole steps (64 rows), and every range has rows: rounding their length
// up may take fewer of them.
int weight_gradient_range(int64_t rows, int c_in, int n) {
    const int64_t tiles = (int64_t)((c_in + 127) / 128) * ((n + 127) / 128);
    const int64_t want = 2 * device_cus() / tiles;
    const int64_t ranges = std::max<int64_t>(1, std::min<int64_t>(want, (rows + 255) / 256));
    return (int)(((rows + ranges - 1) / ranges + 63) / 64 * 64);
}

hipError_t launch_weight_gradient(ProductArgs p, int dt, hipStream_t s) {
    return dt == kF16 ? launch_product<kF16, false, kAcrossK, kAcrossK, kEpiPartial, TileMid>(p, s)
                      : launch_product<kBF16, false, kAcrossK, kAcrossK, kEpiPartial, TileMid>(p, s);
}

namespace {

// dw (and db, the row after) = the splits' float32 sums, added in a fixed order
// and rounded once; kSumWord consecutive elements a thread (halves start at
// multiples of 8 columns). G threads share an element's splits (each a strided
// sum) where there are many of them and few elements. Bound by reading the sums:
// 8 splits of 2048 x 512, 16.8 MB, 7.0 us.
constexpr int kSumWord = 4;

template <int DT, int G>
__global__ __launch_bounds__(256) void k_sum_parts(SumArgs a) {
    constexpr int W = kSumWord;
    constexpr int kPer = 256 / G;                   // words a block
    __shared__ float s_v[G > 1 ? G : 1][kPer * W + 1];
    const int64_t total = (a.m + (a.db ? 1 : 0)) * a.n;
    const int x = threadIdx.x % kPer, g = threadIdx.x / kPer;
    const int64_t i = ((int64_t)blockIdx.x * kPer + x) * W;
    float v[W] = {};
    if (i < total) {
#pragma unroll 4
        for (int sp = g; sp < a.splits; sp += G) {
            const float* src = a.part + (int64_t)sp * total + i;
            const f32x4 u = *reinterpret_cast<const f32x4*>(src);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] += u[e];
        }
    }
    if constexpr (G > 1) {
#pragma unroll
        for (int e = 0; e < W; ++e) s_v[g][x * W + e] = v[e];
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int o = 1; o < G; ++o)
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] += s_v[o][x * W + e];
    }
    if (i >= total) return;
    const float by = a.unscale ? *a.unscale : 1.f;
    const int64_t row = i / a.n;
    const int col = (int)(i - row * a.n), h = col / a.half_p, c = col - h * a.half_p;   // (a word lies in one half)
    uint16_t* o = row < a.m ? static_cast<uint16_t*>(a.dw) + row * a.ldw : static_cast<uint16_t*>(a.db);
    o += h * a.c_out + c;
#pragma unroll
    for (int e = 0; e < W; ++e)
        if (c + e < a.c_out) o[e] = (uint16_t)from_f32<DT>(v[e] * by);
}

template <int DT>
void sum_parts(const SumArgs& a, hipStream_t s) {
    const int64_t words = ((a.m + (a.db ? 1 : 0)) * a.n + kSumWord - 1) / kSumWord;
    if (a.splits >= 32)             // 247 splits of 129 x 16 sums: 25 us by one thread an element
        launch(k_sum_parts<DT, 16>, dim3((unsigned)((words + 15) / 16)), dim3(256), 0, s, a);
    else
        launch(k_sum_parts<DT, 1>, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, a);
}

// 16 bytes of dst a thread. Bound by memory. (Divided in 32 bits where they do.)
template <typename E>
__global__ __launch_bounds__(256) void k_pad_rows(const E* __restrict__ src, int64_t lds, int64_t rows, int halves,
                                                  int c, E* __restrict__ dst, int64_t ldd, int64_t rows_p, int half_p) {
    constexpr int kPer = 16 / sizeof(E);
    const int words = (int)(ldd / kPer);
    const int64_t i = block_number() * 256 + threadIdx.x;
    const int64_t row = rows_p * words < ((int64_t)1 << 31) ? (int64_t)((uint32_t)i / (uint32_t)words) : i / words;
    if (row >= rows_p) return;
    const int col = (int)(i - row * words) * kPer, h = col / half_p, k = col - h * half_p;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (row < rows && h < halves) {
        const E* e0 = src + row * lds + (int64_t)h * c + k;
        if (k + kPer <= c) {
            v = load_unaligned(e0);
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (k + e < c) v[e * (int)sizeof(E) / 4] |= (uint32_t)e0[e] << (e * (int)sizeof(E) % 4 * 8);
        }
    }
    *reinterpret_cast<u32x4*>(dst + row * ldd + col) = v;
}

}  // namespace

hipError_t launch_sum_parts(const SumArgs& a, int dt, hipStream_t s) {
    (dt == kF16 ? sum_parts<kF16> : sum_parts<kBF16>)(a, s);
    return hipGetLastError();
}

hipError_t launch_pad_rows(int esize, const void* src, int64_t lds, int64_t rows, int halves, int c, void* dst,
                           int64_t ldd, int64_t rows_p, int half_p, hipStream_t s) {
    const dim3 grid = grid_of((rows_p * (ldd * esize / 16) + 255) / 256);
    if (esize == 1)
        launch(k_pad_rows<uint8_t>, grid, dim3(256), 0, s, static_cast<const uint8_t*>(src), lds, rows, halves, c,
               static_cast<uint8_t*>(dst), ldd, rows_p, half_p);
    else
        launch(k_pad_rows<uint16_t>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(src), lds, rows, halves, c,
               static_cast<uint16_t*>(dst), ldd, rows_p, half_p);
    return hipGetLastError();
}

}  // namespace smc
