// Forward products of a few rows (up to 8) on 16-bit operands: the serving form
// of the linear and gated layers, bound by reading the weights once and by the
// launch.
//
// A block owns CB output columns (gated: of both halves) and the whole
// contraction: lane l reads 8 consecutive columns of weight row k as one 16-byte
// word (unaligned where the rows are), the block's 256 lanes cover CB columns
// of 2048 / CB weight rows at a time, and their partial sums are added across
// the lanes, then across the waves through LDS, in a fixed order. Few columns a
// block give many blocks, each with few loads in turn.
#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {
namespace {

constexpr int kFewThreads = 256;

template <int DT, int EPI, int R, int CB>
__global__ __launch_bounds__(kFewThreads) void k_few_rows(ProductArgs p) {
    constexpr bool kGated = EPI == kEpiGated;
    constexpr int kHalves = kGated ? 2 : 1;
    constexpr int kWide = CB / 8;                       // lanes side by side
    constexpr int kDeep = kFewThreads / kWide;          // weight rows at a time
    __shared__ float s_sum[4][R][kHalves][CB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int width = kGated ? p.half : p.n;
    const int c0 = blockIdx.x * CB, col = c0 + (tid % kWide) * 8;
    const uint16_t* x = static_cast<const uint16_t*>(p.a);
    const uint16_t* w = static_cast<const uint16_t*>(p.b);
    const int cols = width - col;                       // of this lane's 8 that exist (or more)

    float acc[R][kHalves][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[r][h][e] = 0.f;
    if (cols > 0) {
#pragma unroll 4
        for (int k = tid / kWide; k < p.k; k += kDeep) {
            float xv[R];
#pragma unroll
            for (int r = 0; r < R; ++r) xv[r] = to_f32<DT>(x[(int64_t)(r < p.m ? r : 0) * p.lda + k]);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const uint16_t* wr = w + (int64_t)k * p.ldb + col + (h ? p.half : 0);
                const u32x4 v = cols >= 8 ? load_unaligned(wr) : load_tail(wr, cols);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float wv = to_f32<DT>((v[e >> 1] >> ((e & 1) * 16)) & 0xffffu);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][h][e] = fmaf(xv[r], wv, acc[r][h][e]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = acc[r][h][e];
#pragma unroll
                for (int o = kWide; o < 64; o <<= 1) v += __shfl_xor(v, o);
                if (lane < kWide) s_sum[wave][r][h][lane * 8 + e] = v;
            }
    __syncthreads();
    for (int i = tid; i < R * CB; i += kFewThreads) {
        const int r = i / CB, c = i - r * CB;
        if (r >= p.m || c0 + c >= width) continue;
        float z[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            z[h] = s_sum[0][r][h][c] + s_sum[1][r][h][c] + s_sum[2][r][h][c] + s_sum[3][r][h][c];
            if (p.bias) z[h] += to_f32<DT>(static_cast<const uint16_t*>(p.bias)[c0 + c + (h ? p.half : 0)]);
        }
        float y = 0.f;
        with_act(p.act, [&](auto act_c) SMC_INLINE { y = act_value<decltype(act_c)::value>(z[0]); });
        if (kGated) y *= z[kHalves - 1];
        if (!kGated && p.extra)
            y += to_f32<DT>(static_cast<const uint16_t*>(p.extra)[(int64_t)r * p.ld_extra + c0 + c]);
        static_cast<uint16_t*>(p.out)[(int64_t)r * p.ldo + c0 + c] = (uint16_t)from_f32<DT>(y);
    }
}

template <int DT, int EPI, int R>
hipError_t few_t(const ProductArgs& p, hipStream_t s) {
    const int width = EPI == kEpiGated ? p.half : p.n;
    // the widest blocks (whole 128-byte lines of a weight row) that still give 128 of them
    if (width >= 128 * 64)
        launch(k_few_rows<DT, EPI, R, 64>, dim3((unsigned)((width + 63) / 64)), dim3(kFewThreads), 0, s, p);
    else if (width >= 128 * 32)
        launch(k_few_rows<DT, EPI, R, 32>, dim3((unsigned)((width + 31) / 32)), dim3(kFewThreads), 0, s, p);
    else
        launch(k_few_rows<DT, EPI, R, 16>, dim3((unsigned)((width + 15) / 16)), dim3(kFewThreads), 0, s, p);
    return hipGetLastError();
}

template <int DT, int EPI>
hipError_t few(const ProductArgs& p, hipStream_t s) {
    if (p.m <= 1) return few_t<DT, EPI, 1>(p, s);
    if (p.m <= 2) return few_t<DT, EPI, 2>(p, s);
    if (p.m <= 4) return few_t<DT, EPI, 4>(p, s);
    return few_t<DT, EPI, 8>(p, s);
}

}  // namespace

hipError_t launch_few_rows(const ProductArgs& p, Epilogue epi, int dt, hipStream_t s) {
    if (dt == kF16) return epi == kEpiGated ? few<kF16, kEpiGated>(p, s) : few<kF16, kEpiStore>(p, s);
    return epi == kEpiGated ? few<kBF16, kEpiGated>(p, s) : few<kBF16, kEpiStore>(p, s);
}

}  // namespace smc
