// Forward products of a few rows (up to 16) on 16-bit operands: the serving form
// of the linear and gated layers, bound by reading the weights once and by the
// launch.
//
// A block owns CB output columns (gated: of both halves) and the whole
// contraction: a lane reads 8 consecutive columns of weight row k as one 16-byte
// word (unaligned where the rows are), the block's 1024 lanes cover CB columns
// of 8192 / CB weight rows at a time, up to four such rounds in flight, and their
// partial sums are added across the lanes, then across the waves through LDS,
// in a fixed order. Few columns a block give many blocks, and 1024 lanes a
// short chain of loads in each.
// More rows than a block takes (8, gated 4: registers) are a second dimension of
// blocks, which read the weights from the cache again. Against 32 x 64 tiles of
// the product kernel (whose time does not depend on the rows), us on the GPU:
//                 2 rows  4 rows  16 rows  tiles
//     64 ->   64     -      4.3     6.4     3.8
//    512 ->  512    3.5     4.7     6.9     6.3
//    768 ->  512    3.8     5.0     7.6     7.5
//   1024 ->  512    4.1     5.2     7.8     8.6
//   2048 -> 2048    6.8     8.0    11.0    13.2
//   gated:
//     64 ->  176    4.3     6.3     6.4     3.6
//    512 -> 1368    4.8     7.0    12.8     6.2
//   1024 -> 1024    6.0     8.6     9.5     8.5
//   2048 ->  512    7.7    10.4    10.8    13.1
// so up to 4 rows come here and up to 16 of contractions above 768; gated, 2 and 4 of
// contractions above 1024.
// Unaligned rows, against copies and the product kernel: 1500 -> 512 with 16 rows 8.4,
// 15.5; 2048 -> 2001 14.1, 19.9; 130 -> 1100 7.6, 9.2; gated 512 -> 1365 with 8 rows 8.8,
// 10.0, but with 12 or 16, whose 258 and more blocks have to take turns, 14.2;
// 700 -> 2001 with 8, 12 and 16 rows 11.8, 18.4, 21.3, 14.5: up to 16 rows while there are no
// more blocks than CUs.
#include "pointwise_gemm.h"
#include "pointwise_launch.h"

namespace smc {
namespace {

constexpr int kFewThreads = 1024;
constexpr int kFewWaves = kFewThreads / 64;

template <int DT, int EPI, int R, int CB>
__global__ __launch_bounds__(kFewThreads) void k_few_rows(ProductArgs p) {
    constexpr bool kGated = EPI == kEpiGated;
    constexpr int kHalves = kGated ? 2 : 1;
    constexpr int kWide = CB / 8;                       // words side by side
    constexpr int kLanes = 64 / kWide;                  // lanes of a wave on one word's column
    constexpr int kDeep = kFewThreads / kWide;          // weight rows at a time
    constexpr int kFewRounds = R <= 2 ? 4 / R : 1;      // (registers)
    __shared__ float s_sum[kFewWaves][R][kHalves][CB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int width = kGated ? p.half : p.n;
    const int c0 = blockIdx.x * CB, col = c0 + lane / kLanes * 8;
    const int r0 = blockIdx.y * R, rows = p.m - r0;     // this block's rows (R of them at most)
    const uint16_t* x = static_cast<const uint16_t*>(p.a) + (int64_t)r0 * p.lda;
    const uint16_t* w = static_cast<const uint16_t*>(p.b);
    const int cols = width - col;                       // of this lane's 8 that exist (or more)

    float acc[R][kHalves][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[r][h][e] = 0.f;
    // `word` reads 8 columns of a weight row; past the last row it is read again
    // and counted as zeros, so that a round's loads need no branches
    auto walk = [&](auto word, auto rounds_c) SMC_INLINE {
        constexpr int kRounds = decltype(rounds_c)::value;
        for (int k0 = wave * kLanes + lane % kLanes; k0 < p.k; k0 += kRounds * kDeep) {
            u32x4 v[kRounds][kHalves];
            float xv[kRounds][R];
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int k = k0 + i * kDeep, kc = k < p.k ? k : p.k - 1;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) v[i][h] = word(w + (int64_t)kc * p.ldb + col + (h ? p.half : 0));
#pragma unroll
                for (int r = 0; r < R; ++r) xv[i][r] = to_f32<DT>(x[(int64_t)(r < rows ? r : 0) * p.lda + kc]);
            }
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                if (k0 + i * kDeep >= p.k) continue;
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float wv = to_f32<DT>((v[i][h][e >> 1] >> ((e & 1) * 16)) & 0xffffu);
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[r][h][e] = fmaf(xv[i][r], wv, acc[r][h][e]);
                    }
            }
        }
    };
    auto words = [](const uint16_t* wr) SMC_INLINE { return load_unaligned(wr); };
    if (cols >= 8 && p.k <= kDeep)
        walk(words, std::integral_constant<int, 1>());
    else if (cols >= 8)
        walk(words, std::integral_constant<int, kFewRounds>());
    else if (cols > 0)
        walk([cols](const uint16_t* wr) SMC_INLINE { return load_tail(wr, cols); }, std::integral_constant<int, 1>());
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = lane_sum<kLanes>(acc[r][h][e]);
                if (lane % kLanes == 0) s_sum[wave][r][h][lane / kLanes * 8 + e] = v;
            }
    __syncthreads();
    static_assert(R * CB <= kFewThreads, "a thread an output");
    {
        const int r = tid / CB, c = tid - r * CB;
        if (r >= rows || r >= R || c0 + c >= width) return;
        float z[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            z[h] = 0.f;
#pragma unroll
            for (int wv = 0; wv < kFewWaves; ++wv) z[h] += s_sum[wv][r][h][c];
            if (p.bias) z[h] += to_f32<DT>(static_cast<const uint16_t*>(p.bias)[c0 + c + (h ? p.half : 0)]);
        }
        float y = 0.f;
        with_act(p.act, [&](auto act_c) SMC_INLINE { y = act_value<decltype(act_c)::value>(z[0]); });
        if (kGated) y *= z[kHalves - 1];
        if (!kGated && p.extra)
            y += to_f32<DT>(static_cast<const uint16_t*>(p.extra)[(int64_t)(r0 + r) * p.ld_extra + c0 + c]);
        static_cast<uint16_t*>(p.out)[(int64_t)(r0 + r) * p.ldo + c0 + c] = (uint16_t)from_f32<DT>(y);
    }
}

// The widest blocks (whole 128-byte lines of a weight row) that still give 128 of
// them, else 16 columns. One row, 2048 -> 512 and gated 512 -> 1365: 8.4 and 7.3 us
// with 8 columns a block, 5.0 and 7.6 with 16, 7.1 and 10.3 with 32, 10.7 and 11.7
// with 64.
int block_columns(int width) { return width >= 128 * 64 ? 64 : width >= 128 * 32 ? 32 : 16; }
int block_rows(int m, bool gated) { return m <= 2 ? m : m <= 4 || gated ? 4 : 8; }

template <int DT, int EPI, int R>
hipError_t few_t(const ProductArgs& p, hipStream_t s) {
    const int width = EPI == kEpiGated ? p.half : p.n;
    const unsigned groups = (unsigned)((p.m + R - 1) / R);
    const int cb = block_columns(width);
    const dim3 grid((unsigned)((width + cb - 1) / cb), groups);
    switch (cb) {
        case 64: launch(k_few_rows<DT, EPI, R, 64>, grid, dim3(kFewThreads), 0, s, p); break;
        case 32: launch(k_few_rows<DT, EPI, R, 32>, grid, dim3(kFewThreads), 0, s, p); break;
        default: launch(k_few_rows<DT, EPI, R, 16>, grid, dim3(kFewThreads), 0, s, p);
    }
    return hipGetLastError();
}

template <int DT, int EPI>
hipError_t few(const ProductArgs& p, hipStream_t s) {
    switch (block_rows(p.m, EPI == kEpiGated)) {
        case 1: return few_t<DT, EPI, 1>(p, s);
        case 2: return few_t<DT, EPI, 2>(p, s);
        case 4: return few_t<DT, EPI, 4>(p, s);
        default:
            if constexpr (EPI == kEpiStore) return few_t<DT, EPI, 8>(p, s);
            else return hipErrorInvalidValue;       // (block_rows has no more for gated layers)
    }
}

}  // namespace

bool few_rows_pay(const ProductArgs& p, Epilogue epi) {
    const bool gated = epi == kEpiGated;
    if (p.m > kFewRows) return false;
    if (p.vec_a && p.vec_b && p.m > (gated ? (p.k > 1024 ? 4 : 2) : p.k > 768 ? kFewRows : 4)) return false;
    const int width = gated ? p.half : p.n, cb = block_columns(width), r = block_rows(p.m, gated);
    return p.m <= r || (int64_t)((width + cb - 1) / cb) * ((p.m + r - 1) / r) <= device_cus();
}

hipError_t launch_few_rows(const ProductArgs& p, Epilogue epi, int dt, hipStream_t s) {
    if (dt == kF16) return epi == kEpiGated ? few<kF16, kEpiGated>(p, s) : few<kF16, kEpiStore>(p, s);
    return epi == kEpiGated ? few<kBF16, kEpiGated>(p, s) : few<kBF16, kEpiStore>(p, s);
}

}  // namespace smc
