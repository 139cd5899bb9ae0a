// RMS norm with the residual's addition, and its gradients; e4m3 weights.
//
//   s = x + r            (float32, rounded once into the new residual stream)
//   y = s rstd w,        rstd = 1 / sqrt(mean(s^2) + eps), from the float32 s
//   e4m3: y_scale = max(amax |y| / 448, 2^-126), q = e4m3(y / y_scale)
//
//   x_hat = s rstd, a = dy w
//   dx = rstd (a - x_hat mean(a x_hat)) + ds,   dw = sum over rows of dy x_hat
//
// Bound by memory: every row is read once and kept in registers between its
// sums and its outputs, by as many lanes as its 16-byte words (16 of them for 128
// channels, so a wave takes four rows and the sums stay inside it); rows too
// long for that are read again. With the residual, bf16: 91,000 x 128 15.5 us (93
// MB, 6.0 TB/s, part of it cached), e4m3 15,000 x 512 12.5 us (4.3 TB/s), backward
// 95,000 x 128 18.5 us (5.3 TB/s) and 4.0 us for the sums of dw.
#include <algorithm>

#include "pointwise_gemm.h"

namespace smc {
namespace {

constexpr int kNormThreads = 256;       // what grid_of counts on
constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;      // 2^-126

constexpr int W = 8;        // elements of a word

// A word of a row as float32: elements i .. i + 7, of which `left` exist (all of
// them where ALIGNED, which also means that the address is a multiple of 16).
template <int DT, bool ALIGNED>
__device__ __forceinline__ void load_f32(const void* p, int64_t i, int left, float (&v)[W]) {
    const uint16_t* e0 = static_cast<const uint16_t*>(p) + i;
    const u32x4 u = ALIGNED ? *reinterpret_cast<const u32x4*>(e0) : left >= W ? load_unaligned(e0) : load_tail(e0, left);
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = to_f32<DT>((u[e >> 1] >> ((e & 1) * 16)) & 0xffffu);
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

template <bool ALIGNED>
__device__ __forceinline__ void store_e4m3(void* p, int64_t i, int left, const float (&v)[W]) {
    uint8_t* e0 = static_cast<uint8_t*>(p) + i;
    u32x2 u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
        u[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true);
    }
    if (ALIGNED) {
        *reinterpret_cast<u32x2*>(e0) = u;
    } else if (left >= W) {
        __builtin_memcpy(e0, &u, 8);
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < left) e0[e] = (uint8_t)(u[e >> 2] >> ((e & 3) * 8));
    }
}

// From the row's largest magnitude by its bits, in which order NaN is above
// infinity: a NaN anywhere in the row makes the scale NaN.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) / kE4m3Max;
    return s < kTinyScale ? kTinyScale : s;        // NaN stays
}

// 1 / sqrt(v); a row of zeros without an epsilon stays zeros.
__device__ __forceinline__ float inverse_root(float v) { return v == 0.f ? 0.f : 1.f / sqrtf(v); }

// L lanes a row, NV words of W elements a lane, the row in registers.
template <int DT, bool A, int L, int NV>
__global__ __launch_bounds__(kNormThreads) void k_norm(NormArgs a) {
    const int lane = threadIdx.x % L;
    const int64_t row = block_number() * (kNormThreads / L) + threadIdx.x / L;
    const bool ok = row < a.n;
    float v[NV][W];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) v[j][e] = 0.f;
        if (ok && c < a.c) {
            load_f32<DT, A>(a.x, row * a.ldx + c, a.c - c, v[j]);
            if (a.residual) {
                float r[W];
                load_f32<DT, A>(a.residual, row * a.ldr + c, a.c - c, r);
#pragma unroll
                for (int e = 0; e < W; ++e) v[j][e] += r[e];
            }
        }
#pragma unroll
        for (int e = 0; e < W; ++e) ss += v[j][e] * v[j][e];
    }
    if (a.s) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * L + lane) * W;
            if (ok && c < a.c) store_16<DT, A>(a.s, row * a.lds + c, a.c - c, v[j]);
        }
    }
    const float rstd = inverse_root(lane_sum<L>(ss) / (float)a.c + a.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * W;
        if (c >= a.c) continue;
        float w[W];
        load_f32<DT, A>(a.weight, c, a.c - c, w);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            v[j][e] = v[j][e] * rstd * w[e];
            amax = max(amax, __float_as_uint(v[j][e]) & 0x7fffffffu);
        }
        if (!a.y_scale && ok) store_16<DT, A>(a.y, row * a.ldy + c, a.c - c, v[j]);
    }
    if (!a.y_scale) return;
    const float scale = row_scale(lane_max<L>(amax));
    if (ok && lane == 0) a.y_scale[row] = scale;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * W;
        if (!ok || c >= a.c) continue;
#pragma unroll
        for (int e = 0; e < W; ++e) v[j][e] = v[j][e] / scale;
        store_e4m3<A>(a.y, row * a.ldy + c, a.c - c, v[j]);
    }
}

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = lane_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return s[0] + s[1] + s[2] + s[3];
}

// Rows too wide for a wave's registers: a block a row, the row read again (from
// the caches) for each use.
template <int DT, bool A>
__global__ __launch_bounds__(kNormThreads) void k_norm_wide(NormArgs a) {
    __shared__ float s_sum[4];
    __shared__ uint32_t s_max[4];
    const int64_t row = block_number();
    if (row >= a.n) return;
    auto value = [&](int c, float (&v)[W]) {
        load_f32<DT, A>(a.x, row * a.ldx + c, a.c - c, v);
        if (a.residual) {
            float r[W];
            load_f32<DT, A>(a.residual, row * a.ldr + c, a.c - c, r);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] += r[e];
        }
    };
    float ss = 0.f;
    for (int c = threadIdx.x * W; c < a.c; c += kNormThreads * W) {
        float v[W];
        value(c, v);
#pragma unroll
        for (int e = 0; e < W; ++e) ss += v[e] * v[e];
    }
    const float rstd = inverse_root(block_sum(ss, s_sum) / (float)a.c + a.eps);
    uint32_t amax = 0;
    for (int pass = a.y_scale ? 0 : 1; pass < 2; ++pass) {
        float scale = 1.f;
        if (pass == 1 && a.y_scale) {
            amax = lane_max<64>(amax);
            if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = amax;
            __syncthreads();
            scale = row_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
            if (threadIdx.x == 0) a.y_scale[row] = scale;
        }
        for (int c = threadIdx.x * W; c < a.c; c += kNormThreads * W) {
            float v[W], w[W];
            value(c, v);
            load_f32<DT, A>(a.weight, c, a.c - c, w);
            if (pass == 1 && a.s) store_16<DT, A>(a.s, row * a.lds + c, a.c - c, v);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                v[e] = v[e] * rstd * w[e];
                amax = max(amax, __float_as_uint(v[e]) & 0x7fffffffu);
                if (a.y_scale) v[e] = v[e] / scale;
            }
            if (pass == 0) continue;
            if (a.y_scale)
                store_e4m3<A>(a.y, row * a.ldy + c, a.c - c, v);
            else
                store_16<DT, A>(a.y, row * a.ldy + c, a.c - c, v);
        }
    }
}

// dx of the rows blockIdx, + gridDim, ... and this block's sums of dy x_hat.
template <int DT, bool A, int L, int NV>
__global__ __launch_bounds__(kNormThreads) void k_norm_backward(NormArgs a) {
    constexpr int kRows = kNormThreads / L;
    __shared__ float s_dw[L * NV * W];
    const int lane = threadIdx.x % L;
    float w[NV][W], dw[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * L + lane) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) w[j][e] = dw[j][e] = 0.f;
        if (c < a.c) load_f32<DT, A>(a.weight, c, a.c - c, w[j]);
    }
    const int64_t first = (int64_t)blockIdx.x * kRows + threadIdx.x / L;
    // every lane of a wave walks the same number of rows: the sums below are
    // exchanged across its lanes
    const int64_t rounds = (a.n - (int64_t)blockIdx.x * kRows + (int64_t)gridDim.x * kRows - 1) /
                           ((int64_t)gridDim.x * kRows);
    for (int64_t it = 0; it < rounds; ++it) {
        const int64_t row = first + it * gridDim.x * kRows;
        const bool ok = row < a.n;
        float x[NV][W], dy[NV][W];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * L + lane) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) x[j][e] = dy[j][e] = 0.f;
            if (ok && c < a.c) {
                load_f32<DT, A>(a.x, row * a.ldx + c, a.c - c, x[j]);
                load_f32<DT, A>(a.dy, row * a.lddy + c, a.c - c, dy[j]);
            }
        }
        float ds[NV][W];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * L + lane) * W;
#pragma unroll
            for (int e = 0; e < W; ++e) ds[j][e] = 0.f;
            if (a.residual && ok && c < a.c) load_f32<DT, A>(a.residual, row * a.ldr + c, a.c - c, ds[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                ss += x[j][e] * x[j][e];
                dot += dy[j][e] * w[j][e] * x[j][e];
            }
        ss = lane_sum<L>(ss);
        dot = lane_sum<L>(dot);
        const float rstd = inverse_root(ss / (float)a.c + a.eps);
        const float mean = dot * rstd / (float)a.c;        // mean(a x_hat)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * L + lane) * W;
            float o[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float xh = x[j][e] * rstd;
                o[e] = rstd * (dy[j][e] * w[j][e] - xh * mean) + ds[j][e];
                if (ok) dw[j][e] += dy[j][e] * xh;
            }
            if (ok && c < a.c) store_16<DT, A>(a.y, row * a.ldy + c, a.c - c, o);
        }
    }
    // the lane groups of a wave, then the waves in turn
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < W; ++e)
#pragma unroll
            for (int o = L; o < 64; o <<= 1) dw[j][e] += __shfl_xor(dw[j][e], o);
    for (int wv = 0; wv < kNormThreads / 64; ++wv) {
        if ((int)(threadIdx.x >> 6) == wv && (threadIdx.x & 63) < L) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    float* d = s_dw + (j * L + lane) * W + e;
                    *d = wv == 0 ? dw[j][e] : *d + dw[j][e];
                }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.c; c += kNormThreads) a.part[(int64_t)blockIdx.x * a.c + c] = s_dw[c];
}

template <int DT, bool A>
__global__ __launch_bounds__(kNormThreads) void k_norm_backward_wide(NormArgs a) {
    __shared__ float s_sum[4];
    float* part = a.part + (int64_t)blockIdx.x * a.c;      // each thread its own columns
    for (int c = threadIdx.x; c < a.c; c += kNormThreads) part[c] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        float ss = 0.f, dot = 0.f;
        for (int c = threadIdx.x * W; c < a.c; c += kNormThreads * W) {
            float x[W], dy[W], w[W];
            load_f32<DT, A>(a.x, row * a.ldx + c, a.c - c, x);
            load_f32<DT, A>(a.dy, row * a.lddy + c, a.c - c, dy);
            load_f32<DT, A>(a.weight, c, a.c - c, w);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                ss += x[e] * x[e];
                dot += dy[e] * w[e] * x[e];
            }
        }
        const float rstd = inverse_root(block_sum(ss, s_sum) / (float)a.c + a.eps);
        const float mean = block_sum(dot, s_sum) * rstd / (float)a.c;
        for (int c = threadIdx.x * W; c < a.c; c += kNormThreads * W) {
            float x[W], dy[W], w[W], o[W], ds[W];
            load_f32<DT, A>(a.x, row * a.ldx + c, a.c - c, x);
            load_f32<DT, A>(a.dy, row * a.lddy + c, a.c - c, dy);
            load_f32<DT, A>(a.weight, c, a.c - c, w);
#pragma unroll
            for (int e = 0; e < W; ++e) ds[e] = 0.f;
            if (a.residual) load_f32<DT, A>(a.residual, row * a.ldr + c, a.c - c, ds);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float xh = x[e] * rstd;
                o[e] = rstd * (dy[e] * w[e] - xh * mean) + ds[e];
                if (c + e < a.c) part[c + e] += dy[e] * xh;
            }
            store_16<DT, A>(a.y, row * a.ldy + c, a.c - c, o);
        }
    }
}

// dw[c] = the blocks' sums: 8 columns a block, 128 runs of blocks (each a
// strided sum, its loads independent), the runs added by a tree.
template <int DT>
__global__ __launch_bounds__(1024) void k_norm_weight_sum(const float* __restrict__ part, int blocks,
                                                          int c, uint16_t* dw) {
    __shared__ float s[128][9];
    const int x = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int col = blockIdx.x * 8 + x;
    float v = 0.f;
    if (col < c) {
#pragma unroll 8
        for (int b = g; b < blocks; b += 128) v += part[(int64_t)b * c + col];
    }
    s[g][x] = v;
    __syncthreads();
    for (int o = 64; o > 0; o >>= 1) {
        if (g < o) s[g][x] += s[g + o][x];
        __syncthreads();
    }
    if (g == 0 && col < c) dw[col] = (uint16_t)from_f32<DT>(s[0][x]);
}

// W [c_in, c_out] -> q [c_out, c_in] e4m3, one scale a column of W. 32 columns
// a block; W is read twice. Made for a call a weight and program, not for the path
// of a step: bound by the latency of a block's chain of loads over c_in (512 x 4096 29
// us, 2048 x 512 109 us).
template <int DT>
__global__ __launch_bounds__(256) void k_quantize_weight(const uint16_t* __restrict__ w, int64_t ldw,
                                                         int c_in, int c_out, uint8_t* q,
                                                         int64_t ldq, float* scale) {
    __shared__ uint32_t s_max[8][32];
    __shared__ float s_scale[32];
    __shared__ float s_t[32][33];
    const int x = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + x;
    uint32_t amax = 0;
    if (col < c_out)
        for (int k = g; k < c_in; k += 8)
            amax = max(amax, __float_as_uint(to_f32<DT>(w[k * ldw + col])) & 0x7fffffffu);
    s_max[g][x] = amax;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < 8; ++i) amax = max(amax, s_max[i][x]);
        s_scale[x] = row_scale(amax);
        if (col < c_out) scale[col] = s_scale[x];
    }
    __syncthreads();
    for (int k0 = 0; k0 < c_in; k0 += 32) {
        for (int i = g; i < 32; i += 8)
            s_t[i][x] = col < c_out && k0 + i < c_in ? to_f32<DT>(w[(k0 + i) * ldw + col]) / s_scale[x] : 0.f;
        __syncthreads();
        for (int i = g; i < 32; i += 8) {
            const int oc = blockIdx.x * 32 + i;
            if (oc < c_out && k0 + x < c_in)
                q[oc * ldq + k0 + x] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(s_t[x][i], 0.f, 0, false);
        }
        __syncthreads();
    }
}

// Lanes and words a row for c channels: the fewest lanes that hold the row in
// one word each, up to a wave; wider rows take up to 8 words a lane (4096
// channels).
template <template <int, bool, int, int> class K, int DT, bool A>
bool by_shape(const NormArgs& a, hipStream_t s) {
    const int words = (a.c + W - 1) / W;
    if (words <= 1) K<DT, A, 1, 1>::go(a, s);
    else if (words <= 2) K<DT, A, 2, 1>::go(a, s);
    else if (words <= 4) K<DT, A, 4, 1>::go(a, s);
    else if (words <= 8) K<DT, A, 8, 1>::go(a, s);
    else if (words <= 16) K<DT, A, 16, 1>::go(a, s);
    else if (words <= 32) K<DT, A, 32, 1>::go(a, s);
    else if (words <= 64) K<DT, A, 64, 1>::go(a, s);
    else if (words <= 128) K<DT, A, 64, 2>::go(a, s);
    else if (words <= 256) K<DT, A, 64, 4>::go(a, s);
    else if (words <= 512) K<DT, A, 64, 8>::go(a, s);
    else return false;
    return true;
}

template <template <int, bool, int, int> class K, int DT>
bool by_shape(const NormArgs& a, hipStream_t s) {
    return a.vec ? by_shape<K, DT, true>(a, s) : by_shape<K, DT, false>(a, s);
}

template <int DT, bool A, int L, int NV>
struct Forward {
    static void go(const NormArgs& a, hipStream_t s) {
        constexpr int kRows = kNormThreads / L;
        launch(k_norm<DT, A, L, NV>, grid_of((a.n + kRows - 1) / kRows), dim3(kNormThreads), 0, s, a);
    }
};

template <int DT, bool A, int L, int NV>
struct Backward {
    static void go(const NormArgs& a, hipStream_t s) {
        launch(k_norm_backward<DT, A, L, NV>, dim3((unsigned)norm_backward_blocks(a.n, a.c)),
               dim3(kNormThreads), 0, s, a);
    }
};

template <int DT>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
    if (!by_shape<Forward, DT>(a, s)) {
        if (a.vec)
            launch(k_norm_wide<DT, true>, grid_of(a.n), dim3(kNormThreads), 0, s, a);
        else
            launch(k_norm_wide<DT, false>, grid_of(a.n), dim3(kNormThreads), 0, s, a);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t norm_backward_t(const NormArgs& a, hipStream_t s) {
    const int blocks = norm_backward_blocks(a.n, a.c);
    if (blocks > 0 && !by_shape<Backward, DT>(a, s)) {
        if (a.vec)
            launch(k_norm_backward_wide<DT, true>, dim3((unsigned)blocks), dim3(kNormThreads), 0, s, a);
        else
            launch(k_norm_backward_wide<DT, false>, dim3((unsigned)blocks), dim3(kNormThreads), 0, s, a);
    }
    launch(k_norm_weight_sum<DT>, dim3((unsigned)((a.c + 7) / 8)), dim3(1024), 0, s, a.part, blocks,
           a.c, static_cast<uint16_t*>(a.dweight));
    return hipGetLastError();
}

}  // namespace

// Blocks of the backward pass: each writes c sums, so no more than fill the
// device, and no more than there are rows (as many a block as its 256 threads hold
// by by_shape; one where they are too wide for that). 95,000 x 128 with 2, 3, 4, 6 and 8
// blocks a CU: rows and sums 24.3, 22.8, 22.5, 23.5 and 24.4 us.
int norm_backward_blocks(int64_t n, int c) {
    const int words = (c + W - 1) / W;
    int lanes = 1;
    while (lanes < words && lanes < 64) lanes *= 2;
    const int64_t rows = words > 64 * 8 ? 1 : kNormThreads / lanes;
    return (int)std::min<int64_t>((n + rows - 1) / rows, (int64_t)4 * device_cus());
}

hipError_t launch_norm(const NormArgs& a, int dt, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    return dt == kF16 ? norm_t<kF16>(a, s) : norm_t<kBF16>(a, s);
}

hipError_t launch_norm_backward(const NormArgs& a, int dt, hipStream_t s) {
    return dt == kF16 ? norm_backward_t<kF16>(a, s) : norm_backward_t<kBF16>(a, s);
}

hipError_t launch_quantize_weight(const void* w, int64_t ldw, int c_in, int c_out, void* q,
                                  int64_t ldq, float* scale, int dt, hipStream_t s) {
    const dim3 grid((unsigned)((c_out + 31) / 32));
    if (dt == kF16)
        launch(k_quantize_weight<kF16>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(w), ldw,
               c_in, c_out, static_cast<uint8_t*>(q), ldq, scale);
    else
        launch(k_quantize_weight<kBF16>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(w), ldw,
               c_in, c_out, static_cast<uint8_t*>(q), ldq, scale);
    return hipGetLastError();
}

}  // namespace smc
