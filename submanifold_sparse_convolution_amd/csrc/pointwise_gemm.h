// The product kernel of the linear and gated layers: out = epilogue(A B^T)
// with A's rows the output's rows and B's rows the output's columns, float32
// accumulation in MFMA registers. One template serves the forward products,
// their recomputation in the backward pass, dz W^T and x^T dz; what differs
// is how each operand lies in memory (Layout) and the epilogue.
//
// Tiles. A block owns BM x BN outputs and walks the contraction in steps of
// 128 bytes (64 16-bit or 128 e4m3 elements). Both operands' steps go from
// memory straight to LDS (buffer loads of 16 bytes a lane that write LDS), the
// next step's loads in flight while the waves multiply the current one. A
// wave owns 16 MT rows x 64 columns as 16 x 16 MFMA tiles, B's rows as the
// MFMA's row operand, so a lane ends up with 4 consecutive output columns
// of one row, and after a swap between neighbouring 16-lane rows with 8 of
// them: one 16-byte store.
//
// LDS images. kAlongK: 128 bytes a row, its eight 16-byte words permuted by
// word ^= row & 7, so that the 16 rows a fragment load reads lie in different
// banks. kAcrossK: the memory rows [k][columns] as they are; a transposing LDS
// read hands each lane 4 consecutive k of its column. A read takes 32-byte
// pieces of 16 k rows, so pieces are permuted by the k row's bits 0, 1 and 3.
// Loads that write LDS place lane l at 16 l, so the permutation is applied to
// the address a lane loads from.
//
// What bounds it. A step of a 128 x 128 tile is 32 KiB to LDS and 128 MFMAs of 16 x 16
// x 32, 16 clocks each: 512 clocks of the CU's four matrix units, 64 bytes a clock at
// their full rate. Measured: dz W^T of 15,000 x 4096 -> 512 and x^T dz of the same keep
// them 45 and 49 % busy at 28 and 31 bytes a clock and CU (14 TB/s to LDS in all):
// no unit is at its end, a step's arrival, fragment reads and products do not
// overlap fully in two blocks a CU. With few steps a tile, or activations after them,
// the tile's start and epilogue stand beside too few products: 24 to 30 % busy at 15
// to 19 bytes in the linear backward's products, the slopes and the e4m3 layer.
// Larger tiles need fewer bytes, but their accumulators leave one block a CU and
// nothing to overlap the epilogue, and were not faster.
// bf16, GPU times: dz W^T of 15,000 x 4096 -> 512 70 us (0.90 PFLOP/s), x^T dz of the
// same 67 us (0.93), the slopes of the gated 512 -> 2048 107 us (0.59, with 184 MB in
// the epilogue), 91,000 x 128 -> 128 with a residual 15.6 us (4.5 TB/s), gated
// 128 -> 344 38.0 us (2.3 TB/s); e4m3 gated 15,000 x 512 -> 2048 51.2 us (1.23 PFLOP/s).
//
// Edges. The buffer descriptors end at the operand's last valid element, and a
// lane whose word is past the end of a row gets an offset outside: such loads
// write zeros to LDS, so every edge multiplies by exact zeros on both sides.
#pragma once

#include <type_traits>

#include "pointwise.h"

namespace smc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define SMC_LDS __attribute__((address_space(3)))
// for lambdas over register arrays: a call that is not inlined puts them in memory
#define SMC_INLINE __attribute__((always_inline))

constexpr uint32_t kOutside = 0x80000000u;      // beyond every buffer's end

// ---- element types ------------------------------------------------------------

template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
    if (DT == kF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
    return __uint_as_float(bits16 << 16);
}

// Round to nearest, ties to even; NaN stays NaN.
template <int DT>
__device__ __forceinline__ uint32_t from_f32(float f) {
    if (DT == kF16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    if (DT == kF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if (DT == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 128 e4m3 products; block scales of 1 (exponent byte 127). The instruction adds
// each group of 8 consecutive products aligned to the group's largest with 13
// bits below its leading bit (measured), the groups and the accumulator in
// float32. That is up to 2^-10 of sum |terms|, beside the 2^-4 by which each
// e4m3 operand was rounded and the 2^-8 of a bf16 output; converting the
// operands to bf16 first would keep full float32 sums at half the MFMA rate.
__device__ __forceinline__ f32x4 mfma_e4m3(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c) {
    const i32x8 a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const i32x8 b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}

// ---- activations, float32 -----------------------------------------------------

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and exp(-z^2 / 2). erf by formula 7.1.26 of
// Abramowitz and Stegun (error below 1.5e-7, what float32 leaves of 1 + erf
// anyway), whose exponential is the Gaussian that the slope needs too.
__device__ __forceinline__ float normal_cdf(float z, float& gauss) {
    gauss = __expf(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3275911f * 0.70710678f, 1.f));
    const float tail = 0.5f * gauss * t *
                       fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f),
                                    -0.284496736f), 0.254829592f);
    return z < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == kActRelu) return z < 0.f ? 0.f : z;
    if (ACT == kActSilu) return z * sigmoid(z);
    if (ACT == kActGelu) {
        float g;
        return z * normal_cdf(z, g);
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == kActRelu) return z > 0.f ? 1.f : 0.f;
    if (ACT == kActSilu) {
        const float g = sigmoid(z);
        return g * (1.f + z * (1.f - g));
    }
    if (ACT == kActGelu) {
        float g;
        const float c = normal_cdf(z, g);
        return c + z * 0.39894228040143268f * g;
    }
    return 1.f;
}

// f(integral constant of the activation): one copy of f for each, so that the
// choice is made once and not for every element.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
        default: f(std::integral_constant<int, kActNone>());
    }
}

// ---- sums and maxima over the lanes ----------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// v combined over aligned groups of L lanes (1 .. 64), the result in every lane,
// by vector instructions alone (a shuffle through the LDS unit costs more than
// the rest of a small kernel: one row of 512 -> 1365 gated 12.0 us with them).
// f is commutative, so lanes may be mirrored once the smaller groups are equal.
template <int L, class F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, F f) {
    if (L >= 2) v = f(v, dpp<0xB1>(v));             // lane ^ 1
    if (L >= 4) v = f(v, dpp<0x4E>(v));             // lane ^ 2
    if (L >= 8) v = f(v, dpp<0x141>(v));            // mirrored in 8
    if (L >= 16) v = f(v, dpp<0x140>(v));           // mirrored in 16
    if (L >= 32) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
        v = f(r.x, r.y);
    }
    if (L >= 64) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
        v = f(r.x, r.y);
    }
    return v;
}

template <int L>
__device__ __forceinline__ float lane_sum(float v) {
    return __uint_as_float(over_lanes<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) SMC_INLINE {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

template <int L>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
    return over_lanes<L>(v, [](uint32_t a, uint32_t b) SMC_INLINE { return a > b ? a : b; });
}

// ---- staging one operand --------------------------------------------------------

// 16 bytes from any element's address.
__device__ __forceinline__ u32x4 load_unaligned(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

__device__ __forceinline__ void store_unaligned(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// 16 bytes a lane from the buffer to LDS, lane l's at lds + 16 l. In assembly
// (it has no output register) because the compiler, where it knows of such
// loads, waits for all of them before every transposing LDS read, and so for
// the next step's; the kernel waits for them itself (wait_vm).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"     // m0 is a reserved register, and it is clobbered
__device__ __forceinline__ void load_to_lds(u32x4 descriptor, uint32_t lds, uint32_t off) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(descriptor)
        : "memory", "m0");
}
#pragma clang diagnostic pop

// Word permutations of the kAcrossK images: over the k rows that one
// transposing read touches (see frag_across, frag_across_e4m3).
__device__ __forceinline__ int swizzle16(int k) { return (k & 3) | ((k >> 1) & 4); }
// e4m3 reads take 16 bytes of the k rows k .. k + 7 and k + 16 .. k + 23 at a time:
// the row's bits that do not choose the bank group by themselves.
template <int ROWS>
__device__ __forceinline__ int swizzle8(int k) {
    return ROWS >= 128 ? ((k >> 1) & 3) | ((k >> 2) & 4) : ((k >> 2) & 1) | ((k >> 3) & 2);
}

// One operand's step of 128 bytes x ROWS into LDS. GATED: row v of the tile is
// column v of the interleaved halves: of every 64, 32 of the gate half, then
// the same 32 of the up half.
template <int ROWS, int LAYOUT, int THREADS, int ESIZE, bool GATED>
struct Stager {
    static constexpr int kWords = ROWS * 8;                 // 16-byte words of a step
    static constexpr int kLoads = kWords / THREADS;
    static constexpr int kPer16 = 16 / ESIZE;               // elements of a word
    static constexpr int kStep = 128 / ESIZE;               // contraction elements of a step
    static_assert(kWords % THREADS == 0, "whole loads");
    uint32_t off[kLoads];                                   // byte offset from the step's base
    uint32_t src;                                           // kAlongK: first k of this lane's words

    __device__ static int gated_col(int v, int j0, int half) {
        const int j = j0 + (v >> 6) * 32 + (v & 31);
        return j < half ? j + ((v & 32) ? half : 0) : -1;
    }

    // row0: the tile's first row (gated: first column of a half); count: rows of
    // the operand (columns for kAcrossK)
    __device__ void setup(int tid, int row0, int64_t ld, int count, int half) {
        src = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + tid;
            if (LAYOUT == kAlongK) {
                const int row = id >> 3;
                src = ((id & 7) ^ (row & 7)) * kPer16;
                // kAlongK bases move with row0 unless gated (two runs of rows)
                const int r = GATED ? gated_col(row, row0, half) : row;
                off[i] = r < 0 ? kOutside : (uint32_t)(r * ld + src) * ESIZE;
            } else {
                int k, v;
                across_word(id, k, v);
                const int col = GATED ? gated_col(v, row0, half) : row0 + v;
                off[i] = col < 0 || col >= count ? kOutside : (uint32_t)(k * ld + col) * ESIZE;
            }
        }
    }
    // kAcrossK: memory row and first column that word `id` of the image holds.
    // 16 columns are permuted together: two words of 16-bit, one of e4m3.
    __device__ static void across_word(int id, int& k, int& v) {
        constexpr int kRowWords = ROWS / kPer16;
        const int pos = id % kRowWords;
        k = id / kRowWords;
        if (ESIZE == 2)
            v = (((pos >> 1) ^ (swizzle16(k) & (ROWS / 16 - 1))) << 4) | ((pos & 1) << 3);
        else
            v = (pos ^ (swizzle8<ROWS>(k) & (ROWS / 16 - 1))) << 4;
    }

    // base: the step's first element (kAlongK: of the tile's first row; else of
    // column 0); bytes: from there to the operand's end; k_left: contraction left,
    // WHOLE where that is known to be a whole step
    template <bool WHOLE>
    __device__ __forceinline__ void load(const char* base, uint32_t bytes, int k_left, char* lds, int wave) const {
        // (the same in every lane, which the compiler does not always see)
        const uint64_t b = (uint64_t)base;
        const u32x4 descriptor = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                                  (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)),
                                  (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
        const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(uint32_t)(uintptr_t)(SMC_LDS char*)lds + wave * 1024);
        const uint32_t dead = !WHOLE && LAYOUT == kAlongK && (int)src >= k_left ? kOutside : 0u;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_to_lds(descriptor, first + i * THREADS * 16, off[i] | dead);
    }

    // The same step through registers, for operands whose rows are not made of
    // 16-byte words: unaligned words, and element by element at the row ends.
    // Every load goes out before the first is waited for.
    __device__ __forceinline__ void fetch(const char* base, uint32_t bytes, int k_left, int tid, int row0,
                                          int count, int half, u32x4 (&w)[kLoads]) const {
        int left[kLoads];                           // elements of the words that exist
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (LAYOUT == kAlongK) {
                left[i] = k_left - (int)src;
            } else {
                int k, v;
                across_word(i * THREADS + tid, k, v);
                left[i] = k >= k_left ? 0 : GATED ? half - (row0 + (v >> 6) * 32 + (v & 31)) : count - row0 - v;
            }
            if (off[i] == kOutside || off[i] + (LAYOUT == kAlongK ? ESIZE : 0) > bytes) left[i] = 0;
            w[i] = (u32x4){0u, 0u, 0u, 0u};
            if (left[i] >= kPer16 && off[i] + 16 <= bytes) w[i] = load_unaligned(base + off[i]);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (left[i] <= 0 || (left[i] >= kPer16 && off[i] + 16 <= bytes)) continue;
#pragma unroll 1
            for (int e = 0; e < kPer16 && e < left[i]; ++e) {
                const uint32_t at = off[i] + e * ESIZE;
                if (at + ESIZE > bytes) break;
                const uint32_t v = ESIZE == 2 ? (uint32_t)*reinterpret_cast<const uint16_t*>(base + at)
                                              : (uint32_t)*reinterpret_cast<const uint8_t*>(base + at);
                const int d = e / (4 / ESIZE);
                const uint32_t placed = v << (8 * ESIZE * (e % (4 / ESIZE)));
                w[i].x |= d == 0 ? placed : 0u;
                w[i].y |= d == 1 ? placed : 0u;
                w[i].z |= d == 2 ? placed : 0u;
                w[i].w |= d == 3 ? placed : 0u;
            }
        }
    }
    __device__ __forceinline__ void commit(char* lds, int tid, const u32x4 (&w)[kLoads]) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(lds + (i * THREADS + tid) * 16) = w[i];
    }
};

// Fragment reads. kAlongK: row `row`, 16-byte word c (contraction 8c .. 8c + 7).
__device__ __forceinline__ u32x4 frag_along(const char* tile, int row, int c) {
    return *reinterpret_cast<const u32x4*>(tile + row * 128 + ((c ^ (row & 7)) << 4));
}

// kAcrossK: the 16 rows from 16 piece, this lane's row l % 16; contraction
// 32 kk + 8 (l / 16) .. + 7 by two transposing reads of 4.
template <int ROWS>
__device__ __forceinline__ u32x4 frag_across(const char* tile, int piece, int kk, int lane) {
    const int s = lane & 15, q = lane >> 4;
    const int k = kk * 32 + q * 8 + (s >> 2);
    const int swz = swizzle16(k) & (ROWS / 16 - 1);       // the same for k + 4
    const char* p = tile + k * (ROWS * 2) + ((piece ^ swz) << 5) + ((s & 3) << 3);
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SMC_LDS s16x4*)(p)));
    const u32x2 hi = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SMC_LDS s16x4*)(p + 4 * ROWS * 2)));
    return (u32x4){lo.x, lo.y, hi.x, hi.y};
}

// The same of e4m3: contraction 64 half + 16 (l / 16) .. + 15 by two reads of 8.
template <int ROWS>
__device__ __forceinline__ u32x4 frag_across_e4m3(const char* tile, int piece, int half, int lane) {
    const int s = lane & 15, q = lane >> 4;
    u32x2 v[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int k = half * 64 + q * 16 + t * 8 + (s >> 1);
        const char* p = tile + k * ROWS + ((piece ^ (swizzle8<ROWS>(k) & (ROWS / 16 - 1))) << 4) + ((s & 1) << 3);
        v[t] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((SMC_LDS i32x2*)(p)));
    }
    return (u32x4){v[0].x, v[0].y, v[1].x, v[1].y};
}

// ---- the kernel -----------------------------------------------------------------

// UNALIGNED: operands that are not whole 16-byte words too.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int BLOCKS_, bool UNALIGNED_ = false>
struct Tile {
    static constexpr bool kUnaligned = UNALIGNED_;
    static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int kThreads = 64 * WAVES_M * WAVES_N;
    static constexpr int MT = BM / (16 * WAVES_M);
    static constexpr int kBlocks = BLOCKS_;             // blocks a CU (LDS and register budget)
    static constexpr int kStepBytes = (BM + BN) * 128;
    static constexpr int kLdsBytes = kStepBytes * STAGES;
    static constexpr int kLoads = (BM + BN) * 8 / kThreads;     // loads a lane and step
    static_assert(BN == 64 * WAVES_N, "a wave owns 64 columns");
    static_assert(kLdsBytes * BLOCKS_ <= 160 * 1024, "LDS");
    static_assert(BLOCKS_ <= kMaxBlocksPerCu, "scratch of the slopes");
};

// 8 consecutive values <-> a lane's two 4-value groups: lanes of odd 16-lane
// rows exchange `lo` with the row below's `hi` (its own inverse).
__device__ __forceinline__ void swap_rows(uint32_t& lo, uint32_t& hi) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(lo, hi, false, false));
    lo = r.x;
    hi = r.y;
}

// The first `count` (at most 8) elements of a row's end, zeros after them.
__device__ __forceinline__ u32x4 load_tail(const uint16_t* p, int count) {
    u32x4 w;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t lo = 2 * d < count ? p[2 * d] : 0u, hi = 2 * d + 1 < count ? p[2 * d + 1] : 0u;
        w[d] = lo | (hi << 16);
    }
    return w;
}

// ---- f16 slopes ---------------------------------------------------------------------
// dz is the operand of two matrix products, so it is rounded to the layers' type
// before dx, dW and db are summed. f16 ends at 65504 and has full precision from
// 2^-14 on, and dz (a gradient times the other half's values, or a gradient that
// nobody scaled) leaves that range where dx and dW do not. So the largest finite
// |dz| is taken along, and where it is above f16's end or below 2^-8 (then values
// 2^-6 of it are still whole, and what the smaller ones lose is a 2^-17 of it) a
// second launch writes dz again times the power of two that brings it to
// [2^14, 2^15); the sums of dx and dW are multiplied by the inverse before they
// are rounded. Within the range the second launch ends at once. bf16 has the
// range of float32. (Two launches, for a scale has to be known before the first
// row is written; bounding it from dy and the weights would be loose by orders.)
// f16 gated backward of 15,000 x 512 -> 2048: 217 us without all this, 227 in range,
// 315 out of it; 300 x 128 -> 96: 16.7, 19.7, 22.9.
__device__ __forceinline__ float range_scale(uint32_t max_bits) {
    const float m = __uint_as_float(max_bits);
    if (m == 0.f || (m >= 0x1p-8f && m <= 65504.f)) return 1.f;
    const int e = 14 - ((int)(max_bits >> 23) - 127);   // 2^e m in [2^14, 2^15), -113 .. 141
    return __uint_as_float((uint32_t)((e < 96 ? e : 96) + 127) << 23);
}

// ---- the epilogue of 16 rows x 64 columns ------------------------------------------
// acc[j] holds row r, columns 16 j + 4 q .. + 3 of the wave's 64; gated: the gate
// half's 32 columns, then the same of the up half. Outputs (and `extra`) are read
// and written as 8 consecutive columns a lane, `kPairs` of them.

template <int EPI>
struct Shape {
    static constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    static constexpr bool kHasExtra = EPI == kEpiStore || EPI == kEpiSlope || EPI == kEpiGatedSlope;
    static constexpr int kPairs = kGated ? 1 : 2;                   // 8-value words of extra
    static constexpr int kOut = EPI == kEpiGated ? 1 : 2;           // 8-value words of out
    // columns of a half (or of out) from column nw on: accumulator (j, e) and word h
    __device__ static int column(int nw, int j, int q, int e) { return nw + (kGated ? (j & 1) : j) * 16 + q * 4 + e; }
    __device__ static int word(int nw, int h, int q) { return nw + (kGated ? 0 : h * 32) + (q & 1) * 16 + (q >> 1) * 8; }
};

// What depends on the columns alone, kept in LDS for the tile (in registers it
// would be 32 of them through the whole contraction): bias and, for e4m3, the
// columns' scales, for virtual column v of the block at [v].
template <int BN, bool E4M3>
struct ColumnTable {
    float bias[BN];
    float scale[E4M3 ? BN : 1];
};

template <int DT, bool E4M3, int EPI, int BN>
__device__ __forceinline__ void fill_columns(ColumnTable<BN, E4M3>& t, const ProductArgs& p, int n0, int width, int v) {
    using Sh = Shape<EPI>;
    if (v >= BN) return;
    const int c = Sh::kGated ? n0 + (v >> 6) * 32 + (v & 31) : n0 + v;
    const int cc = c < width ? c : width - 1;       // past the last column the last one (not stored)
    const int b = Sh::kGated && (v & 32) ? cc + p.half_out : cc;
    t.bias[v] = p.bias ? to_f32<DT>(static_cast<const uint16_t*>(p.bias)[b]) : 0.f;
    if (E4M3) t.scale[v] = p.b_scale[b];
}

// (Past extra's last row or column another is read, where nothing is stored.)
template <int EPI>
__device__ __forceinline__ u32x4 load_extra(const ProductArgs& p, int row, int nw, int h, int q, int width) {
    const int col = Shape<EPI>::word(nw, h, q), own = p.extra_width ? p.extra_width : width;
    const uint16_t* e0 = static_cast<const uint16_t*>(p.extra) + (int64_t)(row < p.m ? row : p.m - 1) * p.ld_extra;
    if (!p.vec_x) return load_tail(e0 + col, own - col);
    u32x4 x = load_unaligned(e0 + (col + 8 <= own ? col : 0));
    if (col < own && col + 8 > own) x = load_tail(e0 + col, own - col);
    return x;
}

// extra's values in the accumulators' order.
template <int DT, int EPI>
__device__ __forceinline__ void unpack_extra(const u32x4 (&extra)[Shape<EPI>::kPairs], float (&x)[4][4]) {
#pragma unroll
    for (int h = 0; h < Shape<EPI>::kPairs; ++h) {
        // (opaque: else all rows' values are unpacked at once, into too many registers)
        u32x4 v = extra[h];
        asm volatile("" : "+v"(v));
        uint32_t l0 = v.x, l1 = v.y, h0 = v.z, h1 = v.w;
        swap_rows(l0, h0);
        swap_rows(l1, h1);
        const uint32_t w[4] = {l0, l1, h0, h1};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[2 * h + (e >> 2)][e & 3] = to_f32<DT>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu);
    }
}

// The values, in place of the sums (kEpiStore: without the residual).
template <int DT, int EPI, int ACT>
__device__ __forceinline__ void row_values(f32x4 (&acc)[4], const u32x4 (&extra)[Shape<EPI>::kPairs]) {
    using Sh = Shape<EPI>;
    float x[4][4];
    if constexpr (EPI == kEpiSlope || EPI == kEpiGatedSlope) unpack_extra<DT, EPI>(extra, x);
#pragma unroll
    for (int j = 0; j < (Sh::kGated ? 2 : 4); ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float z = acc[j][e], u = acc[(j + 2) & 3][e];
            if (EPI == kEpiStore) acc[j][e] = act_value<ACT>(z);
            if (EPI == kEpiSlope) acc[j][e] = x[j][e] * act_slope<ACT>(z);
            if (EPI == kEpiGated) acc[j][e] = act_value<ACT>(z) * u;
            if (EPI == kEpiGatedSlope) {
                acc[j][e] = x[j][e] * u * act_slope<ACT>(z);
                acc[(j + 2) & 3][e] = x[j][e] * act_value<ACT>(z);
            }
        }
}

// The largest finite magnitude, by its bits, of `most` and the first `left` columns
// from the wave's first on (FULL: of all).
template <int EPI, bool FULL>
__device__ __forceinline__ uint32_t row_most(const f32x4 (&acc)[4], uint32_t most, int q, int left) {
    // (opaque: else every comparison of a tile's columns is made once and kept)
    if (!FULL) asm volatile("" : "+v"(left));
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t m = __float_as_uint(acc[j][e]) & 0x7fffffffu;
            most = max(most, m < 0x7f800000u && (FULL || Shape<EPI>::column(0, j, q, e) < left) ? m : 0u);
        }
    return most;
}

template <int DT, int EPI>
__device__ __forceinline__ void row_residual(f32x4 (&acc)[4], const u32x4 (&extra)[Shape<EPI>::kPairs]) {
    float x[4][4];
    unpack_extra<DT, EPI>(extra, x);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += x[j][e];
}

// Rounds and stores them, one store for each whole word, whatever its alignment
// (91,000 rows of 341 columns, gated from 128: 81 us where unaligned words went
// out element by element, 46 so). FULL: the row and its columns exist.
template <int DT, int EPI, bool FULL>
__device__ __forceinline__ void row_store(const ProductArgs& p, const f32x4 (&acc)[4], int row, int nw, int q, int width) {
    using Sh = Shape<EPI>;
#pragma unroll
    for (int h = 0; h < Sh::kOut; ++h) {
        const int col = Sh::word(nw, h, q);     // the second word of a gated pair is the up half's
        uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)row * p.ldo + col + (Sh::kGated && h ? p.half : 0);
        uint32_t l0 = pack2<DT>(acc[2 * h][0], acc[2 * h][1]), l1 = pack2<DT>(acc[2 * h][2], acc[2 * h][3]);
        uint32_t h0 = pack2<DT>(acc[2 * h + 1][0], acc[2 * h + 1][1]);
        uint32_t h1 = pack2<DT>(acc[2 * h + 1][2], acc[2 * h + 1][3]);
        swap_rows(l0, h0);
        swap_rows(l1, h1);
        if (FULL || (row < p.m && col + 8 <= width)) {
            store_unaligned(dst, (u32x4){l0, l1, h0, h1});
        } else if (row < p.m) {
            const uint32_t w[4] = {l0, l1, h0, h1};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < width) dst[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
        }
    }
}

// At most N of this wave's memory operations are still in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N < 64, "a 6-bit counter");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One tile of the walk. Tiles are numbered split by split (kEpiPartial), within
// a split group by group of 2^group_log row tiles, within a group column tile by
// column tile, its row tiles in turn.
template <class T, int EPI>
struct Place {
    int t, in_group, group, tn, tm, n0, split, steps;
    int m0, k0, k_len;
    __device__ int group_rows(const ProductArgs& p) const {
        const int left = p.tiles_m - (group << p.group_log);
        return left < (1 << p.group_log) ? left : 1 << p.group_log;
    }
    __device__ void start(const ProductArgs& p, int tile, int step_k) {
        t = tile;
        split = 0;
        int rest = t;
        if (EPI == kEpiPartial) {
            split = t / (p.tiles_m * p.tiles_n);
            rest = t - split * p.tiles_m * p.tiles_n;
        }
        group = rest / (p.tiles_n << p.group_log);
        in_group = rest - group * (p.tiles_n << p.group_log);
        derive(p, step_k);
    }
    __device__ void advance(const ProductArgs& p, int by, int step_k) {
        t += by;
        in_group += by;
        for (int size = group_rows(p) * p.tiles_n; in_group >= size; size = group_rows(p) * p.tiles_n) {
            in_group -= size;
            ++group;
            if (EPI == kEpiPartial && (group << p.group_log) >= p.tiles_m) {
                group = 0;
                ++split;
            }
        }
        derive(p, step_k);
    }
    __device__ void derive(const ProductArgs& p, int step_k) {
        constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
        const int rows = group_rows(p);
        tn = rows == 1 << p.group_log ? in_group >> p.group_log : in_group / rows;
        tm = (group << p.group_log) + in_group - tn * rows;
        n0 = tn * (kGated ? T::BN / 2 : T::BN);         // gated: column of a half
        m0 = tm * T::BM;
        k0 = split * p.k_split;
        k_len = p.k - k0 < p.k_split ? p.k - k0 : p.k_split;
        // At least one: launch_product refuses empty splits. The walk is written as if
        // there were none now and then, which the compiler schedules better: 91,000 x
        // 128 -> 128 with a residual 15.6 us, as straight code 16.0; e4m3 gated 91,000 x
        // 128 -> 344 from [k, n] weights 59 and 64.
        steps = k_len > 0 ? (k_len + step_k - 1) / step_k : 0;
    }
};

template <int DT, bool E4M3, int LA, int LB, int EPI, class T, bool ALIGNED>
__global__ __launch_bounds__(T::kThreads, T::kBlocks* T::kThreads / 256) void k_product(ProductArgs p) {
    constexpr int MT = T::MT;
    constexpr int ESIZE = E4M3 ? 1 : 2;
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    constexpr bool kHasExtra = EPI == kEpiStore || EPI == kEpiSlope || EPI == kEpiGatedSlope;
    constexpr int kPairs = kGated ? 1 : 2;
    constexpr int kStep = 128 / ESIZE;
    constexpr int S = T::STAGES;
    extern __shared__ __align__(1024) char s_tile[];
    __shared__ __align__(16) ColumnTable<T::BN, E4M3> s_columns;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    // Blocks are dealt to the XCDs in turn; each XCD walks a contiguous run of
    // tiles, its blocks side by side: at any time they read a group of row
    // panels of a that stays in the XCD's L2 and a few column tiles of b.
    const int total = p.tiles_m * p.tiles_n * p.splits;
    const int xcd = blockIdx.x % p.xcds, slot = blockIdx.x / p.xcds;
    const int per = total / p.xcds, more = total % p.xcds;
    const int t_end = (xcd + 1) * per + (xcd + 1 < more ? xcd + 1 : more);
    const int t_step = ((int)gridDim.x - xcd + p.xcds - 1) / p.xcds;
    const int t_first = xcd * per + (xcd < more ? xcd : more) + slot;
    constexpr bool kRanged = DT == kF16 && (EPI == kEpiSlope || EPI == kEpiGatedSlope);
    constexpr bool kUnscale = DT == kF16 && !E4M3 && EPI == kEpiStore && LB == kAlongK;     // the input gradient
    __shared__ uint32_t s_most[kRanged ? T::kThreads / 64 : 1];
    float dz_scale = 1.f;
    uint32_t most = 0;                  // this lane's largest |dz|
    auto block_most = [&]() SMC_INLINE {
        most = lane_max<64>(most);
        if (lane == 0) s_most[wave] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T::kThreads / 64; ++w) most = max(most, s_most[w]);
    };
    if constexpr (kRanged) {
        if (p.dz_unscale) {
            for (int i = tid; i < (int)gridDim.x; i += T::kThreads) most = max(most, __float_as_uint(p.dz_max[i]));
            block_most();
            dz_scale = __uint_as_float(
                (uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(range_scale(most))));
            if (blockIdx.x == 0 && tid == 0) *p.dz_unscale = 1.f / dz_scale;
            if (dz_scale == 1.f) return;
        } else if (t_first >= t_end && tid == 0) {
            p.dz_max[blockIdx.x] = 0.f;
        }
    }
    if (t_first >= t_end) return;

    // ---- loads: the step that is issued next, S - 1 steps ahead ----
    Place<T, EPI> ahead;
    Stager<T::BM, LA, T::kThreads, ESIZE, false> sa;
    Stager<T::BN, LB, T::kThreads, ESIZE, kGated> sb;
    const char *next_a, *next_b;        // first element of the next step
    const char *end_a = nullptr, *end_b = nullptr;      // along k: the end of the tile's rows
    uint32_t bytes_a, bytes_b;          // from there to the operand's end (for a whole step)
    int ahead_step = 0;
    int ahead_buf = 0;                  // byte offset of the buffer it goes to
    // along k a step is 128 bytes further in every row; across k, 128 / ESIZE rows on
    const int64_t by_a = LA == kAlongK ? 128 : (int64_t)kStep * p.lda * ESIZE;
    const int64_t by_b = LB == kAlongK ? 128 : (int64_t)kStep * p.ldb * ESIZE;
    // The range check is by 4-byte words: a last element that fills one only
    // partly needs the whole word in range (aligned, so on its page).
    auto whole_words = [](int64_t bytes) SMC_INLINE { return (uint32_t)(bytes + 3) & ~3u; };
    auto enter = [&](bool first, bool new_rows, bool new_columns) SMC_INLINE {
        ahead_step = 0;
        // along k a tile's rows are told by the base alone
        if (first || (LA == kAcrossK && new_rows))
            sa.setup(tid, LA == kAlongK ? 0 : ahead.m0, p.lda, p.m, 0);
        if (first || ((LB == kAcrossK || kGated) && new_columns))
            sb.setup(tid, LB == kAlongK && !kGated ? 0 : ahead.n0, p.ldb, p.n, p.half);
        const int rows_a = p.m - ahead.m0 < T::BM ? p.m - ahead.m0 : T::BM;
        const int rows_b = kGated ? p.n : (p.n - ahead.n0 < T::BN ? p.n - ahead.n0 : T::BN);
        next_a = static_cast<const char*>(p.a) +
                 (LA == kAlongK ? (int64_t)ahead.m0 * p.lda + ahead.k0 : (int64_t)ahead.k0 * p.lda) * ESIZE;
        next_b = static_cast<const char*>(p.b) +
                 (LB == kAlongK ? (int64_t)(kGated ? 0 : ahead.n0) * p.ldb + ahead.k0 : (int64_t)ahead.k0 * p.ldb) * ESIZE;
        if (LA == kAlongK) end_a = next_a + ((int64_t)(rows_a - 1) * p.lda + p.k - ahead.k0) * ESIZE;
        if (LB == kAlongK) end_b = next_b + ((int64_t)(rows_b - 1) * p.ldb + p.k - ahead.k0) * ESIZE;
        bytes_a = whole_words((LA == kAlongK ? (rows_a - 1) * p.lda + p.k - ahead.k0
                                             : (kStep - 1) * p.lda + p.m) * ESIZE);
        bytes_b = whole_words((LB == kAlongK ? (rows_b - 1) * p.ldb + p.k - ahead.k0
                                             : (kStep - 1) * p.ldb + p.n) * ESIZE);
    };
    auto issued = [&]() SMC_INLINE {
        next_a += by_a;
        next_b += by_b;
        if (LA == kAlongK) bytes_a -= 128;
        if (LB == kAlongK) bytes_b -= 128;
        ++ahead_step;
        ahead_buf = ahead_buf == (S - 1) * T::kStepBytes ? 0 : ahead_buf + T::kStepBytes;
    };
    // a step that is known to exist and to be whole
    auto issue_whole = [&]() SMC_INLINE {
        char* dst = s_tile + ahead_buf;
        sa.template load<true>(next_a, bytes_a, kStep, dst, wave);
        sb.template load<true>(next_b, bytes_b, kStep, dst + T::BM * 128, wave);
        issued();
    };
    // moves on to a step that exists; false when the walk is over
    auto next_step = [&]() SMC_INLINE {
        while (ahead_step >= ahead.steps) {             // (once: see Place::derive)
            if (ahead.t + t_step >= t_end) return false;
            const int tm = ahead.tm, tn = ahead.tn;
            ahead.advance(p, t_step, kStep);
            enter(false, ahead.tm != tm, ahead.tn != tn);
        }
        return true;
    };
    auto step_left = [&]() SMC_INLINE {                 // contraction elements of it
        const int rest = ahead.k_len - ahead_step * kStep;
        return rest < kStep ? rest : kStep;
    };
    // any step, whole words
    auto issue = [&]() SMC_INLINE {
        if (!next_step()) return false;
        const int left = step_left();
        char* dst = s_tile + ahead_buf;
        sa.template load<false>(next_a, LA == kAlongK ? bytes_a : whole_words(((left - 1) * p.lda + p.m) * ESIZE),
                                left, dst, wave);
        sb.template load<false>(next_b, LB == kAlongK ? bytes_b : whole_words(((left - 1) * p.ldb + p.n) * ESIZE),
                                left, dst + T::BM * 128, wave);
        issued();
        return true;
    };
    // Operands that are not whole words: a step's words are held in registers
    // while the step before it is multiplied, then put into LDS.
    u32x4 held_a[decltype(sa)::kLoads], held_b[decltype(sb)::kLoads];
    auto fetch = [&]() SMC_INLINE {
        if (!next_step()) return false;
        const int left = step_left();
        // (bytes to the operand's end itself, not in whole words)
        sa.fetch(next_a, LA == kAlongK ? (uint32_t)(end_a - next_a) : (uint32_t)(((left - 1) * p.lda + p.m) * ESIZE),
                 left, tid, ahead.m0, p.m, 0, held_a);
        sb.fetch(next_b, LB == kAlongK ? (uint32_t)(end_b - next_b) : (uint32_t)(((left - 1) * p.ldb + p.n) * ESIZE),
                 left, tid, ahead.n0, p.n, p.half, held_b);
        return true;
    };
    auto commit = [&]() SMC_INLINE {
        sa.commit(s_tile + ahead_buf, tid, held_a);
        sb.commit(s_tile + ahead_buf + T::BM * 128, tid, held_b);
        issued();
    };

    ahead.start(p, t_first, kStep);
    Place<T, EPI> here = ahead;
    enter(true, true, true);
    // The vector memory counter is in order: the oldest step in flight has landed
    // when no more operations are left than were issued after it. `ops` counts the
    // operations that are certain (a step's loads, the loads of extra in words,
    // the stores of a full tile); others only make a wait longer.
    int ops = 0, mark[S] = {}, in_flight = 0;           // mark: ops when a step had been issued
    bool over = false;                                  // every step has been issued
    auto issued_one = [&]() SMC_INLINE {
        ops += T::kLoads;
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (i == in_flight) mark[i] = ops;
        ++in_flight;
    };
    if constexpr (ALIGNED) {
#pragma unroll 1
        for (int i = 0; i < S; ++i) {
            over = !issue();
            if (!over) issued_one();
        }
    } else {
        over = !fetch();
        if (!over) commit();
    }

    int buf = 0;                        // byte offset of the step's buffer
#pragma unroll 1
    for (;; here.advance(p, t_step, kStep)) {
        // What the epilogue reads: columns of this lane's pair of 4-value groups
        // and of its 8 stored values. Past the last row or column the last one
        // is read (and not stored), so that the loads need no branches.
        const int width = kGated ? p.half_out : p.n;    // columns of out (and extra)
        const int nw = here.n0 + wn * (kGated ? 32 : 64);
        const int row_base = here.m0 + wm * MT * 16 + r;
        u32x4 extra[MT][kPairs];
        float ascale[MT];
        auto load_epilogue = [&]() SMC_INLINE {
            if constexpr (EPI != kEpiPartial) {
                if (E4M3 || p.bias) fill_columns<DT, E4M3, EPI, T::BN>(s_columns, p, here.n0, width, tid);
                if (E4M3) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const int row = row_base + i * 16;
                        ascale[i] = p.a_scale[row < p.m ? row : p.m - 1];
                    }
                }
            }
            if constexpr (kHasExtra) {
                if (p.extra) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < kPairs; ++h)
                            extra[i][h] = load_extra<EPI>(p, row_base + i * 16, nw, h, q, width);
                }
            }
        };

        f32x4 acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        f32x4 sum[4];                           // column sums of b (kEpiPartial)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        const bool colsum = EPI == kEpiPartial && p.colsum && here.tm == 0 && wm == 0;

        // One step: the products of the buffer at `buf`.
        auto compute = [&]() SMC_INLINE {
            const char* ta = s_tile + buf;
            const char* tb = ta + T::BM * 128;
            buf = buf == (S - 1) * T::kStepBytes ? 0 : buf + T::kStepBytes;
            if constexpr (E4M3) {
                u32x4 fb[4][2], fa[MT][2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        fb[j][h] = LB == kAlongK ? frag_along(tb, wn * 64 + j * 16 + r, 4 * h + q)
                                                 : frag_across_e4m3<T::BN>(tb, wn * 4 + j, h, lane);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) fa[i][h] = frag_along(ta, (wm * MT + i) * 16 + r, 4 * h + q);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = mfma_e4m3(fb[j][0], fb[j][1], fa[i][0], fa[i][1], acc[i][j]);
                __builtin_amdgcn_s_setprio(0);
            } else {
                u32x4 fb[2][4], fa[2][MT];
                auto read = [&](int kk) SMC_INLINE {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        fb[kk][j] = LB == kAlongK ? frag_along(tb, wn * 64 + j * 16 + r, kk * 4 + q)
                                                  : frag_across<T::BN>(tb, wn * 4 + j, kk, lane);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        fa[kk][i] = LA == kAlongK ? frag_along(ta, (wm * MT + i) * 16 + r, kk * 4 + q)
                                                  : frag_across<T::BM>(ta, wm * MT + i, kk, lane);
                };
                auto multiply = [&](int kk) SMC_INLINE {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<DT>(fb[kk][j], fa[kk][i], acc[i][j]);
                };
                // the second half's reads go out between the first half's products
                read(0);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
                multiply(0);
                read(1);
                constexpr int kReads = (LB == kAlongK ? 4 : 8) + (LA == kAlongK ? MT : 2 * MT);
                constexpr int kBetween = MT * 4 / kReads > 0 ? MT * 4 / kReads : 1;
#pragma unroll
                for (int i = 0; i < kReads; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, kBetween, 0);   // MFMA
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);          // LDS read
                }
                __builtin_amdgcn_sched_barrier(0);
                multiply(1);
                __builtin_amdgcn_s_setprio(0);
                if (EPI == kEpiPartial && colsum) {
                    constexpr uint32_t one = DT == kF16 ? 0x3c003c00u : 0x3f803f80u;
                    const u32x4 ones = {one, one, one, one};
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum[j] = mfma16<DT>(fb[kk][j], ones, sum[j]);
                }
            }
        };

        // At a step's start its words have landed, and every wave is done with the
        // buffer that the next loads overwrite.
        auto arrive = [&]() SMC_INLINE {
            constexpr int kSteady = (S - 2) * T::kLoads;
            const int newer = ops - mark[0];
            if (newer == kSteady)
                wait_vm<kSteady>();
            else if (newer >= 16)
                wait_vm<16>();
            else if (newer >= 12)
                wait_vm<12>();
            else if (newer >= 8)
                wait_vm<8>();
            else if (newer >= 4)
                wait_vm<4>();
            else
                wait_vm<0>();
#pragma unroll
            for (int i = 0; i + 1 < S; ++i) mark[i] = mark[i + 1];
            --in_flight;
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        // S steps are in flight at a tile's start: its first step issues none.
        // What the epilogue reads is loaded beside it, two steps before a wait
        // includes it.
        if constexpr (ALIGNED) {
            int step = 0;
            if (here.steps > 0) {                       // (always: see Place::derive)
                arrive();
                load_epilogue();
                if (kHasExtra && p.extra && p.vec_x) ops += MT * kPairs;
                compute();
                ++step;
            }
            // the step issued is a whole one of this tile
            const int main_steps = here.k_len / kStep - (S - 1);
#pragma unroll 1
            for (; step < main_steps; ++step) {
                arrive();
                issue_whole();
                issued_one();
                compute();
            }
#pragma unroll 1
            for (; step < here.steps; ++step) {
                arrive();
                if (!over) {
                    over = !issue();
                    if (!over) issued_one();
                }
                compute();
            }
            if (kHasExtra && p.extra) {
                // the compiler's own wait for them belongs here, before the next
                // tile's loads, which it does not count
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < kPairs; ++h) asm volatile("" : "+v"(extra[i][h]));
            }
            // The last step's buffer is free once every wave has read it.
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (!over) {
                over = !issue();
                if (!over) issued_one();
            }
        } else {
#pragma unroll 1
            for (int step = 0; step < here.steps; ++step) {
                __syncthreads();                        // the step's words are in LDS
                const bool more = !over && fetch();
                over = !more;
                if (step == 0) load_epilogue();
                compute();
                if (more) commit();
            }
            __syncthreads();                            // (the column table of a one-step tile)
        }

        // ---- epilogue: acc[i][j] holds row 16 i + r, columns 16 j + 4 q .. + 3 ----
        if constexpr (EPI == kEpiPartial) {
            float* part = p.part + (int64_t)here.split * (p.m + p.colsum) * p.n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = here.n0 + wn * 64 + j * 16 + q * 4;
                if (col >= p.n) continue;
                const bool whole = col + 4 <= p.n && (p.n & 3) == 0;
#pragma unroll
                for (int i = 0; i <= MT; ++i) {
                    const bool is_sum = i == MT;
                    const int row = is_sum ? p.m : row_base + i * 16;
                    if (is_sum ? !(colsum && r == 0) : row >= p.m) continue;
                    const f32x4 v = is_sum ? sum[j] : acc[i < MT ? i : 0][j];
                    float* o = part + (int64_t)row * p.n + col;
                    if (whole) {
                        *reinterpret_cast<f32x4*>(o) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (col + e < p.n) o[e] = v[e];
                    }
                }
            }
        } else {
            if (E4M3 || p.bias) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = wn * 64 + j * 16 + q * 4;
                    const f32x4 b = *reinterpret_cast<const f32x4*>(&s_columns.bias[v]);
                    if constexpr (E4M3) {
                        const f32x4 sc = *reinterpret_cast<const f32x4*>(&s_columns.scale[v]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) acc[i][j] = acc[i][j] * (ascale[i] * sc) + b;
                    } else {
#pragma unroll
                        for (int i = 0; i < MT; ++i) acc[i][j] += b;
                    }
                }
            }
            if constexpr (kUnscale) {
                if (p.unscale) {
                    const float by = *p.unscale;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] *= by;
                }
            }
            with_act(p.act, [&](auto act_c) SMC_INLINE {
                constexpr int ACT = decltype(act_c)::value;
#pragma unroll
                for (int i = 0; i < MT; ++i) row_values<DT, EPI, ACT>(acc[i], extra[i]);
            });
            if constexpr (EPI == kEpiStore) {
                if (p.extra) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) row_residual<DT, EPI>(acc[i], extra[i]);
                }
            }
            // in a full tile as many stores as the waits above rely on
            const bool full = here.m0 + T::BM <= p.m &&
                              here.n0 + (kGated ? T::BN / 2 : T::BN) <= width;
            if constexpr (kRanged) {
                if (p.dz_unscale) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] *= dz_scale;
                } else if (full) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) most = row_most<EPI, true>(acc[i], most, q, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        most = row_most<EPI, false>(acc[i], most, q, row_base + i * 16 < p.m ? width - nw : 0);
                }
            }
            if (full) {
#pragma unroll
                for (int i = 0; i < MT; ++i) row_store<DT, EPI, true>(p, acc[i], row_base + i * 16, nw, q, width);
            } else {
#pragma unroll
                for (int i = 0; i < MT; ++i) row_store<DT, EPI, false>(p, acc[i], row_base + i * 16, nw, q, width);
            }
            if (full) ops += MT * Shape<EPI>::kOut;
        }
        if (here.t + t_step >= t_end) break;
    }
    if constexpr (kRanged) {
        if (!p.dz_unscale) {
            block_most();
            if (tid == 0) p.dz_max[blockIdx.x] = __uint_as_float(most);
        }
    }
}

// Lets a kernel take `bytes` of dynamic LDS (above 64 KiB it has to be asked for).
template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DT, bool E4M3, int LA, int LB, int EPI, class T, bool ALIGNED>
hipError_t launch_aligned(const ProductArgs& p, int64_t total, hipStream_t s) {
    static const hipError_t ok = allow_lds(k_product<DT, E4M3, LA, LB, EPI, T, ALIGNED>, T::kLdsBytes);
    if (ok != hipSuccess) return ok;
    const int64_t resident = (int64_t)T::kBlocks * device_cus();    // each walks several tiles
    launch(k_product<DT, E4M3, LA, LB, EPI, T, ALIGNED>, dim3((unsigned)(total < resident ? total : resident)),
           dim3(T::kThreads), T::kLdsBytes, s, p);
    return hipGetLastError();
}

template <int DT, bool E4M3, int LA, int LB, int EPI, class T>
hipError_t launch_product(ProductArgs p, hipStream_t s) {
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    p.tiles_m = (int)((p.m + T::BM - 1) / T::BM);
    p.tiles_n = kGated ? (p.half + T::BN / 2 - 1) / (T::BN / 2) : (p.n + T::BN - 1) / T::BN;
    if (!p.half_out) p.half_out = p.half;
    const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.splits;
    if (total <= 0) return hipSuccess;
    if (total > 0x7fffffff) return hipErrorInvalidValue;
    // the walk counts on a step in every tile
    if (p.k_split <= 0 || (int64_t)(p.splits - 1) * p.k_split >= p.k) return hipErrorInvalidValue;
    // row tiles a group: 1 MiB of a at most, a quarter of an XCD's L2 (columns
    // fastest over single row tiles, b was read from memory again for nearly
    // every row tile: 15,000 x 512 -> 4096 backward 380 MB of fetches)
    p.group_log = 0;
    while (p.group_log < 6 && ((int64_t)T::BM * p.k * (E4M3 ? 1 : 2) << (p.group_log + 1)) <= (1 << 20))
        ++p.group_log;
    if (EPI == kEpiPartial) p.group_log = 0;
    if (p.vec_a && p.vec_b) return launch_aligned<DT, E4M3, LA, LB, EPI, T, true>(p, total, s);
    // (backward passes have their operands aligned)
    if constexpr (T::kUnaligned && (EPI == kEpiStore || EPI == kEpiGated) && (E4M3 || LB == kAcrossK))
        return launch_aligned<DT, E4M3, LA, LB, EPI, T, false>(p, total, s);
    return hipErrorInvalidValue;                    // (launch_tiled picks a tile that takes them)
}

typedef Tile<128, 128, 2, 2, 2, 2> TileMid;             // 64 x 64 a wave
typedef Tile<128, 128, 4, 2, 2, 2, true> TileWide;      // 32 x 64 a wave, twice the waves
typedef Tile<64, 128, 2, 2, 2, 3, true> TileRows;       // three blocks a CU
typedef Tile<32, 64, 2, 1, 6, 2, true> TileSmall;       // deep: few blocks, long contractions

}  // namespace
}  // namespace smc
