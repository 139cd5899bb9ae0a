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
// Edges. The buffer descriptors end at the operand's last valid element, and a
// lane whose word is past the end of a row gets an offset outside: such loads
// write zeros to LDS, so every edge multiplies by exact zeros on both sides.
#pragma once

#include "pointwise.h"

namespace smc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define SMC_LDS __attribute__((address_space(3)))

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
    return from_f32<DT>(a) | (from_f32<DT>(b) << 16);
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

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case kActRelu: return z < 0.f ? 0.f : z;
        case kActSilu: return z * sigmoid(z);
        case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case kActRelu: return z > 0.f ? 1.f : 0.f;
        case kActSilu: {
            const float g = sigmoid(z);
            return g * (1.f + z * (1.f - g));
        }
        case kActGelu:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
                   z * 0.39894228040143268f * __expf(-0.5f * z * z);
        default: return 1.f;
    }
}

// ---- staging one operand --------------------------------------------------------

// 16 bytes a lane from the buffer to LDS, lane l's at lds + 16 l. (Kept out of
// the templates: the host pass drops a template that calls this builtin with a
// size of 16 without a word.)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (SMC_LDS void*)lds, 16, off, 0, 0, 0);
}

// Word permutations of the kAcrossK images: over the k rows that one
// transposing read touches (see frag_across, frag_across_e4m3).
__device__ __forceinline__ int swizzle16(int k) { return (k & 3) | ((k >> 1) & 4); }
__device__ __forceinline__ int swizzle8(int k) { return k & 7; }

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
            v = (pos ^ (swizzle8(k) & (ROWS / 16 - 1))) << 4;
    }

    // base: the step's first element (kAlongK: of the tile's first row; else of
    // column 0); bytes: from there to the operand's end; k_left: contraction left
    __device__ void load(const char* base, uint32_t bytes, int k_left, char* lds, int wave) const {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(base), 0, (int)bytes, 0x00020000);
        const uint32_t dead = LAYOUT == kAlongK && (int)src >= k_left ? kOutside : 0u;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(r, lds + (i * THREADS + wave * 64) * 16, off[i] | dead);
    }

    // The same step by element loads, for operands that 16-byte words do not fit.
    __device__ void load_elements(const char* base, uint32_t bytes, int k_left, int tid, char* lds,
                                  int row0, int count, int half) const {
#pragma unroll 1
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + tid;
            uint32_t o = off[0];                // selected without a register array index
#pragma unroll
            for (int j = 1; j < kLoads; ++j) o = i == j ? off[j] : o;
            int left;                           // elements of this word that exist
            if (LAYOUT == kAlongK) {
                left = k_left - (int)src;
            } else {
                int k, v;
                across_word(id, k, v);
                left = k < k_left ? (GATED ? half - (row0 + (v >> 6) * 32 + (v & 31)) : count - row0 - v) : 0;
            }
            if (o == kOutside) left = 0;
            u32x4 w;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t u = 0;
#pragma unroll
                for (int e = 0; e < 4 / ESIZE; ++e) {
                    const int el = d * (4 / ESIZE) + e;
                    const uint32_t at = o + el * ESIZE;
                    if (el < left && at + ESIZE <= bytes)
                        u |= (ESIZE == 2 ? (uint32_t)*reinterpret_cast<const uint16_t*>(base + at)
                                         : (uint32_t)*reinterpret_cast<const uint8_t*>(base + at))
                             << (8 * ESIZE * e);
                }
                w[d] = u;
            }
            *reinterpret_cast<u32x4*>(lds + id * 16) = w;
        }
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
        const char* p = tile + k * ROWS + ((piece ^ (swizzle8(k) & (ROWS / 16 - 1))) << 4) + ((s & 1) << 3);
        v[t] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((SMC_LDS i32x2*)(p)));
    }
    return (u32x4){v[0].x, v[0].y, v[1].x, v[1].y};
}

// ---- the kernel -----------------------------------------------------------------

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int BLOCKS_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int kThreads = 64 * WAVES_M * WAVES_N;
    static constexpr int MT = BM / (16 * WAVES_M);
    static constexpr int kBlocks = BLOCKS_;             // blocks a CU (register budget)
    static constexpr int kStepBytes = (BM + BN) * 128;
    static constexpr int kLdsBytes = kStepBytes * STAGES;
    static_assert(BN == 64 * WAVES_N, "a wave owns 64 columns");
};

// 8 consecutive values <-> a lane's two 4-value groups: lanes of odd 16-lane
// rows exchange `lo` with the row below's `hi` (its own inverse).
__device__ __forceinline__ void swap_rows(uint32_t& lo, uint32_t& hi) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(lo, hi, false, false));
    lo = r.x;
    hi = r.y;
}

template <int DT, bool E4M3, int LA, int LB, int EPI, class T, bool ALIGNED>
__global__ __launch_bounds__(T::kThreads, T::kBlocks* T::kThreads / 256) void k_product(ProductArgs p) {
    constexpr int MT = T::MT;
    constexpr int ESIZE = E4M3 ? 1 : 2;
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    constexpr int kStep = 128 / ESIZE;
    extern __shared__ __align__(1024) char s_tile[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    // Blocks are dealt to the XCDs in turn; each XCD walks a contiguous run of
    // tiles, columns fastest, so a row panel is read into one L2.
    const int total = p.tiles_m * p.tiles_n * p.splits;
    int t;
    {
        const int x = blockIdx.x % p.xcds, i = blockIdx.x / p.xcds;
        const int per = total / p.xcds, more = total % p.xcds;
        t = x * per + (x < more ? x : more) + i;
    }
    const int tn = t % p.tiles_n;
    const int tm = (t / p.tiles_n) % p.tiles_m;
    const int split = t / (p.tiles_n * p.tiles_m);
    const int64_t m0 = (int64_t)tm * T::BM;
    const int n0 = kGated ? tn * (T::BN / 2) : tn * T::BN;      // gated: column of a half
    const int64_t k0 = split * p.k_split;
    const int64_t k_len = (p.k - k0 < p.k_split ? p.k - k0 : p.k_split);
    const int steps = (int)((k_len + kStep - 1) / kStep);

    Stager<T::BM, LA, T::kThreads, ESIZE, false> sa;
    Stager<T::BN, LB, T::kThreads, ESIZE, kGated> sb;
    sa.setup(tid, (int)(LA == kAlongK ? 0 : m0), p.lda, (int)p.m, 0);
    sb.setup(tid, LB == kAlongK && !kGated ? 0 : n0, p.ldb, p.n, p.half);
    const int rows_a = (int)(p.m - m0 < T::BM ? p.m - m0 : T::BM);
    const int rows_b = kGated ? p.n : (p.n - n0 < T::BN ? p.n - n0 : T::BN);
    const char* base_a = static_cast<const char*>(p.a) +
                         (LA == kAlongK ? m0 * p.lda + k0 : k0 * p.lda) * ESIZE;
    const char* base_b = static_cast<const char*>(p.b) +
                         (LB == kAlongK ? (kGated ? 0 : n0) * p.ldb + k0 : k0 * p.ldb) * ESIZE;

    auto issue = [&](int step) {
        const int kd = step * kStep;
        const int64_t left64 = k_len - kd;
        const int left = (int)(left64 < kStep ? left64 : kStep);
        char* dst = s_tile + (step % T::STAGES) * T::kStepBytes;
        const int64_t k_rest = p.k - k0 - kd;       // along k the row goes on past a split's end
        const char* pa = base_a + (LA == kAlongK ? (int64_t)kd : kd * p.lda) * ESIZE;
        const char* pb = base_b + (LB == kAlongK ? (int64_t)kd : kd * p.ldb) * ESIZE;
        const uint32_t ba = (uint32_t)((LA == kAlongK ? (rows_a - 1) * p.lda + k_rest
                                                      : (left - 1) * p.lda + p.m) * ESIZE);
        const uint32_t bb = (uint32_t)((LB == kAlongK ? (rows_b - 1) * p.ldb + k_rest
                                                      : (left - 1) * p.ldb + p.n) * ESIZE);
        // the range check is by 4-byte words: a last element that fills one
        // only partly needs the whole word in range (aligned, so on its page)
        const uint32_t wa = (ba + 3) & ~3u, wb = (bb + 3) & ~3u;
        if (ALIGNED || p.vec_a)
            sa.load(pa, wa, left, dst, wave);
        else
            sa.load_elements(pa, ba, left, tid, dst, (int)m0, (int)p.m, 0);
        if (ALIGNED || p.vec_b)
            sb.load(pb, wb, left, dst + T::BM * 128, wave);
        else
            sb.load_elements(pb, bb, left, tid, dst + T::BM * 128, n0, p.n, p.half);
    };

    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    f32x4 sum[4];                                   // column sums of b (kEpiPartial)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const bool colsum = EPI == kEpiPartial && p.colsum && tm == 0 && wm == 0;

#pragma unroll 1
    for (int st = 0; st < T::STAGES - 1 && st < steps; ++st) issue(st);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
        // this step's words have landed, and every wave is done with the buffer
        // that the next loads will overwrite
        if (ALIGNED)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        else
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (step + T::STAGES - 1 < steps) issue(step + T::STAGES - 1);
        const char* ta = s_tile + (step % T::STAGES) * T::kStepBytes;
        const char* tb = ta + T::BM * 128;
        if constexpr (E4M3) {
            u32x4 fb[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fb[j][h] = LB == kAlongK ? frag_along(tb, wn * 64 + j * 16 + r, 4 * h + q)
                                             : frag_across_e4m3<T::BN>(tb, wn * 4 + j, h, lane);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const u32x4 a0 = frag_along(ta, (wm * MT + i) * 16 + r, q);
                const u32x4 a1 = frag_along(ta, (wm * MT + i) * 16 + r, 4 + q);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma_e4m3(fb[j][0], fb[j][1], a0, a1, acc[i][j]);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                u32x4 fb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    fb[j] = LB == kAlongK ? frag_along(tb, wn * 64 + j * 16 + r, kk * 4 + q)
                                          : frag_across<T::BN>(tb, wn * 4 + j, kk, lane);
                u32x4 fa[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    fa[i] = LA == kAlongK ? frag_along(ta, (wm * MT + i) * 16 + r, kk * 4 + q)
                                          : frag_across<T::BM>(ta, wm * MT + i, kk, lane);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
                if (EPI == kEpiPartial && colsum) {
                    constexpr uint32_t one = DT == kF16 ? 0x3c003c00u : 0x3f803f80u;
                    const u32x4 ones = {one, one, one, one};
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = mfma16<DT>(fb[j], ones, sum[j]);
                }
            }
        }
    }

    // ---- epilogue: acc[i][j] holds row 16 i + r, columns 16 j + 4 q .. + 3 ----
    const int64_t row_base = m0 + wm * MT * 16 + r;
    if constexpr (EPI == kEpiPartial) {
        float* part = p.part + (int64_t)split * (p.m + p.colsum) * p.n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + wn * 64 + j * 16 + q * 4;
            if (col >= p.n) continue;
            const bool whole = col + 4 <= p.n && (p.n & 3) == 0;
#pragma unroll
            for (int i = 0; i <= MT; ++i) {
                const bool is_sum = i == MT;
                const int64_t row = is_sum ? p.m : row_base + i * 16;
                if (is_sum ? !(colsum && r == 0) : row >= p.m) continue;
                const f32x4 v = is_sum ? sum[j] : acc[i < MT ? i : 0][j];
                float* o = part + row * p.n + col;
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
        // columns of this lane's pair of 4-value groups, and of its 8 stored values
        constexpr int kPairs = kGated ? 1 : 2;
        const int width = kGated ? p.half : p.n;            // columns of out (and extra)
        const int nw = n0 + wn * (kGated ? 32 : 64);
        float bias[4][4], bscale[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = nw + (kGated ? (j & 1) : j) * 16 + q * 4 + e;
                const int b = kGated && j >= 2 ? c + p.half : c;
                bias[j][e] = p.bias && c < width ? to_f32<DT>(static_cast<const uint16_t*>(p.bias)[b]) : 0.f;
                if (E4M3) bscale[j][e] = c < width ? p.b_scale[b] : 0.f;
            }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t row = row_base + i * 16;
            const bool row_ok = row < p.m;
            if (E4M3) {
                const float as = row_ok ? p.a_scale[row] : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] *= as * bscale[j][e];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] += bias[j][e];
#pragma unroll
            for (int h = 0; h < kPairs; ++h) {
                const int col = nw + h * 32 + (q & 1) * 16 + (q >> 1) * 8;   // 8 values stored
                const bool whole = row_ok && p.vec_o && col + 8 <= width;
                // extra's 8 values, then exchanged to the accumulators' order
                float ex[2][4];
                if (EPI == kEpiSlope || EPI == kEpiGatedSlope || (EPI == kEpiStore && p.extra)) {
                    u32x4 x = {0u, 0u, 0u, 0u};
                    const uint16_t* e0 = static_cast<const uint16_t*>(p.extra) + row * p.ld_extra + col;
                    if (whole) {
                        x = *reinterpret_cast<const u32x4*>(e0);
                    } else if (row_ok) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = col + e < width ? e0[e] : 0u;
                        x = (u32x4){v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                                    v[6] | (v[7] << 16)};
                    }
                    uint32_t l0 = x.x, l1 = x.y, h0 = x.z, h1 = x.w;
                    swap_rows(l0, h0);
                    swap_rows(l1, h1);
                    ex[0][0] = to_f32<DT>(l0 & 0xffffu); ex[0][1] = to_f32<DT>(l0 >> 16);
                    ex[0][2] = to_f32<DT>(l1 & 0xffffu); ex[0][3] = to_f32<DT>(l1 >> 16);
                    ex[1][0] = to_f32<DT>(h0 & 0xffffu); ex[1][1] = to_f32<DT>(h0 >> 16);
                    ex[1][2] = to_f32<DT>(h1 & 0xffffu); ex[1][3] = to_f32<DT>(h1 >> 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ex[e >> 2][e & 3] = 0.f;
                }
                float v[2][2][4];                   // [output part][group][value]
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = acc[i][h * 2 + g][e];
                        if (EPI == kEpiStore) {
                            v[0][g][e] = act_value(z, p.act) + ex[g][e];
                        } else if (EPI == kEpiSlope) {
                            v[0][g][e] = ex[g][e] * act_slope(z, p.act);
                        } else {
                            const float u = acc[i][2 + g][e];
                            if (EPI == kEpiGated) {
                                v[0][g][e] = act_value(z, p.act) * u;
                            } else {
                                v[0][g][e] = ex[g][e] * u * act_slope(z, p.act);
                                v[1][g][e] = ex[g][e] * act_value(z, p.act);
                            }
                        }
                    }
#pragma unroll
                for (int o = 0; o < (EPI == kEpiGatedSlope ? 2 : 1); ++o) {
                    uint32_t l0 = pack2<DT>(v[o][0][0], v[o][0][1]), l1 = pack2<DT>(v[o][0][2], v[o][0][3]);
                    uint32_t h0 = pack2<DT>(v[o][1][0], v[o][1][1]), h1 = pack2<DT>(v[o][1][2], v[o][1][3]);
                    swap_rows(l0, h0);
                    swap_rows(l1, h1);
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + row * p.ldo + col + (o ? p.half : 0);
                    if (whole) {
                        *reinterpret_cast<u32x4*>(dst) = (u32x4){l0, l1, h0, h1};
                    } else if (row_ok) {
                        const uint32_t w[4] = {l0, l1, h0, h1};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e < width) dst[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
                    }
                }
            }
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
hipError_t launch_aligned(const ProductArgs& p, unsigned blocks, hipStream_t s) {
    static const hipError_t ok = allow_lds(k_product<DT, E4M3, LA, LB, EPI, T, ALIGNED>, T::kLdsBytes);
    if (ok != hipSuccess) return ok;
    launch(k_product<DT, E4M3, LA, LB, EPI, T, ALIGNED>, dim3(blocks), dim3(T::kThreads), T::kLdsBytes, s, p);
    return hipGetLastError();
}

template <int DT, bool E4M3, int LA, int LB, int EPI, class T>
hipError_t launch_product(ProductArgs p, hipStream_t s) {
    constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedSlope;
    p.tiles_m = (int)((p.m + T::BM - 1) / T::BM);
    p.tiles_n = kGated ? (p.half + T::BN / 2 - 1) / (T::BN / 2) : (p.n + T::BN - 1) / T::BN;
    const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.splits;
    if (total <= 0) return hipSuccess;
    if (total > 0x7fffffff) return hipErrorInvalidValue;
    if (p.vec_a && p.vec_b) return launch_aligned<DT, E4M3, LA, LB, EPI, T, true>(p, (unsigned)total, s);
    return launch_aligned<DT, E4M3, LA, LB, EPI, T, false>(p, (unsigned)total, s);
}

typedef Tile<256, 256, 2, 4, 2, 1> TileLarge;
typedef Tile<128, 128, 2, 2, 2, 2> TileMid;
typedef Tile<32, 64, 2, 1, 2, 4> TileSmall;

}  // namespace
}  // namespace smc
