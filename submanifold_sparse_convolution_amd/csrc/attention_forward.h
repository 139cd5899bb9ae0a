// Window attention, forward: out_i = sum over the window's keys j of P_ij v_j, P the softmax of
// s_ij = scale q_i k_j + bias_ij, and lse_i = log sum_j exp(s_ij).
//
// A block takes a tile of one window's queries and a head, or two after each other; it walks
// the window's keys 64 at a time, keys and values through LDS with the next 64 on their way in
// registers, and keeps the running maximum and sum of the softmax.
// P, at most 2^8 (see `maxima`), is rounded to the rows' type for its product with v (half an
// ulp of each term, beside half an ulp of the sum); the sum of P is taken before
// the rounding. In f16 it is times 2^7, at most 2^15: keys of little weight, of which a long window may have
// enough to count, would be below its normal numbers (95,000 of 5 10^-6 beside one of 1 came out 0.55 % off).
//
// 15,000 x 512 in four windows of 3,750, 8 heads of 64: 182 us a call for a floor of 77 (products at
// 1.5 PFLOP/s), vector units 51 % busy, matrix units 26 %: a score's exponential, scale, sum and rounding
// stand beside 256 operations of products. 91,000 x 128 in 2,905 windows of 31 rows, 4 heads, cells: 48.0 us
// for 18.4 (bytes), where blocks wait for their first loads (places, then rows) half of the time.
#pragma once

#include "attention.h"

namespace smc {
namespace {

// (waves a SIMD by what the registers take; left at three, f16's long blocks of heads up to 32 with up to 32 cells take 132:
// 40,000 x 4 heads in windows of 100 19.1 us for 18.0)
template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads, DP <= 32 && EXT <= 32 ? 4 : DP + EXT <= 64 ? 3 : DP + EXT < 192 ? 2 : 1) void k_attention(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    constexpr int NQ = B::kColumns, TH = B::kThreads;
    // two buffers cost registers (addresses): us for windows of 1,000, 16,000 x 8 heads of 64 without and 40,000 x 4 of 32
    // with cells, one and two: long 73.4, 67.9 and 78.6, 85.2; mid 86.5, 76.6 and 90.1, 82.1
    constexpr int kBuffers = B::kWaves > 2 && (NQ == 1 || EXT == 0) ? 2 : 1;
    constexpr float kLift = DT == kF16 ? 7.f : 0.f, kSlack = DT == kF16 ? 7.f : 8.f;     // powers of two (see `maxima`)
    typedef Walk<DT, DP, EXT, A, B, kBuffers> Keys;
    __shared__ __align__(16) typename Keys::Memory s_keys;
    __shared__ __align__(16) uint16_t s_table[B::kHeads][EXT ? 2 * kTableEntries<EXT> : 2];
    int tile, head;
    if (!tile_and_head(a.n_tiles, a.heads, a.heads_each, tile, head)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int share = a.heads / a.kv_heads, first_head = head, heads = min(a.heads_each, a.heads - head);
    const int length = t.end - t.begin;
    const bool active = wave * NQ * 16 < t.count, one = length <= kKeys;    // one step a head
    // exponents in base 2: of the products times their scale, or of the scaled sums
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const TileLane<RW> at(lane);
    const TileLane<RE> at_cells(lane);
    WindowPlace own[NQ];
#pragma unroll
    for (int u = 0; u < NQ; ++u) own[u] = own_place(a, t, (wave * NQ + u) * 16 + col);
    Keys keys;
    keys.places(a, t, 0);
    if (EXT) load_tables<DT, EXT, TH, B::kHeads>(a, head, heads, s_table);
    u32x4 fq[NQ][CK], fb[NQ][CE ? CE : 1];
    auto load_queries = [&](int h, u32x4 (&f)[NQ][CK]) SMC_INLINE {
#pragma unroll
        for (int u = 0; u < NQ; ++u)
#pragma unroll
            for (int c = 0; c < CK; ++c)
                f[u][c] = row_word<A>(a.q, (int64_t)own[u].row * a.ldq + h * a.dim + 32 * c + 8 * q,
                                      own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q);
    };
    load_queries(head, fq);
    keys.point(a.k, a.v, head / share * a.dim);
    keys.load(a, a.ldk, a.ldv);
    if (!one) keys.places(a, t, 1);
    float top[NQ], base[NQ], sum[NQ];
    f32x4 o[NQ][DT16];
    auto begin_head = [&]() SMC_INLINE {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            top[u] = -INFINITY;
            base[u] = sum[u] = 0.f;
#pragma unroll
            for (int d = 0; d < DT16; ++d) o[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if (EXT) table_words<EXT>(a, s_table[head - first_head], own[u].cells, q, fb[u]);
        }
    };
    // The scores of a step's 16 KB keys from 16 b0 on
    constexpr int KB = B::kHalves ? 2 : 4;
    auto scores = [&](f32x4 (&s)[KB][NQ], int b0, const char* s_k, const char* s_e) SMC_INLINE {
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int u = 0; u < NQ; ++u) s[b][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                const u32x4 fk = at.along(s_k, 16 * (b0 + b), c);
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[b][u] = mfma16<DT>(fk, fq[u][c], s[b][u]);
            }
            if (EXT) {
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[b][u] *= a.scale;
#pragma unroll
                for (int c = 0; c < CE; ++c) {
                    const u32x4 fe = at_cells.along(s_e, 16 * (b0 + b), c);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[b][u] = mfma16<DT>(fe, fb[u][c], s[b][u]);
                }
            }
        }
    };
    auto cut = [&](f32x4 (&s)[KB][NQ], int left) SMC_INLINE {      // keys past the window's end
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[b][u][e] = 16 * b + 4 * q + e < left ? s[b][u][e] : -INFINITY;
    };
    // The base of the exponentials follows the maximum only where that is 2^kSlack above it: P then stays below 2^8
    // (f16: 2^15, as a base beyond 2^24 may be rounded 8 down where it was meant to be kLift), as exact as below 1, and
    // out and the sums are seldom rescaled.
    auto maxima = [&](const f32x4 (&s)[KB][NQ]) SMC_INLINE {
        float most[NQ];
        bool grows = false;
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            float m = s[0][u][0];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = fmaxf(m, s[b][u][e]);
            most[u] = quad_max(m);
            grows |= (most[u] - top[u]) * to_log2 > kSlack;    // (of two -inf: no)
        }
        if (any_lane(grows))
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                const float m = fmaxf(top[u], most[u]), next = (m == -INFINITY ? 0.f : m * to_log2) - kLift;   // (every score -inf so far)
                const float shrink = top[u] == -INFINITY ? 0.f : exp2_of(base[u] - next);
                sum[u] *= shrink;
#pragma unroll
                for (int d = 0; d < DT16; ++d) o[u][d] *= shrink;
                top[u] = m;
                base[u] = next;
            }
    };
    auto products = [&](f32x4 (&s)[KB][NQ], int b0, const char* s_v) SMC_INLINE {
        u32x4 p[NQ][KB / 2];
        float part[NQ];         // of the step: little weights after a large one are not added to it one by one
        // values before the exponentials, which cover their latency (else read two at a time, when they are needed)
        constexpr bool kEarly = DP <= 64 && EXT == 0;
        u32x4 fv[kEarly ? KB / 2 : 1][DT16];
        if (kEarly) {
#pragma unroll
            for (int h = 0; h < KB / 2; ++h)
#pragma unroll
                for (int d = 0; d < DT16; ++d) fv[kEarly ? h : 0][d] = at.across(s_v, d, 16 * b0 + 32 * h);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[b][u][e] = exp2_of(s[b][u][e] * to_log2 - base[u]);
                    part[u] = b + e == 0 ? s[b][u][e] : part[u] + s[b][u][e];
                }
                p[u][b >> 1][2 * (b & 1)] = pack2<DT>(s[b][u][0], s[b][u][1]);
                p[u][b >> 1][2 * (b & 1) + 1] = pack2<DT>(s[b][u][2], s[b][u][3]);
            }
#pragma unroll
        for (int u = 0; u < NQ; ++u) sum[u] += part[u];
#pragma unroll
        for (int h = 0; h < KB / 2; ++h)
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                if (!kEarly) fv[0][d] = at.across(s_v, d, 16 * b0 + 32 * h);
#pragma unroll
                for (int u = 0; u < NQ; ++u) o[u][d] = mfma16<DT>(fv[kEarly ? h : 0][d], p[u][h], o[u][d]);
            }
    };
    auto step = [&](int b0, int left, const char* s_k, const char* s_v, const char* s_e) SMC_INLINE {
        f32x4 s[KB][NQ];
        scores(s, b0, s_k, s_e);
        if (left < 16 * KB) cut(s, left);
        maxima(s);
        products(s, b0, s_v);
    };
    auto end_head = [&]() SMC_INLINE {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const float total = quad_sum(sum[u]);
            // no key, or every score -inf: zeros
            store_row<DT, DP, A>(o[u], total == 0.f ? 0.f : 1.f / total, a.out,
                                 own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ldo + head * a.dim, a.dim, lane);
            if (a.lse && q == 0 && own[u].row >= 0)
                a.lse[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] =
                    total == 0.f ? -INFINITY : top[u] * (EXT ? 1.f : a.scale) + logf(total * exp2f(-kLift));
        }
    };
    int i = 0, buf = 0;                 // the step of the head, and its buffer
    keys.commit(s_keys, buf, true);
    begin_head();
    for (;;) {
        const int left = length - i * kKeys;
        const bool last = left <= kKeys, more = !last || head + 1 < first_head + heads;
        u32x4 fq_next[B::kHeads > 1 ? NQ : 1][CK];
        if (more) {
            if constexpr (B::kHeads > 1)
                if (last) {
                    keys.point(a.k, a.v, (head + 1) / share * a.dim);
                    load_queries(head + 1, fq_next);
                }
            keys.load(a, a.ldk, a.ldv);
            if (!one) keys.places(a, t, (last ? 1 : i + 2) * kKeys < length ? (last ? 1 : i + 2) : 0);
        }
        // (the cells of a window of one step lie in the first buffer)
        if (active)
#pragma unroll
            for (int b0 = 0; b0 < 4; b0 += KB)
                if (b0 == 0 || 16 * b0 < left) step(b0, left - 16 * b0, s_keys.x[buf], s_keys.y[buf], s_keys.e[one ? 0 : buf]);
        if (last) end_head();
        if (!more) break;
        if (kBuffers == 2) buf ^= 1;
        keys.commit(s_keys, buf, !one);
        ++i;
        if constexpr (B::kHeads > 1)
            if (last) {
                i = 0;
                ++head;
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int c = 0; c < CK; ++c) fq[u][c] = fq_next[u][c];
                begin_head();
            }
    }
}

template <int DT, int DP, int EXT, bool A, class B>
void attention_t(AttentionArgs a, hipStream_t s) {
    a.heads_each = heads_a_block(a.n_tiles, a.heads, B::kHeads);
    launch(k_attention<DT, DP, EXT, A, B>, attention_grid(a.n_tiles, a.heads, a.heads_each), dim3(B::kThreads), 0, s, a);
}

// Rows that are no whole 16-byte words take one kernel a width, which keeps the library small and costs most where
// there is a bias (128 cells): 91,000 x 4 heads of 32 in windows of 31, forward / backward in us, 53 / 260 for 24 / 87
// aligned, without a bias 25.7 / 76.6 for 23.8 / 65.8.
template <int DT, int DP>
hipError_t attention_by_cells(const AttentionArgs& a, int lengths, hipStream_t s) {
    const int cells = a.table ? Cells(a.extent).all() : 0;
#define SMC_GO(EXT, A, B) attention_t<DT, DP, EXT, A, B>(a, s)
#define SMC_CELLS(EXT)                                                         \
    do {                                                                       \
        if (lengths == kShortWindows) SMC_GO(EXT, true, BlockShort);       \
        else if (lengths == kMidWindows) SMC_GO(EXT, true, BlockMid);          \
        else SMC_GO(EXT, true, BlockLong);                                     \
    } while (0)
    if (!a.vec) {
        if (cells == 0) SMC_GO(0, false, BlockMid);
        else SMC_GO(128, false, BlockMid);
    } else if (cells == 0) SMC_CELLS(0);
    else if (cells <= 32) SMC_CELLS(32);
    else if (cells <= 64) SMC_CELLS(64);
    else SMC_CELLS(128);
#undef SMC_CELLS
#undef SMC_GO
    return hipGetLastError();
}

template <int DT>
hipError_t attention_of_type(const AttentionArgs& a, int lengths, hipStream_t s) {
    if (a.dim <= 32) return attention_by_cells<DT, 32>(a, lengths, s);
    if (a.dim <= 64) return attention_by_cells<DT, 64>(a, lengths, s);
    return attention_by_cells<DT, 128>(a, lengths, s);
}

}  // namespace
}  // namespace smc
