// Window attention, forward: out_i = sum over the window's keys j of P_ij v_j, P the softmax of
// s_ij = scale q_i k_j + bias_ij, and lse_i = log sum_j exp(s_ij).
//
// A block takes a tile of one window's queries and one head; it walks the window's keys 64
// at a time, keys and values through LDS with the next 64 on their way in registers, and
// keeps the running maximum and sum of the softmax.
// P is at most 1 and is rounded to the rows' type for its product with v (half an
// ulp of each term, beside half an ulp of the sum); the sum of P is taken before
// the rounding.
#pragma once

#include "attention.h"

namespace smc {
namespace {

template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads) void k_attention(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    constexpr int NQ = B::kColumns, TH = B::kThreads;
    // two buffers cost registers (addresses): us for windows of 1,000, 16,000 x 8 heads of 64 without and 40,000 x 4 of 32
    // with cells, one and two: long 73.4, 67.9 and 78.6, 85.2; mid 86.5, 76.6 and 90.1, 82.1
    constexpr int kBuffers = B::kWaves > 2 && (NQ == 1 || EXT == 0) ? 2 : 1;
    typedef Walk<DT, DP, EXT, A, B, kBuffers> Keys;
    __shared__ __align__(16) typename Keys::Memory s_keys;
    __shared__ __align__(16) uint16_t s_table[EXT ? 2 * kTableEntries<EXT> : 2];
    int tile, head;
    if (!tile_and_head(a.n_tiles, a.heads, tile, head)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int kv = head / (a.heads / a.kv_heads);
    if (EXT) load_table<DT, EXT, TH, false>(a, head, s_table);
    // exponents in base 2: of the products times their scale, or of the scaled sums
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const bool active = wave * NQ * 16 < t.count;
    WindowPlace own[NQ];
    u32x4 fq[NQ][CK], fb[NQ][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        own[u] = own_place(a, t, (wave * NQ + u) * 16 + col);
#pragma unroll
        for (int c = 0; c < CK; ++c)
            fq[u][c] = row_word<A>(a.q, (int64_t)own[u].row * a.ldq + head * a.dim + 32 * c + 8 * q,
                                own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q);
    }
    Keys keys;
    keys.start(a, s_keys, t, a.k, a.ldk, a.v, a.ldv, kv * a.dim);
    if (EXT)
#pragma unroll
        for (int u = 0; u < NQ; ++u)
            table_words<EXT>(a, s_table, own[u].cells, q, fb[u]);
    float top[NQ], sum[NQ];
    f32x4 o[NQ][DT16];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        top[u] = -INFINITY;
        sum[u] = 0.f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    // 64 keys, or the window's last `left`
    auto step = [&](int left, const char* s_k, const char* s_v, const char* s_e) SMC_INLINE {
        f32x4 s[4][NQ];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int u = 0; u < NQ; ++u) s[b][u] = (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (B::kSkips && 16 * b >= left) continue;
#pragma unroll
            for (int u = 0; u < NQ; ++u) s[b][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                const u32x4 fk = tile_row<RW>(s_k, 16 * b + col, 4 * c + q);
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[b][u] = mfma16<DT>(fk, fq[u][c], s[b][u]);
            }
            if (EXT) {
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[b][u] *= a.scale;
#pragma unroll
                for (int c = 0; c < CE; ++c) {
                    const u32x4 fe = tile_row<RE>(s_e, 16 * b + col, 4 * c + q);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[b][u] = mfma16<DT>(fe, fb[u][c], s[b][u]);
                }
            }
        }
        if (left < kKeys)                           // keys past the window's end
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[b][u][e] = 16 * b + 4 * q + e < left ? s[b][u][e] : -INFINITY;
        u32x4 p[NQ][2];
        float most[NQ], base[NQ];
        bool grows = false;
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            float m = top[u];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = fmaxf(m, s[b][u][e]);
            most[u] = quad_max(m);
            base[u] = most[u] == -INFINITY ? 0.f : most[u] * to_log2;       // (every score -inf so far)
            grows |= most[u] > top[u];
        }
        if (any_lane(grows))
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                const float shrink = exp2_of(top[u] * to_log2 - base[u]);
                sum[u] *= shrink;
#pragma unroll
                for (int d = 0; d < DT16; ++d) o[u][d] *= shrink;
                top[u] = most[u];
            }
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                p[u][b >> 1][2 * (b & 1)] = p[u][b >> 1][2 * (b & 1) + 1] = 0u;
                if (B::kSkips && 16 * b >= left) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[b][u][e] = exp2_of(s[b][u][e] * to_log2 - base[u]);
                    sum[u] += s[b][u][e];
                }
                p[u][b >> 1][2 * (b & 1)] = pack2<DT>(s[b][u][0], s[b][u][1]);
                p[u][b >> 1][2 * (b & 1) + 1] = pack2<DT>(s[b][u][2], s[b][u][3]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (B::kSkips && 32 * h >= left) continue;
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const u32x4 fv = tile_columns<RW>(s_v, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
#pragma unroll
                for (int u = 0; u < NQ; ++u) o[u][d] = mfma16<DT>(fv, p[u][h], o[u][d]);
            }
        }
    };
    const int length = t.end - t.begin;
    if (length > 0) keys.commit(a, s_keys, 0, t);
    for (int i = 0; i * kKeys < length; ++i) {
        const int left = length - i * kKeys, buf = kBuffers == 2 ? i & 1 : 0;
        if (left > kKeys) keys.load(a, s_keys, i + 1, a.k, a.ldk, a.v, a.ldv, kv * a.dim);
        if (active) step(left, s_keys.x[buf], s_keys.y[buf], s_keys.e[buf]);
        if (left > kKeys) keys.commit(a, s_keys, i + 1, t);
    }
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        const float total = quad_sum(sum[u]);
        // no key, or every score -inf: zeros
        store_row<DT, DP, A>(o[u], total == 0.f ? 0.f : 1.f / total, a.out,
                          own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ldo + head * a.dim, a.dim, lane);
        if (a.lse && q == 0 && own[u].row >= 0)
            a.lse[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] =
                total == 0.f ? -INFINITY : top[u] * (EXT ? 1.f : a.scale) + logf(total);
    }
}

// Rows that are no whole 16-byte words take one kernel a width: their loads cost more than a better
// fitting block or contraction would save.
template <int DT, int DP>
hipError_t attention_by_cells(const AttentionArgs& a, int lengths, hipStream_t s) {
    const int cells = a.table ? Cells(a.extent).all() : 0;
    const dim3 grid = attention_grid(a.n_tiles, a.heads);
#define SMC_GO(EXT, A, B) launch(k_attention<DT, DP, EXT, A, B>, grid, dim3(B::kThreads), 0, s, a)
#define SMC_CELLS(EXT)                                                         \
    do {                                                                       \
        if (lengths == kShortWindows) SMC_GO(EXT, true, BlockShort<DP>);       \
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
