// Window attention, forward: out_i = sum over the window's keys j of P_ij v_j, P the softmax of
// s_ij = scale q_i k_j + bias_ij, and lse_i = log sum_j exp(s_ij).
//
// A block takes a tile of 64 NQ queries of one window and one head, a wave 16 NQ of
// them; it walks the window's keys 64 at a time, keys and values through LDS with the next
// 64 on their way in registers, and keeps the running maximum and sum of the softmax.
// P is at most 1 and is rounded to the rows' type for its product with v (half an
// ulp of each term, beside half an ulp of the sum); the sum of P is taken before
// the rounding.
#pragma once

#include "attention.h"

namespace smc {
namespace {

template <int DT, int DP, int EXT, int NQ>
__global__ __launch_bounds__(kAttentionThreads) void k_attention(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT / 8, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    __shared__ __align__(16) char s_k[kKeys * DP * 2], s_v[kKeys * DP * 2], s_e[EXT ? kKeys * EXT * 2 : 16];
    __shared__ WindowPlace s_places[2][kKeys];
    __shared__ uint16_t s_table[EXT ? 3 * kDistances : 1];
    int tile, head;
    if (!tile_and_head(a.n_tiles, a.heads, tile, head)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int kv = head / (a.heads / a.kv_heads);
    if (threadIdx.x < kKeys) s_places[0][threadIdx.x] = place_at(a, t.begin + threadIdx.x, t.end);
    if (EXT) load_table<DT>(a, head, s_table);
    WindowPlace own[NQ];
#pragma unroll
    for (int u = 0; u < NQ; ++u) own[u] = own_place(a, t, (wave * NQ + u) * 16 + col);
    u32x4 fq[NQ][CK], fb[NQ][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u)
#pragma unroll
        for (int c = 0; c < CK; ++c)
            fq[u][c] = row_word(a.q, (int64_t)own[u].row * a.ldq + head * a.dim + 32 * c + 8 * q,
                                own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q, a.vec);
    __syncthreads();
    if (EXT)
#pragma unroll
        for (int u = 0; u < NQ; ++u)
#pragma unroll
            for (int c = 0; c < CE; ++c) fb[u][c] = table_word<1>(a, s_table, own[u].cells, 32 * c + 8 * q);
    RowLoads<RW> lk, lv;
    lk.load(a.k, a.ldk, kv * a.dim, a.dim, s_places[0], a.vec);
    lv.load(a.v, a.ldv, kv * a.dim, a.dim, s_places[0], a.vec);
    WindowPlace next = WindowPlace{-1, 0u};
    if (threadIdx.x < kKeys) next = place_at(a, t.begin + kKeys + threadIdx.x, t.end);

    // exponents in base 2: of the products times their scale, or of the scaled sums
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const bool active = wave * NQ * 16 < t.count;
    float top[NQ], sum[NQ];
    f32x4 o[NQ][DT16];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        top[u] = -INFINITY;
        sum[u] = 0.f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    int buf = 0;
    for (int k0 = t.begin; k0 < t.end; k0 += kKeys, buf ^= 1) {
        __syncthreads();
        lk.commit(s_k);
        lv.commit(s_v);
        if (EXT) commit_cells<DT, RE ? RE : 4>(s_e, s_places[buf]);
        if (threadIdx.x < kKeys) s_places[buf ^ 1][threadIdx.x] = next;
        __syncthreads();
        if (k0 + kKeys < t.end) {
            lk.load(a.k, a.ldk, kv * a.dim, a.dim, s_places[buf ^ 1], a.vec);
            lv.load(a.v, a.ldv, kv * a.dim, a.dim, s_places[buf ^ 1], a.vec);
            if (threadIdx.x < kKeys) next = place_at(a, k0 + 2 * kKeys + threadIdx.x, t.end);
        }
        if (!active) continue;
        f32x4 s[4][NQ];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
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
                    const u32x4 fe = tile_row<RE ? RE : 4>(s_e, 16 * b + col, 4 * c + q);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[b][u] = mfma16<DT>(fe, fb[u][c], s[b][u]);
                }
            }
        }
        if (k0 + kKeys > t.end) {           // keys past the window's end
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k0 + 16 * b + 4 * q + e >= t.end)
#pragma unroll
                        for (int u = 0; u < NQ; ++u) s[b][u][e] = -INFINITY;
        }
        u32x4 p[NQ][2];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            float m = top[u];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = fmaxf(m, s[b][u][e]);
            m = quad_max(m);
            const float base = m == -INFINITY ? 0.f : m * to_log2;      // (every score -inf so far)
            const float shrink = exp2_of(top[u] * to_log2 - base);
            top[u] = m;
            float add = 0.f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[b][u][e] = exp2_of(s[b][u][e] * to_log2 - base);
                    add += s[b][u][e];
                }
                p[u][b >> 1][2 * (b & 1)] = pack2<DT>(s[b][u][0], s[b][u][1]);
                p[u][b >> 1][2 * (b & 1) + 1] = pack2<DT>(s[b][u][2], s[b][u][3]);
            }
            sum[u] = sum[u] * shrink + add;
#pragma unroll
            for (int d = 0; d < DT16; ++d) o[u][d] *= shrink;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const u32x4 fv = tile_columns<RW>(s_v, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
#pragma unroll
                for (int u = 0; u < NQ; ++u) o[u][d] = mfma16<DT>(fv, p[u][h], o[u][d]);
            }
    }
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        const float total = quad_sum(sum[u]);
        // no key, or every score -inf: zeros
        store_row<DT, DP>(o[u], total == 0.f ? 0.f : 1.f / total, a.out,
                          own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ldo + head * a.dim, a.dim, lane, a.vec);
        if (a.lse && q == 0 && own[u].row >= 0)
            a.lse[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] =
                total == 0.f ? -INFINITY : top[u] * (EXT ? 1.f : a.scale) + logf(total);
    }
}

template <int DT, int DP, int EXT>
hipError_t attention_t(const AttentionArgs& a, bool wide, hipStream_t s) {
    const dim3 grid = attention_grid(a.n_tiles, a.heads);
    if (wide)
        launch(k_attention<DT, DP, EXT, 2>, grid, dim3(kAttentionThreads), 0, s, a);
    else
        launch(k_attention<DT, DP, EXT, 1>, grid, dim3(kAttentionThreads), 0, s, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t attention_by_cells(const AttentionArgs& a, bool wide, hipStream_t s) {
    const int cells = a.table ? a.extent[0] + a.extent[1] + a.extent[2] : 0;
    if (cells == 0) return attention_t<DT, DP, 0>(a, wide, s);
    if (cells <= 32) return attention_t<DT, DP, 32>(a, wide, s);
    if (cells <= 64) return attention_t<DT, DP, 64>(a, wide, s);
    return attention_t<DT, DP, 128>(a, wide, s);
}

template <int DT>
hipError_t attention_of_type(const AttentionArgs& a, bool wide, hipStream_t s) {
    if (a.dim <= 32) return attention_by_cells<DT, 32>(a, wide, s);
    if (a.dim <= 64) return attention_by_cells<DT, 64>(a, wide, s);
    return attention_by_cells<DT, 128>(a, wide, s);
}

}  // namespace
}  // namespace smc
