// Gradients of window attention. P is computed again from q, k, the bias and lse;
// with delta_i = dout_i . out_i (the mean of dP_i under P_i) and dP = dout v^T,
//   dS = P (dP - delta),  dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout,
//   dbias[axis][b] = sum of dS over the pairs whose distance is in bucket b.
//
// Two kernels, each without atomics. By queries: a block takes 64 NQ queries of a window and
// a head and walks the keys, for delta, dq and the table's gradient; by keys: a block takes 64
// NK keys and a head of k and v and walks the queries of that head's group, for dk and dv. Both
// compute S and dP: 7 products a pair where 5 would do, but dq needs no sum over blocks.
// dB = dS E comes out as sums over the cells of a key for each query; a block adds
// them up by distance and writes its buckets, k_table_sum adds the blocks.
//
// P and dS are rounded to the rows' type as operands (half an ulp of each term). dS follows
// the gradient's size, which in f16 may leave the type's range where dq and dk do not,
// so in f16 it is taken times a power of two: |dP - delta| <= 2 dim max |dout| max |v| over
// the window (finite values), brought to [2^14, 2^15]; k_attention_range finds the maxima.
#pragma once

#include "attention.h"

namespace smc {
namespace {

// Largest finite |x| of a word's 8 elements, by its float32 bits.
template <int DT>
__device__ __forceinline__ uint32_t word_most(u32x4 w, uint32_t most) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t m = __float_as_uint(to_f32<DT>((w[e >> 1] >> (16 * (e & 1))) & 0x7fffu));
        most = max(most, m < 0x7f800000u ? m : 0u);
    }
    return most;
}

// f16: largest |dout| of each head and |v| of each of its heads in a tile of 64 places; a wave a head.
template <int DT>
__global__ __launch_bounds__(kAttentionThreads) void k_attention_range(AttentionArgs a) {
    const WindowTile t = a.tiles64[block_number() < a.n_tiles64 ? block_number() : 0];
    if (block_number() >= a.n_tiles64) return;
    const int lane = threadIdx.x & 63, all = a.heads + a.kv_heads;
    const int row = lane < t.count ? a.places[t.first + lane].row : -1;
    for (int h = threadIdx.x >> 6; h < all; h += kAttentionThreads / 64) {
        const bool of_v = h >= a.heads;
        const void* base = of_v ? a.v : a.dout;
        const int64_t at = (int64_t)row * (of_v ? a.ldv : a.ld_dout) + (of_v ? h - a.heads : h) * a.dim;
        uint32_t most = 0;
        if (row >= 0)
            for (int c = 0; c < a.dim; c += W) most = word_most<DT>(row_word(base, at + c, a.dim - c, a.vec), most);
        most = lane_max<64>(most);
        if (lane == 0) reinterpret_cast<uint32_t*>(a.range)[block_number() * all + h] = most;
    }
}

// The power of two that dS is taken times, for the head of k and v that `kv` heads `head` .. share
// (head_count of them), over the window of tile t.
__device__ __forceinline__ float gradient_scale(const AttentionArgs& a, const WindowTile& t, int head, int kv) {
    __shared__ uint32_t s_most[2][kAttentionThreads / 64];
    // the window's tiles of 64 lie behind each other; find its first by its place
    int lo = 0, hi = a.n_tiles64 - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.tiles64[mid].first < t.begin) lo = mid + 1;
        else hi = mid;
    }
    const int count = (t.end - t.begin + 63) / 64, all = a.heads + a.kv_heads;
    uint32_t most[2] = {0u, 0u};
    for (int i = threadIdx.x; i < count; i += kAttentionThreads) {
        const uint32_t* r = reinterpret_cast<const uint32_t*>(a.range) + (int64_t)(lo + i) * all;
        most[0] = max(most[0], r[head]);
        most[1] = max(most[1], r[a.heads + kv]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        most[k] = lane_max<64>(most[k]);
        if ((threadIdx.x & 63) == 0) s_most[k][threadIdx.x >> 6] = most[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) most[k] = max(max(s_most[k][0], s_most[k][1]), max(s_most[k][2], s_most[k][3]));
    const float bound = 2.f * (float)a.dim * __uint_as_float(most[0]) * __uint_as_float(most[1]);
    if (!(bound > 0.f)) return 1.f;
    // bound is within 2^-46 and 2^40
    return __uint_as_float((uint32_t)(127 + 14 - ((int)(__float_as_uint(bound) >> 23) - 127)) << 23);
}

// lse as an exponent's base: where there is no key P is 0.
__device__ __forceinline__ float lse_base(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

template <int DT, int DP, int EXT, int NQ>
__global__ __launch_bounds__(kAttentionThreads) void k_attention_queries(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16, ET16 = EXT / 16;
    constexpr int kTileBytes = kKeys * (2 * DP + EXT) * 2;
    // the sums by cell of the block's queries, where the tiles were (rows 4 floats longer than their cells)
    constexpr int kSumBytes = EXT ? 64 * (EXT + 4) * 4 + 3 * kDistances * 4 : 0;
    __shared__ __align__(16) char s_mem[kTileBytes > kSumBytes ? kTileBytes : kSumBytes];
    char* const s_k = s_mem;
    char* const s_v = s_mem + kKeys * DP * 2;
    char* const s_e = s_mem + 2 * kKeys * DP * 2;
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
    float base[NQ], delta[NQ];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        const int i = (wave * NQ + u) * 16 + col;
        own[u] = own_place(a, t, i);
        base[u] = own[u].row < 0 ? INFINITY : lse_base(a.lse[(int64_t)head * a.n + t.first + i]);
    }
    u32x4 fq[NQ][CK], fo[NQ][CK], fb[NQ][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        f32x4 diagonal = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CK; ++c) {
            const int at = head * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
            fq[u][c] = row_word(a.q, (int64_t)own[u].row * a.ldq + at, left, a.vec);
            fo[u][c] = row_word(a.dout, (int64_t)own[u].row * a.ld_dout + at, left, a.vec);
            const u32x4 out = row_word(a.out, (int64_t)own[u].row * a.ldo + at, left, a.vec);
            // by the instruction that makes dP: a window of one row, where out is v, has dP = delta to the bit
            diagonal = mfma16<DT>(out, fo[u][c], diagonal);
        }
        // row 4 q + e, column col: the diagonal lies in the lanes with q = col / 4
        const float mine = (col & 3) == 0 ? diagonal[0] : (col & 3) == 1 ? diagonal[1] : (col & 3) == 2 ? diagonal[2] : diagonal[3];
        delta[u] = quad_sum(q == (col >> 2) ? mine : 0.f);
        if (q == 0 && own[u].row >= 0) a.delta[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] = delta[u];
    }
    const float grow = DT == kF16 ? gradient_scale(a, t, head, kv) : 1.f;
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

    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const bool active = wave * NQ * 16 < t.count;
    f32x4 dq[NQ][DT16], db[NQ][ET16 ? ET16 : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
#pragma unroll
        for (int d = 0; d < DT16; ++d) dq[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < ET16; ++d) db[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    int buf = 0;
    for (int k0 = t.begin; k0 < t.end; k0 += kKeys, buf ^= 1) {
        __syncthreads();
        lk.commit(s_k);
        lv.commit(s_v);
        if (EXT) commit_cells<DT, RE>(s_e, s_places[buf]);
        if (threadIdx.x < kKeys) s_places[buf ^ 1][threadIdx.x] = next;
        __syncthreads();
        if (k0 + kKeys < t.end) {
            lk.load(a.k, a.ldk, kv * a.dim, a.dim, s_places[buf ^ 1], a.vec);
            lv.load(a.v, a.ldv, kv * a.dim, a.dim, s_places[buf ^ 1], a.vec);
            if (threadIdx.x < kKeys) next = place_at(a, k0 + 2 * kKeys + threadIdx.x, t.end);
        }
        if (!active) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {           // 32 keys at a time
            u32x4 g[NQ];
#pragma unroll
            for (int b = 2 * h; b < 2 * h + 2; ++b) {
                f32x4 s[NQ], dp[NQ];
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[u] = dp[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < CK; ++c) {
                    const u32x4 fk = tile_row<RW>(s_k, 16 * b + col, 4 * c + q);
                    const u32x4 fv = tile_row<RW>(s_v, 16 * b + col, 4 * c + q);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) {
                        s[u] = mfma16<DT>(fk, fq[u][c], s[u]);
                        dp[u] = mfma16<DT>(fv, fo[u][c], dp[u]);
                    }
                }
                if (EXT) {
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[u] *= a.scale;
#pragma unroll
                    for (int c = 0; c < CE; ++c) {
                        const u32x4 fe = tile_row<RE>(s_e, 16 * b + col, 4 * c + q);
#pragma unroll
                        for (int u = 0; u < NQ; ++u) s[u] = mfma16<DT>(fe, fb[u][c], s[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < NQ; ++u) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = exp2_of(s[u][e] * to_log2 - base[u]);
                        v[e] = p * (dp[u][e] - delta[u]);
                        if (DT == kF16) v[e] *= grow;
                        // (keys past the end: their exponential may be infinite)
                        if (k0 + 16 * b + 4 * q + e >= t.end) v[e] = 0.f;
                    }
                    g[u][2 * (b & 1)] = pack2<DT>(v[0], v[1]);
                    g[u][2 * (b & 1) + 1] = pack2<DT>(v[2], v[3]);
                }
            }
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const u32x4 f = tile_columns<RW>(s_k, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
#pragma unroll
                for (int u = 0; u < NQ; ++u) dq[u][d] = mfma16<DT>(f, g[u], dq[u][d]);
            }
            if (EXT)
#pragma unroll
                for (int d = 0; d < ET16; ++d) {
                    const u32x4 f = tile_columns<RE>(s_e, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) db[u][d] = mfma16<DT>(f, g[u], db[u][d]);
                }
        }
    }
    const float shrink = 1.f / grow;            // (a power of two)
#pragma unroll
    for (int u = 0; u < NQ; ++u)
        store_row<DT, DP>(dq[u], a.scale * shrink, a.dq, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dq + head * a.dim,
                          a.dim, lane, a.vec);
    if constexpr (EXT > 0) {
        // The table's gradient. 64 queries at a time: their sums by cell to LDS, then a thread a
        // distance adds those at that distance, query after query.
        float* const s_db = reinterpret_cast<float*>(s_mem);
        float* const s_by = s_db + 64 * (EXT + 4);      // [axis][128 + distance]
        __shared__ uint32_t s_cells[64];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            __syncthreads();
            // wave w's queries lie at 16 w + col: their order does not matter
            if (q == 0) s_cells[wave * 16 + col] = own[u].row < 0 ? 0xffffffffu : own[u].cells;
#pragma unroll
            for (int d = 0; d < ET16; ++d)
                *reinterpret_cast<f32x4*>(s_db + (wave * 16 + col) * (EXT + 4) + 16 * d + 4 * q) = db[u][d];
            __syncthreads();
            for (int i = threadIdx.x; i < 3 * kDistances; i += kAttentionThreads) {
                const int axis = i / kDistances, away = i % kDistances - 128, extent = a.extent[axis];
                if (away <= -extent || away >= extent) continue;
                const int first = axis == 0 ? 0 : axis == 1 ? a.extent[0] : a.extent[0] + a.extent[1];
                float v = u == 0 ? 0.f : s_by[i];
                for (int r = 0; r < 64; ++r) {
                    const uint32_t cells = s_cells[r];
                    const int c = (int)((cells >> (8 * axis)) & 255u) - away;       // the key's cell
                    if (cells != 0xffffffffu && c >= first && c < first + extent) v += s_db[r * (EXT + 4) + c];
                }
                s_by[i] = v;
            }
        }
        __syncthreads();
        const int buckets = 2 * a.reach + 1;
        float* const part = a.part + ((int64_t)tile * a.heads + head) * 3 * buckets;
        for (int i = threadIdx.x; i < 3 * buckets; i += kAttentionThreads) {
            const int axis = i / buckets, d = i % buckets - a.reach, extent = a.extent[axis];
            // the outermost buckets hold every distance beyond them
            const int from = d == -a.reach ? 1 - extent : max(d, 1 - extent), to = d == a.reach ? extent - 1 : min(d, extent - 1);
            float v = 0.f;
            for (int k = from; k <= to; ++k) v += s_by[axis * kDistances + 128 + k];
            part[i] = v * shrink;
        }
    }
}

template <int DT, int DP, int EXT, int NK>
__global__ __launch_bounds__(kAttentionThreads) void k_attention_keys(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    __shared__ __align__(16) char s_q[kKeys * DP * 2], s_o[kKeys * DP * 2], s_e[EXT ? kKeys * EXT * 2 : 16];
    __shared__ __align__(16) float s_base[kKeys], s_delta[kKeys];
    __shared__ WindowPlace s_places[2][kKeys];
    __shared__ uint16_t s_table[EXT ? 3 * kDistances : 1];
    int tile, kv;
    if (!tile_and_head(a.n_tiles, a.kv_heads, tile, kv)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int each = a.heads / a.kv_heads;
    WindowPlace own[NK];
#pragma unroll
    for (int u = 0; u < NK; ++u) own[u] = own_place(a, t, (wave * NK + u) * 16 + col);
    u32x4 fk[NK][CK], fv[NK][CK], fb[NK][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
        for (int c = 0; c < CK; ++c) {
            const int at = kv * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
            fk[u][c] = row_word(a.k, (int64_t)own[u].row * a.ldk + at, left, a.vec);
            fv[u][c] = row_word(a.v, (int64_t)own[u].row * a.ldv + at, left, a.vec);
        }
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const bool active = wave * NK * 16 < t.count;
    f32x4 dk[NK][DT16], dv[NK][DT16];
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
        for (int d = 0; d < DT16; ++d) dk[u][d] = dv[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float grow = 1.f;
    if (DT == kF16) {                           // the smallest factor of the group's heads serves all
        grow = gradient_scale(a, t, kv * each, kv);
        for (int i = 1; i < each; ++i) grow = fminf(grow, gradient_scale(a, t, kv * each + i, kv));
    }
    for (int head = kv * each; head < (kv + 1) * each; ++head) {
        __syncthreads();
        if (threadIdx.x < kKeys) s_places[0][threadIdx.x] = place_at(a, t.begin + threadIdx.x, t.end);
        if (EXT) load_table<DT>(a, head, s_table);
        __syncthreads();
        if (EXT)
#pragma unroll
            for (int u = 0; u < NK; ++u)
#pragma unroll
                for (int c = 0; c < CE; ++c) fb[u][c] = table_word<-1>(a, s_table, own[u].cells, 32 * c + 8 * q);
        RowLoads<RW> lq, lo;
        lq.load(a.q, a.ldq, head * a.dim, a.dim, s_places[0], a.vec);
        lo.load(a.dout, a.ld_dout, head * a.dim, a.dim, s_places[0], a.vec);
        const float* const lse = a.lse + (int64_t)head * a.n;
        const float* const deltas = a.delta + (int64_t)head * a.n;
        WindowPlace next = WindowPlace{-1, 0u};
        float base = INFINITY, delta = 0.f;     // of this thread's query, in the first 64 threads
        if (threadIdx.x < kKeys) {
            next = place_at(a, t.begin + kKeys + threadIdx.x, t.end);
            if (t.begin + (int)threadIdx.x < t.end) {
                base = lse_base(lse[t.begin + threadIdx.x]);
                delta = deltas[t.begin + threadIdx.x];
            }
        }
        int buf = 0;
        for (int q0 = t.begin; q0 < t.end; q0 += kKeys, buf ^= 1) {
            __syncthreads();
            lq.commit(s_q);
            lo.commit(s_o);
            if (EXT) commit_cells<DT, RE>(s_e, s_places[buf]);
            if (threadIdx.x < kKeys) {
                s_places[buf ^ 1][threadIdx.x] = next;
                s_base[threadIdx.x] = base;
                s_delta[threadIdx.x] = delta;
            }
            __syncthreads();
            if (q0 + kKeys < t.end) {
                lq.load(a.q, a.ldq, head * a.dim, a.dim, s_places[buf ^ 1], a.vec);
                lo.load(a.dout, a.ld_dout, head * a.dim, a.dim, s_places[buf ^ 1], a.vec);
                if (threadIdx.x < kKeys) {
                    const int at = q0 + kKeys + threadIdx.x;
                    next = place_at(a, at + kKeys, t.end);
                    base = at < t.end ? lse_base(lse[at]) : INFINITY;       // past the end: P is 0
                    delta = at < t.end ? deltas[at] : 0.f;
                }
            }
            if (!active) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 p[NK], g[NK];
#pragma unroll
                for (int b = 2 * h; b < 2 * h + 2; ++b) {
                    f32x4 s[NK], dp[NK];
#pragma unroll
                    for (int u = 0; u < NK; ++u) s[u] = dp[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < CK; ++c) {
                        const u32x4 fq = tile_row<RW>(s_q, 16 * b + col, 4 * c + q);
                        const u32x4 fo = tile_row<RW>(s_o, 16 * b + col, 4 * c + q);
#pragma unroll
                        for (int u = 0; u < NK; ++u) {
                            s[u] = mfma16<DT>(fq, fk[u][c], s[u]);
                            dp[u] = mfma16<DT>(fo, fv[u][c], dp[u]);
                        }
                    }
                    if (EXT) {
#pragma unroll
                        for (int u = 0; u < NK; ++u) s[u] *= a.scale;
#pragma unroll
                        for (int c = 0; c < CE; ++c) {
                            const u32x4 fe = tile_row<RE>(s_e, 16 * b + col, 4 * c + q);
#pragma unroll
                            for (int u = 0; u < NK; ++u) s[u] = mfma16<DT>(fe, fb[u][c], s[u]);
                        }
                    }
                    const f32x4 bs = *reinterpret_cast<const f32x4*>(s_base + 16 * b + 4 * q);
                    const f32x4 dl = *reinterpret_cast<const f32x4*>(s_delta + 16 * b + 4 * q);
#pragma unroll
                    for (int u = 0; u < NK; ++u) {
                        float v[4], w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = exp2_of(s[u][e] * to_log2 - bs[e]);
                            w[e] = v[e] * (dp[u][e] - dl[e]);
                            if (DT == kF16) w[e] *= grow;
                        }
                        p[u][2 * (b & 1)] = pack2<DT>(v[0], v[1]);
                        p[u][2 * (b & 1) + 1] = pack2<DT>(v[2], v[3]);
                        g[u][2 * (b & 1)] = pack2<DT>(w[0], w[1]);
                        g[u][2 * (b & 1) + 1] = pack2<DT>(w[2], w[3]);
                    }
                }
#pragma unroll
                for (int d = 0; d < DT16; ++d) {
                    const u32x4 fo = tile_columns<RW>(s_o, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
                    const u32x4 fq = tile_columns<RW>(s_q, d, 32 * h + 4 * q, 32 * h + 16 + 4 * q, lane);
#pragma unroll
                    for (int u = 0; u < NK; ++u) {
                        dv[u][d] = mfma16<DT>(fo, p[u], dv[u][d]);
                        dk[u][d] = mfma16<DT>(fq, g[u], dk[u][d]);
                    }
                }
            }
        }
    }
    const float f = a.scale / grow;
#pragma unroll
    for (int u = 0; u < NK; ++u) {
        const int at = kv * a.dim;
        store_row<DT, DP>(dk[u], f, a.dk, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dk + at, a.dim, lane, a.vec);
        store_row<DT, DP>(dv[u], 1.f, a.dv, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dv + at, a.dim, lane, a.vec);
    }
}

// dtable = the blocks' buckets: 16 buckets a block, 64 strided runs of tiles joined by a tree.
template <int DT>
__global__ __launch_bounds__(1024) void k_table_sum(AttentionArgs a) {
    __shared__ float s[64][17];
    const int buckets = 3 * (2 * a.reach + 1), x = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int i = blockIdx.x * 16 + x, head = blockIdx.y;
    float v = 0.f;
    if (i < buckets) {
#pragma unroll 8
        for (int k = run; k < a.n_tiles; k += 64) v += a.part[((int64_t)k * a.heads + head) * buckets + i];
    }
    s[run][x] = v;
    __syncthreads();
    for (int o = 32; o > 0; o >>= 1) {
        if (run < o) s[run][x] += s[run + o][x];
        __syncthreads();
    }
    if (run == 0 && i < buckets) static_cast<uint16_t*>(a.dtable)[(int64_t)i * a.heads + head] = (uint16_t)from_f32<DT>(s[0][x]);
}

template <int DT, int DP, int EXT, int NQ, int NK>
hipError_t attention_backward_t(const AttentionArgs& a, hipStream_t s) {
    if (a.n_tiles > 0) {
        if (DT == kF16) launch(k_attention_range<DT>, grid_of(a.n_tiles64), dim3(kAttentionThreads), 0, s, a);
        launch(k_attention_queries<DT, DP, EXT, NQ>, attention_grid(a.n_tiles, a.heads), dim3(kAttentionThreads), 0, s, a);
        AttentionArgs b = a;
        if (NK != NQ) {
            b.tiles = a.tiles64;
            b.n_tiles = a.n_tiles64;
        }
        launch(k_attention_keys<DT, DP, EXT, NK>, attention_grid(b.n_tiles, a.kv_heads), dim3(kAttentionThreads), 0, s, b);
    }
    if (EXT)
        launch(k_table_sum<DT>, dim3((unsigned)((3 * (2 * a.reach + 1) + 15) / 16), (unsigned)a.heads), dim3(1024), 0, s, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t attention_backward_by_cells(const AttentionArgs& a, bool wide, hipStream_t s) {
    constexpr int NK = DP == 128 ? 1 : 2;       // (of 128 keys of 128 elements, two gradients do not fit the registers)
    const int cells = a.table ? a.extent[0] + a.extent[1] + a.extent[2] : 0;
#define SMC_CELLS(EXT) wide ? attention_backward_t<DT, DP, EXT, 2, NK>(a, s) : attention_backward_t<DT, DP, EXT, 1, 1>(a, s)
    if (cells == 0) return SMC_CELLS(0);
    if (cells <= 32) return SMC_CELLS(32);
    if (cells <= 64) return SMC_CELLS(64);
    return SMC_CELLS(128);
#undef SMC_CELLS
}

template <int DT>
hipError_t attention_backward_of_type(const AttentionArgs& a, bool wide, hipStream_t s) {
    if (a.dim <= 32) return attention_backward_by_cells<DT, 32>(a, wide, s);
    if (a.dim <= 64) return attention_backward_by_cells<DT, 64>(a, wide, s);
    return attention_backward_by_cells<DT, 128>(a, wide, s);
}

}  // namespace
}  // namespace smc
