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
// delta is taken from out, which was rounded: an error of half an ulp of each out term, over the
// window's mean of k on its way into dq. Where a window's keys fit one tile delta is the sum of P dP
// itself instead (long windows average the error away; blocks of 128 queries have no registers for it).
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
template <int DT, bool A>
__global__ __launch_bounds__(256) void k_attention_range(AttentionArgs a) {
    if (block_number() >= a.n_tiles64) return;
    const WindowTile t = a.tiles64[block_number()];
    const int lane = threadIdx.x & 63, all = a.heads + a.kv_heads;
    const int row = lane < t.count ? a.places[t.first + lane].row : -1;
    for (int h = threadIdx.x >> 6; h < all; h += 4) {
        const bool of_v = h >= a.heads;
        const void* base = of_v ? a.v : a.dout;
        const int64_t at = (int64_t)row * (of_v ? a.ldv : a.ld_dout) + (of_v ? h - a.heads : h) * a.dim;
        uint32_t most = 0;
        if (row >= 0)
            for (int c = 0; c < a.dim; c += W) most = word_most<DT>(row_word<A>(base, at + c, a.dim - c), most);
        most = lane_max<64>(most);
        if (lane == 0) reinterpret_cast<uint32_t*>(a.range)[block_number() * all + h] = most;
    }
}

// The power of two that dS is taken times in tile t's window, for a head and its head of v.
template <int THREADS>
__device__ __forceinline__ float gradient_scale(const AttentionArgs& a, const WindowTile& t, int head, int kv) {
    __shared__ uint32_t s_most[2][THREADS / 64];
    // the window's tiles of 64 lie behind each other; find its first by its place
    int lo = 0, hi = a.n_tiles64 - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.tiles64[mid].first < t.begin) lo = mid + 1;
        else hi = mid;
    }
    const int count = (t.end - t.begin + 63) / 64, all = a.heads + a.kv_heads;
    uint32_t most[2] = {0u, 0u};
    for (int i = threadIdx.x; i < count; i += THREADS) {
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
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) most[k] = max(most[k], s_most[k][w]);
    const float bound = 2.f * (float)a.dim * __uint_as_float(most[0]) * __uint_as_float(most[1]);
    if (!(bound > 0.f)) return 1.f;
    // bound is within 2^-46 and 2^40
    return __uint_as_float((uint32_t)(127 + 14 - ((int)(__float_as_uint(bound) >> 23) - 127)) << 23);
}

// lse as an exponent's base: where there is no key P is 0.
__device__ __forceinline__ float lse_base(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads) void k_attention_queries(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16, ET16 = EXT / 16;
    constexpr int NQ = B::kColumns, TH = B::kThreads, kBins = EXT ? EXT / 32 : 1;
    constexpr bool kOwnDelta = B::kRows <= 64;          // (see the top)
    typedef Walk<DT, DP, EXT, A, B, 1> Keys;
    __shared__ __align__(16) typename Keys::Memory s_keys;
    __shared__ __align__(16) uint16_t s_table[EXT ? 2 * kTableEntries<EXT> : 2];
    // dB of 16 queries a wave (rows 4 floats longer than their cells), then the waves' sums by distance
    __shared__ __align__(16) float s_db[EXT ? B::kWaves * 16 * (EXT + 4) : 1];
    int tile, head;
    if (!tile_and_head(a.n_tiles, a.heads, tile, head)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int kv = head / (a.heads / a.kv_heads);
    if (EXT) load_table<DT, EXT, TH, false>(a, head, s_table);
    const float grow = DT == kF16 ? gradient_scale<TH>(a, t, head, kv) : 1.f;
    const float shrink = 1.f / grow;                    // (a power of two)
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const bool one = t.end - t.begin <= kKeys;
    // a window of one row: P is 1 whatever q, k and the bias are
    const float keep = t.end - t.begin == 1 ? 0.f : grow;
    float bins[kBins];                                  // sums of dS by distance, 64 of them a word: a lane each
#pragma unroll
    for (int i = 0; i < kBins; ++i) bins[i] = 0.f;

    const bool active = wave * NQ * 16 < t.count;
    WindowPlace own[NQ];
    float base[NQ], delta[NQ];
    u32x4 fq[NQ][CK], fo[NQ][CK], fb[NQ][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        const int i = (wave * NQ + u) * 16 + col;
        own[u] = own_place(a, t, i);
        base[u] = own[u].row < 0 ? INFINITY : lse_base(a.lse[(int64_t)head * a.n + t.first + i]);
        delta[u] = 0.f;
#pragma unroll
        for (int c = 0; c < CK; ++c) {
            const int at = head * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
            fq[u][c] = row_word<A>(a.q, (int64_t)own[u].row * a.ldq + at, left);
            fo[u][c] = row_word<A>(a.dout, (int64_t)own[u].row * a.ld_dout + at, left);
            if (kOwnDelta && one) continue;
            const u32x4 out = row_word<A>(a.out, (int64_t)own[u].row * a.ldo + at, left);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                delta[u] += to_f32<DT>(out[d] & 0xffffu) * to_f32<DT>(fo[u][c][d] & 0xffffu) +
                            to_f32<DT>(out[d] >> 16) * to_f32<DT>(fo[u][c][d] >> 16);
        }
    }
    Keys keys;
    keys.start(a, s_keys, t, a.k, a.ldk, a.v, a.ldv, kv * a.dim);
    if (EXT)
#pragma unroll
        for (int u = 0; u < NQ; ++u)
                table_words<EXT>(a, s_table, own[u].cells, q, fb[u]);
    f32x4 dq[NQ][DT16], db[NQ][ET16 ? ET16 : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        delta[u] = quad_sum(delta[u]);
#pragma unroll
        for (int d = 0; d < DT16; ++d) dq[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < ET16; ++d) db[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    // 64 keys, or the window's last `left`
    const char *const s_k = s_keys.x[0], *const s_v = s_keys.y[0], *const s_e = s_keys.e[0];
    auto step = [&](int left) SMC_INLINE {
        // P and dP of 16 keys each, `b`
        auto pair = [&](int b, f32x4 (&s)[NQ], f32x4 (&dp)[NQ]) SMC_INLINE {
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
            if (left < kKeys)                   // keys past the end
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][e] = 16 * b + 4 * q + e < left ? s[u][e] : -INFINITY;
#pragma unroll
            for (int u = 0; u < NQ; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[u][e] = exp2_of(s[u][e] * to_log2 - base[u]);
        };
        auto slope = [&](const f32x4& p, const f32x4& dp, int u, u32x4& g, int b) SMC_INLINE {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = p[e] * fmaf(dp[e], keep, -(delta[u] * keep));
            g[2 * (b & 1)] = pack2<DT>(v[0], v[1]);
            g[2 * (b & 1) + 1] = pack2<DT>(v[2], v[3]);
        };
        auto products = [&](int h, const u32x4 (&g)[NQ]) SMC_INLINE {
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
        };
        if constexpr (kOwnDelta) {
            f32x4 s[4][NQ], dp[4][NQ];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (!B::kSkips || 16 * b < left) {
                    pair(b, s[b], dp[b]);
                } else {
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[b][u] = dp[b][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
                }
            }
            if (one)
#pragma unroll
                for (int u = 0; u < NQ; ++u) {
                    float v = 0.f;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v += s[b][u][e] * dp[b][u][e];
                    delta[u] = quad_sum(v);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (B::kSkips && 32 * h >= left) continue;
                u32x4 g[NQ];
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int b = 2 * h; b < 2 * h + 2; ++b) slope(s[b][u], dp[b][u], u, g[u], b);
                products(h, g);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {           // 32 keys at a time
                if (B::kSkips && 32 * h >= left) continue;
                u32x4 g[NQ];
#pragma unroll
                for (int b = 2 * h; b < 2 * h + 2; ++b) {
                    f32x4 s[NQ], dp[NQ];
                    pair(b, s, dp);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) slope(s[u], dp[u], u, g[u], b);
                }
                products(h, g);
            }
        }
    };
    const int length = t.end - t.begin;
    if (length > 0) keys.commit(a, s_keys, 0, t);
    for (int i = 0; i * kKeys < length; ++i) {
        const int left = length - i * kKeys;
        if (left > kKeys) keys.load(a, s_keys, i + 1, a.k, a.ldk, a.v, a.ldv, kv * a.dim);
        if (active) step(left);
        if (left > kKeys) keys.commit(a, s_keys, i + 1, t);
    }
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        if (q == 0 && own[u].row >= 0)
            a.delta[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] = delta[u];
        store_row<DT, DP, A>(dq[u], a.scale * shrink, a.dq,
                          own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dq + head * a.dim, a.dim, lane);
    }
    if constexpr (EXT > 0) {
        // 16 queries at a time: dB to LDS, then each lane adds what lies at its distances, query
        // after query
        const Cells cells(a.extent);
        float* const mine = s_db + wave * 16 * (EXT + 4);
        if (active)
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                const int rows = min(16, t.count - (wave * NQ + u) * 16);
                if (rows <= 0) continue;
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int d = 0; d < ET16; ++d) *reinterpret_cast<f32x4*>(mine + col * (EXT + 4) + 16 * d + 4 * q) = db[u][d];
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < kBins; ++i) {
                    const int bin = 64 * i + lane, axis = cells.axis_of_entry(bin), first = cells.pick(cells.first, axis);
                    const int away = cells.pick(cells.up, axis) - (bin - 2 * first), extent = cells.pick(a.extent, axis);
                    float v = 0.f;
                    if (64 * i < 2 * cells.all())
                        for (int r = 0; r < rows; ++r) {
                            const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)own[u].cells, r);
                            const int c = (int)((at >> (8 * axis)) & 255u) - away;      // the key's cell
                            const bool in = c >= first && c < first + extent;
                            const float x = mine[r * (EXT + 4) + (in ? c : 0)];
                            v += in ? x : 0.f;
                        }
                    bins[i] += bin < 2 * cells.all() ? v : 0.f;
                }
            }
    }
    if constexpr (EXT > 0) {
        // the waves' sums, then buckets: the outermost ones hold every distance beyond them
        float* const s_by = s_db;                       // [wave][64 kBins]
        static_assert(B::kWaves * 64 * kBins <= B::kWaves * 16 * (EXT + 4), "room");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBins; ++i) s_by[(wave * kBins + i) * 64 + lane] = bins[i];
        __syncthreads();
        const int buckets = 2 * a.reach + 1;
        float* const part = a.part + ((int64_t)tile * a.heads + head) * 3 * buckets;
        for (int i = threadIdx.x; i < 3 * buckets; i += TH) {
            const Cells cells(a.extent);
            const int axis = i / buckets, d = i % buckets - a.reach, far = cells.pick(a.extent, axis) - 1;
            const int zero = 2 * cells.pick(cells.first, axis) + cells.pick(cells.up, axis);
            const int from = d == -a.reach ? -far : max(d, -far), to = d == a.reach ? far : min(d, far);
            float v = 0.f;
            for (int k = from; k <= to; ++k)
#pragma unroll
                for (int w = 0; w < B::kWaves; ++w) v += s_by[w * kBins * 64 + zero - k];
            part[i] = v * shrink;
        }
    }
}

template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads) void k_attention_keys(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    constexpr int NK = B::kColumns, TH = B::kThreads;
    typedef Walk<DT, DP, EXT, A, B, 1> Queries;
    __shared__ __align__(16) typename Queries::Memory s_queries;
    __shared__ __align__(16) float s_base[kKeys], s_delta[kKeys];
    __shared__ __align__(16) uint16_t s_table[EXT ? 2 * kTableEntries<EXT> : 2];
    int tile, kv;
    if (!tile_and_head(a.n_tiles, a.kv_heads, tile, kv)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int each = a.heads / a.kv_heads;
    float grow = 1.f;
    if (DT == kF16) {                           // the smallest factor of the group's heads serves all
        grow = gradient_scale<TH>(a, t, kv * each, kv);
        for (int i = 1; i < each; ++i) grow = fminf(grow, gradient_scale<TH>(a, t, kv * each + i, kv));
    }
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    // a window of one row: P is 1 whatever q, k and the bias are
    const float keep = t.end - t.begin == 1 ? 0.f : grow;
    const bool active = wave * NK * 16 < t.count;
    WindowPlace own[NK];
#pragma unroll
    for (int u = 0; u < NK; ++u) own[u] = own_place(a, t, (wave * NK + u) * 16 + col);
    u32x4 fk[NK][CK], fv[NK][CK], fb[NK][CE ? CE : 1];
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
        for (int c = 0; c < CK; ++c) {
            const int at = kv * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
            fk[u][c] = row_word<A>(a.k, (int64_t)own[u].row * a.ldk + at, left);
            fv[u][c] = row_word<A>(a.v, (int64_t)own[u].row * a.ldv + at, left);
        }
    f32x4 dk[NK][DT16], dv[NK][DT16];
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
        for (int d = 0; d < DT16; ++d) dk[u][d] = dv[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int head = kv * each; head < (kv + 1) * each; ++head) {
        __syncthreads();                        // (the tiles and the table of the head before)
        if (EXT) load_table<DT, EXT, TH, true>(a, head, s_table);
        Queries queries;
        queries.start(a, s_queries, t, a.q, a.ldq, a.dout, a.ld_dout, head * a.dim);
        if (EXT)
#pragma unroll
            for (int u = 0; u < NK; ++u) table_words<EXT>(a, s_table, own[u].cells, q, fb[u]);
        const float* const lse = a.lse + (int64_t)head * a.n;
        const float* const deltas = a.delta + (int64_t)head * a.n;
        float base = INFINITY, delta = 0.f;     // of this thread's query, in the first 64 threads
        auto load_query = [&](int i) SMC_INLINE {
            const int at = t.begin + i * kKeys + (int)threadIdx.x;
            const bool in = threadIdx.x < kKeys && at < t.end;
            base = in ? lse_base(lse[at]) : INFINITY;       // past the end: P is 0
            delta = in ? deltas[at] * keep : 0.f;
        };
        auto commit = [&](int i) SMC_INLINE {
            __syncthreads();
            if (threadIdx.x < kKeys) {
                s_base[threadIdx.x] = base;
                s_delta[threadIdx.x] = delta;
            }
            queries.commit(a, s_queries, i, t);
        };
        load_query(0);
        const int length = t.end - t.begin;
        if (length > 0) commit(0);
        for (int i = 0; i * kKeys < length; ++i) {
            const int left = length - i * kKeys;
            if (left > kKeys) {
                queries.load(a, s_queries, i + 1, a.q, a.ldq, a.dout, a.ld_dout, head * a.dim);
                load_query(i + 1);
            }
            const char *const s_q = s_queries.x[0], *const s_o = s_queries.y[0], *const s_e = s_queries.e[0];
            if (active)
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
                            w[e] = v[e] * fmaf(dp[u][e], keep, -dl[e]);
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
            if (left > kKeys) commit(i + 1);
        }
    }
    const float f = a.scale / grow;
#pragma unroll
    for (int u = 0; u < NK; ++u) {
        const int at = kv * a.dim;
        store_row<DT, DP, A>(dk[u], f, a.dk, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dk + at, a.dim, lane);
        store_row<DT, DP, A>(dv[u], 1.f, a.dv, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dv + at, a.dim, lane);
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

template <int DT, int DP, int EXT, bool A, class BQ, class BK>
hipError_t attention_backward_t(const AttentionArgs& a, hipStream_t s) {
    if (a.n_tiles > 0) {
        if (DT == kF16) launch(k_attention_range<DT, A>, grid_of(a.n_tiles64), dim3(256), 0, s, a);
        launch(k_attention_queries<DT, DP, EXT, A, BQ>, attention_grid(a.n_tiles, a.heads), dim3(BQ::kThreads), 0, s, a);
        AttentionArgs b = a;
        if (BK::kRows == 64) {
            b.tiles = a.tiles64;
            b.n_tiles = a.n_tiles64;
        }
        launch(k_attention_keys<DT, DP, EXT, A, BK>, attention_grid(b.n_tiles, a.kv_heads), dim3(BK::kThreads), 0, s, b);
    }
    if (EXT)
        launch(k_table_sum<DT>, dim3((unsigned)((3 * (2 * a.reach + 1) + 15) / 16), (unsigned)a.heads), dim3(1024), 0, s, a);
    return hipGetLastError();
}

template <int DT, int DP, int EXT>
hipError_t attention_backward_by_length(const AttentionArgs& a, int lengths, hipStream_t s) {
    // (of 128 keys of 128 elements, two gradients do not fit the registers)
    typedef typename std::conditional<DP == 128, BlockMid, BlockLong>::type BlockKeys;
    if (lengths == kShortWindows) return attention_backward_t<DT, DP, EXT, true, BlockShort<DP>, BlockShort<DP>>(a, s);
    if (lengths == kMidWindows) return attention_backward_t<DT, DP, EXT, true, BlockMid, BlockMid>(a, s);
    return attention_backward_t<DT, DP, EXT, true, BlockLong, BlockKeys>(a, s);
}

template <int DT, int DP>
hipError_t attention_backward_by_cells(const AttentionArgs& a, int lengths, hipStream_t s) {
    const int cells = a.table ? Cells(a.extent).all() : 0;
    if (!a.vec)                                 // (one kernel a width, as in the forward pass)
        return cells == 0 ? attention_backward_t<DT, DP, 0, false, BlockMid, BlockMid>(a, s)
                          : attention_backward_t<DT, DP, 128, false, BlockMid, BlockMid>(a, s);
    if (cells == 0) return attention_backward_by_length<DT, DP, 0>(a, lengths, s);
    if (cells <= 32) return attention_backward_by_length<DT, DP, 32>(a, lengths, s);
    if (cells <= 64) return attention_backward_by_length<DT, DP, 64>(a, lengths, s);
    return attention_backward_by_length<DT, DP, 128>(a, lengths, s);
}

template <int DT>
hipError_t attention_backward_of_type(const AttentionArgs& a, int lengths, hipStream_t s) {
    if (a.dim <= 32) return attention_backward_by_cells<DT, 32>(a, lengths, s);
    if (a.dim <= 64) return attention_backward_by_cells<DT, 64>(a, lengths, s);
    return attention_backward_by_cells<DT, 128>(a, lengths, s);
}

}  // namespace
}  // namespace smc
