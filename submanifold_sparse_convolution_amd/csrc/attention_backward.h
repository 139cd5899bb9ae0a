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
// them up by distance and writes its buckets, k_table_sum adds the blocks. 91,000 rows in 2,905
// windows: queries 93.9 us, keys 68.1, sums 9.8; 15,000 x 512 in windows of 1,024: 131, 118 and 4.8.
// (Distances looked up for each entry of dB in place of rows shifted by the query's cell: 107.2 and 134.)
//
// P and dS are rounded to the rows' type as operands (half an ulp of each term). Not so for the
// table's gradient, whose sums over all windows cancel: it takes what the rounding leaves of dS as
// a second operand (without it up to 1.6 times float32's error; 15,000 x 512 in windows of 1,024
// 236 us for 226 a call, 91,000 rows in 2,905 windows 180.4 for 179.8). dS follows
// the gradient's size, which in f16 may leave the type's range where dq and dk do not,
// so in f16 it is taken times a power of two: |dP - delta| <= 2 dim max |dout| max |v| over
// the window (finite values), brought to [2^14, 2^15]; k_attention_range finds the maxima. P, for dv, is taken times
// 2^12 there: in windows of more than some 16,000 rows the mean P is below f16's normal numbers (2^-14), and so are
// keys of little weight in any (with it 95,000 rows of equal scores lost 0.2 % of dv). (12 taken off a base is exact up
// to 2^26; beyond, P is off by the base's half ulp, 4 powers of two and more, and may leave f16.)
// delta is taken from out, which was rounded: an error of half an ulp of each out term, over the
// window's mean of k on its way into dq. Where a window's keys fit one tile delta is the mean of dP
// under P itself instead (long windows average the error away; blocks of 128 queries have no registers for it).
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

// f16: largest |dout| of each head and |v| of each of its heads in a tile of 64 places. The block's threads
// take the tile's words in order, so that loads are whole lines.
template <int DT, bool A>
__global__ __launch_bounds__(256) void k_attention_range(AttentionArgs a) {
    __shared__ uint32_t s_most[256];
    __shared__ int s_row[64];
    if (block_number() >= a.n_tiles64) return;
    const WindowTile t = a.tiles64[block_number()];
    const int all = a.heads + a.kv_heads, per = (a.dim + W - 1) / W;
    if (threadIdx.x < 64) s_row[threadIdx.x] = threadIdx.x < t.count ? a.places[t.first + threadIdx.x].row : -1;
    for (int h0 = 0; h0 < all; h0 += 256) {
        const int heads = min(all - h0, 256), words = heads * per, n = t.count * words;
        __syncthreads();
        s_most[threadIdx.x] = 0;
        __syncthreads();
        for (int i0 = threadIdx.x; i0 < n; i0 += 4 * 256) {
            u32x4 w[4];
            int head[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = min(i0 + 256 * k, n - 1), r = i / words, x = i - r * words;
                head[k] = x / per;
                const int c = (x - head[k] * per) * W, h = h0 + head[k];
                const bool of_v = h >= a.heads;
                w[k] = row_word<A>(of_v ? a.v : a.dout, (int64_t)s_row[r] * (of_v ? a.ldv : a.ld_dout) +
                                   (int64_t)(of_v ? h - a.heads : h) * a.dim + c, a.dim - c);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) atomicMax(&s_most[head[k]], word_most<DT>(w[k], 0u));
        }
        __syncthreads();
        if (threadIdx.x < heads)
            reinterpret_cast<uint32_t*>(a.range)[block_number() * all + h0 + threadIdx.x] = s_most[threadIdx.x];
    }
}

// The maxima of tile t's window, for a head and its head of v: each lane's share of them. Every wave takes them
// for itself, before its rows are loaded (by the block, between barriers, 91,000 f16 rows in windows of 31 took
// 120.6 us a backward call; so 105.4; bf16, which needs none of it, 81.5).
struct WindowMost {
    uint32_t most[2];
    __device__ __forceinline__ void load(const AttentionArgs& a, const WindowTile& t, int head, int kv) {
        const int count = (t.end - t.begin + 63) / 64, all = a.heads + a.kv_heads;
        most[0] = most[1] = 0u;
        for (int i = threadIdx.x & 63; i < count; i += 64) {
            const uint32_t* r = reinterpret_cast<const uint32_t*>(a.range) + (int64_t)(t.first64 + i) * all;
            most[0] = max(most[0], r[head]);
            most[1] = max(most[1], r[a.heads + kv]);
        }
    }
    // The power of two that dS is taken times, of whole waves.
    __device__ __forceinline__ float scale(int dim) const {
        const float bound = 2.f * (float)dim * __uint_as_float(lane_max<64>(most[0])) * __uint_as_float(lane_max<64>(most[1]));
        // bound is within 2^-46 and 2^40
        const uint32_t by = (uint32_t)(127 + 14 - ((int)(__float_as_uint(bound) >> 23) - 127)) << 23;
        return __uint_as_float(__builtin_amdgcn_readfirstlane(bound > 0.f ? by : __float_as_uint(1.f)));
    }
};

// lse as an exponent's base: where there is no key P is 0.
__device__ __forceinline__ float lse_base(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// (waves a SIMD by what the registers take; 91,000 rows at three 93.8 us, at two 120; 16,000 x 8 heads of 64 in windows
// of 60, a backward call with three 40.1 us, with two 42.7)
template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads, (DP <= 32 && EXT <= 32) || (DP == 64 && EXT == 0 && B::kRows == 64) ? 3 : DP <= 64 && DP + EXT <= 160 ? 2 : 1)
void k_attention_queries(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16, ET16 = EXT / 16;
    constexpr int NQ = B::kColumns, TH = B::kThreads, kBins = EXT ? EXT / 32 : 1;
    constexpr bool kOwnDelta = B::kRows <= 64;          // (see the top)
    typedef Walk<DT, DP, EXT, A, B, 1> Keys;
    __shared__ __align__(16) typename Keys::Memory s_keys;
    __shared__ __align__(16) uint16_t s_table[B::kHeads][EXT ? 2 * kTableEntries<EXT> : 2];
    // dB of 16 or 8 queries a wave by distance (rows five floats longer than their entries, for other banks)
    constexpr int kRow = 2 * EXT + 5, kRowsOf = EXT <= 32 ? 16 : 8;
    __shared__ __align__(16) float s_db[EXT ? B::kWaves * kRowsOf * kRow : 1];
    int tile, head;
    if (!tile_and_head(a.n_tiles, a.heads, a.heads_each, tile, head)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int share = a.heads / a.kv_heads, first_head = head, heads = min(a.heads_each, a.heads - head);
    const int length = t.end - t.begin;
    // (rows of no window walk none: products of what they hold with zeros need not be zero)
    const bool active = wave * NQ * 16 < t.count && length > 0, one = length <= kKeys;      // one: one step a head
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const TileLane<RW> at(lane);
    const TileLane<RE> at_cells(lane);
    WindowPlace own[NQ];
#pragma unroll
    for (int u = 0; u < NQ; ++u) own[u] = own_place(a, t, (wave * NQ + u) * 16 + col);
    Keys keys;
    keys.places(a, t, 0);
    if (EXT) load_tables<DT, EXT, TH, B::kHeads>(a, head, heads, s_table);
    u32x4 fq[NQ][CK], fo[NQ][CK], fb[NQ][CE ? CE : 1];
    float base[NQ], delta[NQ], grow = 1.f, keep = 1.f;
    auto load_queries = [&](int h, u32x4 (&f)[NQ][CK], u32x4 (&g)[NQ][CK], float (&lse)[NQ]) SMC_INLINE {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            lse[u] = -INFINITY;
            if (own[u].row >= 0) lse[u] = a.lse[(int64_t)h * a.n + t.first + (wave * NQ + u) * 16 + col];
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                const int c0 = h * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
                f[u][c] = row_word<A>(a.q, (int64_t)own[u].row * a.ldq + c0, left);
                g[u][c] = row_word<A>(a.dout, (int64_t)own[u].row * a.ld_dout + c0, left);
            }
        }
    };
    WindowMost most[B::kHeads];
    if (DT == kF16)
#pragma unroll
        for (int h = 0; h < B::kHeads; ++h)
            if (h < heads) most[h].load(a, t, head + h, (head + h) / share);
    load_queries(head, fq, fo, base);
    keys.point(a.k, a.v, head / share * a.dim);
    keys.load(a, a.ldk, a.ldv);
    if (!one) keys.places(a, t, 1);
    float grows[B::kHeads];
#pragma unroll
    for (int h = 0; h < B::kHeads; ++h) grows[h] = DT == kF16 && h < heads ? most[h].scale(a.dim) : 1.f;
    f32x4 dq[NQ][DT16], db[NQ][ET16 ? ET16 : 1];
    auto begin_head = [&]() SMC_INLINE {
        if (DT == kF16) grow = grows[B::kHeads > 1 && head > first_head];
        keep = length == 1 ? 0.f : grow;        // a window of one row: P is 1 whatever q, k and the bias are
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            base[u] = lse_base(base[u]);
            delta[u] = 0.f;
            if (!kOwnDelta || !one) {
#pragma unroll
                for (int c = 0; c < CK; ++c) {
                    const u32x4 out = row_word<A>(a.out, (int64_t)own[u].row * a.ldo + head * a.dim + 32 * c + 8 * q,
                                                  own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q);
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        delta[u] += to_f32<DT>(out[d] & 0xffffu) * to_f32<DT>(fo[u][c][d] & 0xffffu) +
                                    to_f32<DT>(out[d] >> 16) * to_f32<DT>(fo[u][c][d] >> 16);
                }
                delta[u] = quad_sum(delta[u]);
            }
            if (EXT) table_words<EXT>(a, s_table[head - first_head], own[u].cells, q, fb[u]);
#pragma unroll
            for (int d = 0; d < DT16; ++d) dq[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < ET16; ++d) db[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
    };
    // 64 keys, or the window's last `left`
    const char *const s_k = s_keys.x[0], *const s_v = s_keys.y[0], *const s_e = s_keys.e[0];
    auto step = [&](int left) SMC_INLINE {
        // P and dP of 16 keys each, `b`
        auto pair = [&](int b, f32x4 (&s)[NQ], f32x4 (&dp)[NQ]) SMC_INLINE {
#pragma unroll
            for (int u = 0; u < NQ; ++u) s[u] = dp[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                const u32x4 fk = at.along(s_k, 16 * b, c);
                const u32x4 fv = at.along(s_v, 16 * b, c);
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
                    const u32x4 fe = at_cells.along(s_e, 16 * b, c);
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
        // dS, and with a table what its rounding leaves
        auto slope = [&](const f32x4& p, const f32x4& dp, int u, u32x4& g, u32x4& rest, int b) SMC_INLINE {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = p[e] * fmaf(dp[e], keep, -(delta[u] * keep));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w = pack2<DT>(v[2 * i], v[2 * i + 1]);
                g[2 * (b & 1) + i] = w;
                if (EXT) rest[2 * (b & 1) + i] = pack2<DT>(v[2 * i] - to_f32<DT>(w & 0xffffu), v[2 * i + 1] - to_f32<DT>(w >> 16));
            }
        };
        auto products = [&](int h, const u32x4 (&g)[NQ], const u32x4 (&rest)[NQ]) SMC_INLINE {
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const u32x4 f = at.across(s_k, d, 32 * h);
#pragma unroll
                for (int u = 0; u < NQ; ++u) dq[u][d] = mfma16<DT>(f, g[u], dq[u][d]);
            }
            if (EXT)
#pragma unroll
                for (int d = 0; d < ET16; ++d) {
                    const u32x4 f = at_cells.across(s_e, d, 32 * h);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) db[u][d] = mfma16<DT>(f, g[u], mfma16<DT>(f, rest[u], db[u][d]));
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
                    float v = 0.f, total = 0.f;         // (over the sum of P: lse of large scores has few digits)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v += s[b][u][e] * dp[b][u][e];
                            total += s[b][u][e];
                        }
                    total = quad_sum(total);
                    delta[u] = total == 0.f ? 0.f : quad_sum(v) / total;
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (B::kSkips && 32 * h >= left) continue;
                u32x4 g[NQ], rest[NQ];
#pragma unroll
                for (int u = 0; u < NQ; ++u)
#pragma unroll
                    for (int b = 2 * h; b < 2 * h + 2; ++b) slope(s[b][u], dp[b][u], u, g[u], rest[u], b);
                products(h, g, rest);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {           // 32 keys at a time
                if (B::kSkips && 32 * h >= left) continue;
                u32x4 g[NQ], rest[NQ];
#pragma unroll
                for (int b = 2 * h; b < 2 * h + 2; ++b) {
                    f32x4 s[NQ], dp[NQ];
                    pair(b, s, dp);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) slope(s[u], dp[u], u, g[u], rest[u], b);
                }
                products(h, g, rest);
            }
        }
    };
    auto end_head = [&]() SMC_INLINE {
        const float shrink = 1.f / grow;        // (a power of two)
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            if (q == 0 && own[u].row >= 0)
                a.delta[(int64_t)head * a.n + t.first + (wave * NQ + u) * 16 + col] = delta[u];
            store_row<DT, DP, A>(dq[u], a.scale * shrink, a.dq,
                                 own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dq + head * a.dim, a.dim, lane);
        }
        if constexpr (EXT > 0) {
            // A few queries at a time: a query's dB to a row of LDS at its own distances (as TableLoads counts the
            // entries), zeros around it, and the rows added, a lane for each 64th entry
            const Cells cells(a.extent);
            float* const mine = s_db + wave * kRowsOf * kRow;
            float bins[kBins];
#pragma unroll
            for (int i = 0; i < kBins; ++i) bins[i] = 0.f;
            if (active)
#pragma unroll
                for (int u = 0; u < NQ; ++u) {
                    int at[3];          // the entry of element 0
#pragma unroll
                    for (int d = 0; d < 3; ++d)
                        at[d] = 2 * cells.first[d] + cells.up[d] - (int)((own[u].cells >> (8 * d)) & 255u);
#pragma unroll
                    for (int half = 0; half < 16 / kRowsOf; ++half) {
                        if (t.count <= (wave * NQ + u) * 16 + 8 * half) continue;
                        __builtin_amdgcn_wave_barrier();
                        // (one set of rows keeps its places from head to head)
                        if (NQ > 1 || kRowsOf < 16 || head == first_head)
                            for (int i = lane; i < kRowsOf * kRow; i += 64) mine[i] = 0.f;
                        __builtin_amdgcn_wave_barrier();
                        if (col / kRowsOf == half && own[u].row >= 0)
#pragma unroll
                            for (int d = 0; d < ET16; ++d) {
                                const int e = 16 * d + 4 * q;
                                float* to = mine + (col & (kRowsOf - 1)) * kRow + e;
                                to += e < cells.first[1] ? at[0] : e < cells.first[2] ? at[1] : at[2];
                                if (e < cells.all())
#pragma unroll
                                    for (int k = 0; k < 4; ++k) to[k] = db[u][d][k];
                            }
                        __builtin_amdgcn_wave_barrier();
#pragma unroll
                        for (int i = 0; i < kBins; ++i) {
                            float v = 0.f;
#pragma unroll
                            for (int r = 0; r < kRowsOf; ++r) v += mine[r * kRow + 64 * i + lane];
                            bins[i] += v;
                        }
                    }
                }
            // the waves' sums, then buckets: the outermost ones hold every distance beyond them
            __shared__ float s_by[B::kWaves * 64 * kBins];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kBins; ++i) s_by[(wave * kBins + i) * 64 + lane] = bins[i];
            __syncthreads();
            const int buckets = 2 * a.reach + 1;
            float* const part = a.part + ((int64_t)tile * a.heads + head) * 3 * buckets;
            for (int i = threadIdx.x; i < 3 * buckets; i += TH) {
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
    };
    int i = 0;                          // the step of the head
    keys.commit(s_keys, 0, true);
    begin_head();
    for (;;) {
        const int left = length - i * kKeys;
        const bool last = left <= kKeys, more = !last || head + 1 < first_head + heads;
        u32x4 fq_next[B::kHeads > 1 ? NQ : 1][CK], fo_next[B::kHeads > 1 ? NQ : 1][CK];
        float base_next[B::kHeads > 1 ? NQ : 1];
        if (more) {
            if constexpr (B::kHeads > 1)
                if (last) {
                    keys.point(a.k, a.v, (head + 1) / share * a.dim);
                    load_queries(head + 1, fq_next, fo_next, base_next);
                }
            keys.load(a, a.ldk, a.ldv);
            if (!one) keys.places(a, t, (last ? 1 : i + 2) * kKeys < length ? (last ? 1 : i + 2) : 0);
        }
        if (active) step(left);
        if (last) end_head();
        if (!more) break;
        keys.commit(s_keys, 0, !one);
        ++i;
        if constexpr (B::kHeads > 1)
            if (last) {
                i = 0;
                ++head;
#pragma unroll
                for (int u = 0; u < NQ; ++u) {
                    base[u] = base_next[u];
#pragma unroll
                    for (int c = 0; c < CK; ++c) {
                        fq[u][c] = fq_next[u][c];
                        fo[u][c] = fo_next[u][c];
                    }
                }
                begin_head();
            }
    }
}

template <int DT, int DP, int EXT, bool A, class B>
__global__ __launch_bounds__(B::kThreads, DP <= 64 && DP + EXT <= 160 ? 2 : 1) void k_attention_keys(AttentionArgs a) {
    constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, CK = DP / 32, CE = EXT / 32, DT16 = DP / 16;
    constexpr int NK = B::kColumns, TH = B::kThreads;
    constexpr float kLift = DT == kF16 ? 12.f : 0.f;            // P is times 2^kLift, by its base
    // (places past the end have a base of inf, P and dS of 0, also beside k of infinities)
    typedef Walk<DT, DP, EXT, A, B, 1, true> Queries;
    __shared__ __align__(16) typename Queries::Memory s_queries;
    __shared__ __align__(16) float s_base[kKeys], s_delta[kKeys];
    __shared__ __align__(16) uint16_t s_table[EXT ? 2 * kTableEntries<EXT> : 2];
    int tile, kv;                       // the block's heads: those of `heads_each` heads of k and v from kv on
    if (!tile_and_head(a.n_tiles, a.kv_heads, a.heads_each, tile, kv)) return;
    const WindowTile t = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
    const int share = a.heads / a.kv_heads, end_head = min(kv + a.heads_each, a.kv_heads) * share;
    const int length = t.end - t.begin;
    // (rows of no window walk none: products of what they hold with zeros need not be zero)
    const bool active = wave * NK * 16 < t.count && length > 0, one = length <= kKeys;      // one: one step a head
    const float to_log2 = EXT ? kLog2e : a.scale * kLog2e;
    const TileLane<RW> at(lane);
    const TileLane<RE> at_cells(lane);
    WindowPlace own[NK];
#pragma unroll
    for (int u = 0; u < NK; ++u) own[u] = own_place(a, t, (wave * NK + u) * 16 + col);
    Queries queries;
    queries.places(a, t, 0);
    u32x4 fk[NK][CK], fv[NK][CK], fb[NK][CE ? CE : 1];
    auto load_keys = [&](int h, u32x4 (&f)[NK][CK], u32x4 (&g)[NK][CK]) SMC_INLINE {
#pragma unroll
        for (int u = 0; u < NK; ++u)
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                const int c0 = h * a.dim + 32 * c + 8 * q, left = own[u].row < 0 ? 0 : a.dim - 32 * c - 8 * q;
                f[u][c] = row_word<A>(a.k, (int64_t)own[u].row * a.ldk + c0, left);
                g[u][c] = row_word<A>(a.v, (int64_t)own[u].row * a.ldv + c0, left);
            }
    };
    int head = kv * share, i = 0;       // the head, and its step
    bool with_cells = true;             // a window of one step has the same for every head
    TableLoads<DT, EXT, TH, true> table;
    float grow = 1.f, keep = 1.f, base = INFINITY, delta = 0.f;     // (of this thread's query, in the first 64)
    f32x4 dk[NK][DT16], dv[NK][DT16];
    auto begin_keys = [&]() SMC_INLINE {
        if (DT == kF16) {                       // the smallest factor of the heads that share them serves all
            grow = INFINITY;
            for (int h = 0; h < share; ++h) {
                WindowMost most;
                most.load(a, t, head + h, kv);
                grow = fminf(grow, most.scale(a.dim));
            }
        }
        keep = length == 1 ? 0.f : grow * exp2f(-kLift);        // a window of one row: P is 1 whatever q, k and the bias are
#pragma unroll
        for (int u = 0; u < NK; ++u)
#pragma unroll
            for (int d = 0; d < DT16; ++d) dk[u][d] = dv[u][d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    };
    auto end_keys = [&]() SMC_INLINE {
        const float f = a.scale / grow;
#pragma unroll
        for (int u = 0; u < NK; ++u) {
            const int c0 = kv * a.dim;
            store_row<DT, DP, A>(dk[u], f, a.dk, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dk + c0, a.dim, lane);
            store_row<DT, DP, A>(dv[u], exp2f(-kLift), a.dv, own[u].row < 0 ? -1 : (int64_t)own[u].row * a.ld_dv + c0, a.dim, lane);
        }
    };
    auto load = [&](int h, int step) SMC_INLINE {
        if (step == 0) {
            queries.point(a.q, a.dout, h * a.dim);
            if (EXT) table.load(a, h);
        }
        queries.load(a, a.ldq, a.ld_dout);
        const int place = t.begin + step * kKeys + (int)threadIdx.x;
        base = -INFINITY;                       // past the end: P is 0
        delta = 0.f;
        if (threadIdx.x < kKeys && place < t.end) {
            base = a.lse[(int64_t)h * a.n + place];
            delta = a.delta[(int64_t)h * a.n + place];
        }
    };
    auto commit = [&](bool first) SMC_INLINE {      // (first: of a head)
        __syncthreads();
        if (threadIdx.x < kKeys) {
            s_base[threadIdx.x] = lse_base(base) - kLift;
            s_delta[threadIdx.x] = delta * keep;
        }
        if (EXT && first) table.commit(a, s_table);
        queries.commit(s_queries, 0, with_cells);
        with_cells = !one;
        if (EXT && first)
#pragma unroll
            for (int u = 0; u < NK; ++u) table_words<EXT>(a, s_table, own[u].cells, q, fb[u]);
    };
    load_keys(kv, fk, fv);
    load(head, 0);
    if (!one) queries.places(a, t, 1);
    begin_keys();
    commit(true);
    const char *const s_q = s_queries.x[0], *const s_o = s_queries.y[0], *const s_e = s_queries.e[0];
    for (;;) {
        const bool last = length - i * kKeys <= kKeys, more = !last || head + 1 < end_head;
        const bool turns = last && head + 1 == (kv + 1) * share;        // other keys and values next
        u32x4 fk_next[B::kHeads > 1 ? NK : 1][CK], fv_next[B::kHeads > 1 ? NK : 1][CK];
        if (more) {
            load(last ? head + 1 : head, last ? 0 : i + 1);
            if constexpr (B::kHeads > 1)
                if (turns) load_keys(kv + 1, fk_next, fv_next);
            if (!one) queries.places(a, t, (last ? 1 : i + 2) * kKeys < length ? (last ? 1 : i + 2) : 0);
        }
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
                    const u32x4 fq = at.along(s_q, 16 * b, c);
                    const u32x4 fo = at.along(s_o, 16 * b, c);
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
                        const u32x4 fe = at_cells.along(s_e, 16 * b, c);
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
                const u32x4 fo = at.across(s_o, d, 32 * h);
                const u32x4 fq = at.across(s_q, d, 32 * h);
#pragma unroll
                for (int u = 0; u < NK; ++u) {
                    dv[u][d] = mfma16<DT>(fo, p[u], dv[u][d]);
                    dk[u][d] = mfma16<DT>(fq, g[u], dk[u][d]);
                }
            }
        }
        if (turns) end_keys();
        if (!more) break;
        ++i;
        if (last) {
            i = 0;
            ++head;
        }
        if constexpr (B::kHeads > 1)
            if (turns) {
                ++kv;
#pragma unroll
                for (int u = 0; u < NK; ++u)
#pragma unroll
                    for (int c = 0; c < CK; ++c) {
                        fk[u][c] = fk_next[u][c];
                        fv[u][c] = fv_next[u][c];
                    }
                begin_keys();
            }
        commit(last);
    }
}

// dtable = the blocks' buckets: 4 buckets a block, 256 strided runs of tiles joined by a tree.
// (16 buckets of 64 runs, whose loads are 64 bytes each but 74 after each other: 11.9 us for 9.8 at
// 4,756 tiles of 4 heads and 69 buckets.)
constexpr int kBucketsOf = 4, kRunsOf = 1024 / kBucketsOf;
template <int DT>
__global__ __launch_bounds__(1024) void k_table_sum(AttentionArgs a) {
    __shared__ float s[kRunsOf][kBucketsOf + 1];
    const int buckets = 3 * (2 * a.reach + 1), x = threadIdx.x % kBucketsOf, run = threadIdx.x / kBucketsOf;
    const int i = blockIdx.x * kBucketsOf + x, head = blockIdx.y;
    float v = 0.f;
    if (i < buckets) {
#pragma unroll 8
        for (int k = run; k < a.n_tiles; k += kRunsOf) v += a.part[((int64_t)k * a.heads + head) * buckets + i];
    }
    s[run][x] = v;
    __syncthreads();
    for (int o = kRunsOf / 2; o > 0; o >>= 1) {
        if (run < o) s[run][x] += s[run + o][x];
        __syncthreads();
    }
    if (run == 0 && i < buckets) static_cast<uint16_t*>(a.dtable)[(int64_t)i * a.heads + head] = (uint16_t)from_f32<DT>(s[0][x]);
}

template <int DT, int DP, int EXT, bool A, class BQ, class BK>
hipError_t attention_backward_t(const AttentionArgs& a, hipStream_t s) {
    if (a.n_tiles > 0) {
        if (DT == kF16) launch(k_attention_range<DT, A>, grid_of(a.n_tiles64), dim3(256), 0, s, a);
        AttentionArgs b = a;
        b.heads_each = heads_a_block(a.n_tiles, a.heads, BQ::kHeads);
        launch(k_attention_queries<DT, DP, EXT, A, BQ>, attention_grid(a.n_tiles, a.heads, b.heads_each), dim3(BQ::kThreads), 0,
               s, b);
        if (BK::kRows == 64) {
            b.tiles = a.tiles64;
            b.n_tiles = a.n_tiles64;
        }
        b.heads_each = heads_a_block(b.n_tiles, a.kv_heads, BK::kHeads);
        launch(k_attention_keys<DT, DP, EXT, A, BK>, attention_grid(b.n_tiles, a.kv_heads, b.heads_each), dim3(BK::kThreads), 0,
               s, b);
    }
    if (EXT)
        launch(k_table_sum<DT>, dim3((unsigned)((3 * (2 * a.reach + 1) + kBucketsOf - 1) / kBucketsOf), (unsigned)a.heads), dim3(1024), 0, s, a);
    return hipGetLastError();
}

template <int DT, int DP, int EXT>
hipError_t attention_backward_by_length(const AttentionArgs& a, int lengths, hipStream_t s) {
    // (of 128 keys of 128 elements, two gradients do not fit the registers)
    typedef typename std::conditional<DP == 128, BlockMid, BlockLong>::type BlockKeys;
    if (lengths == kShortWindows) return attention_backward_t<DT, DP, EXT, true, BlockShort, BlockShort>(a, s);
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
