// What the kernels of window attention share: tiles of 64 rows in LDS, the bias as
// a matrix product, softmax over lanes.
//
// Products. Scores are computed transposed, S^T = K Q^T with 16 x 16 x 32 MFMAs: a lane
// holds four consecutive keys of one query, so what belongs to a query (maximum, sum,
// rescaling, log-sum-exp) is one value a lane, and two neighbouring 16-key results of a
// lane are, rounded, the operand of the next product as they stand: its contraction runs
// over the keys 16 a + 4 q + e, 16 (a + 1) + 4 q + e in that order (q: lane / 16, e < 4),
// and the other operand is read from LDS in the same order, four at a time, by transposing
// reads. Nothing is exchanged between lanes but row maxima and sums.
//
// Bias. bias_ij = sum over the axes of T[clamp(x_i - x_j, -R, R)] is a product too: B_i, the
// table seen from cell x_i (one entry for each cell x of the window's extent), times E_j, one-hot
// at x_j; the axes' cells lie side by side in the contraction. Table entries are exact in
// the rows' type, so the sum is float32's. The gradient of B is dS E, by the same tiles.
// (Looking entries up costs three LDS reads and nine vector operations a score, more than
// the rest of the softmax.) Infinities would make 0 x inf: they count as the type's
// largest values, whose exponentials are the same.
#pragma once

#include "mixing.h"
#include "row_words.h"

namespace smc {
namespace {

constexpr int kAttentionThreads = 256;
constexpr int kKeys = 64;               // rows of a tile in LDS
constexpr float kLog2e = 1.44269504088896340736f;

// A tile: rows of RW 16-byte words, permuted so that 8 rows read along, and 4 rows read by a
// transposing read (32 bytes each), lie in different banks.
template <int RW>
__device__ __forceinline__ int tile_word(int row, int word) {
    const int f = RW == 4 ? (row & 2) | ((row >> 2) & 1) : ((row & 3) << 1) | ((row >> 2) & 1);
    return (row * RW + (word ^ f)) * 16;
}
template <int RW>
__device__ __forceinline__ u32x4 tile_row(const char* tile, int row, int word) {
    return *reinterpret_cast<const u32x4*>(tile + tile_word<RW>(row, word));
}
// Columns 16 piece + lane % 16 of the rows r0 .. r0 + 3 and r1 .. r1 + 3 (the lane's own).
template <int RW>
__device__ __forceinline__ u32x4 tile_columns(const char* tile, int piece, int r0, int r1, int lane) {
    const int s = lane & 15;
    u32x2 v[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const char* p = tile + tile_word<RW>((t ? r1 : r0) + (s >> 2), 2 * piece + ((s >> 1) & 1)) + (s & 1) * 8;
        v[t] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SMC_LDS s16x4*)(p)));
    }
    return (u32x4){v[0].x, v[0].y, v[1].x, v[1].y};
}

// Elements i .. i + 7 of a row, zeros from `left` on.
__device__ __forceinline__ u32x4 row_word(const void* base, int64_t i, int left, int vec) {
    if (left <= 0) return (u32x4){0u, 0u, 0u, 0u};
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (vec) return *reinterpret_cast<const u32x4*>(p);
    return left >= W ? load_unaligned(p) : load_tail(p, left);
}

// One-hot row: word `word` of a row with a one at each of the three cells.
template <int DT>
__device__ __forceinline__ u32x4 one_hot(uint32_t cells, int word) {
    const uint64_t one = DT == kF16 ? 0x3c00 : 0x3f80;
    uint64_t lo = 0, hi = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const uint32_t r = ((cells >> (8 * d)) & 255u) - 8u * word;
        const uint64_t v = one << (16 * (r & 3));
        if (r < 4) lo |= v;
        if (r - 4 < 4) hi |= v;
    }
    return (u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// A head's table by distance: [axis][128 + distance], distances clamped to the reach.
constexpr int kDistances = 256;
template <int DT>
__device__ __forceinline__ void load_table(const AttentionArgs& a, int head, uint16_t* s_table) {
    const uint16_t* t = static_cast<const uint16_t*>(a.table);
    for (int i = threadIdx.x; i < 3 * kDistances; i += kAttentionThreads) {
        const int axis = i / kDistances, d = min(max(i % kDistances - 128, -a.reach), a.reach);
        uint16_t v = t[(int64_t)(axis * (2 * a.reach + 1) + a.reach + d) * a.heads + head];
        const uint16_t inf = DT == kF16 ? 0x7c00 : 0x7f80;
        if ((v & 0x7fff) == inf) v -= 1;
        s_table[i] = v;
    }
}

// Word of B: contraction elements i .. i + 7 of the table seen from `cells`. SIGN +1: entries
// T[own cell - cell], -1: T[cell - own cell].
template <int SIGN>
__device__ __forceinline__ u32x4 table_word(const AttentionArgs& a, const uint16_t* s_table, uint32_t cells, int i) {
    u32x4 w;
    const int y0 = a.extent[0], z0 = y0 + a.extent[1], end = z0 + a.extent[2];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t v = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = i + 2 * d + h, axis = (c >= y0) + (c >= z0);
            const int away = SIGN * ((int)((cells >> (8 * axis)) & 255u) - c);
            const uint32_t e = c < end ? s_table[axis * kDistances + 128 + away] : 0;
            v |= e << (16 * h);
        }
        w[d] = v;
    }
    return w;
}

// The block's tile and head: consecutive ones lie on one XCD, whose L2 then holds the other
// heads' columns of the rows that are read (blocks go round the 8 XCDs in turn).
__device__ __forceinline__ bool tile_and_head(int n_tiles, int heads, int& tile, int& head) {
    const uint32_t b = (uint32_t)block_number(), total = (uint32_t)n_tiles * (uint32_t)heads, each = (total + 7) / 8;
    const uint32_t i = (b & 7) * each + (b >> 3);
    if ((b >> 3) >= each || i >= total) return false;
    tile = (int)(i / (uint32_t)heads);
    head = (int)(i % (uint32_t)heads);
    return true;
}
inline dim3 attention_grid(int64_t n_tiles, int heads) { return grid_of((n_tiles * heads + 7) / 8 * 8); }

// v over the four lanes of a query.
__device__ __forceinline__ float quad_max(float v) {
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float quad_sum(float v) {
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// acc[d][e]: column 16 d + 4 q + e of the lane's row, times f, into the row at `to` of `dim` elements.
template <int DT, int DP>
__device__ __forceinline__ void store_row(const f32x4 (&acc)[DP / 16], float f, void* to, int64_t i, int dim, int lane, int vec) {
    const int q = lane >> 4;
#pragma unroll
    for (int d = 0; d < DP / 16; d += 2) {
        uint32_t l0 = pack2<DT>(acc[d][0] * f, acc[d][1] * f), l1 = pack2<DT>(acc[d][2] * f, acc[d][3] * f);
        uint32_t h0 = pack2<DT>(acc[d + 1][0] * f, acc[d + 1][1] * f), h1 = pack2<DT>(acc[d + 1][2] * f, acc[d + 1][3] * f);
        swap_rows(l0, h0);
        swap_rows(l1, h1);
        const u32x4 u = {l0, l1, h0, h1};
        const int c = 16 * (d + (q & 1)) + 8 * (q >> 1), left = dim - c;
        if (left <= 0 || i < 0) continue;
        uint16_t* p = static_cast<uint16_t*>(to) + i + c;
        if (vec) {
            *reinterpret_cast<u32x4*>(p) = u;
        } else if (left >= W) {
            store_unaligned(p, u);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e < left) p[e] = (uint16_t)(u[e >> 1] >> ((e & 1) * 16));
        }
    }
}

// Rows of a tile on their way from memory to LDS: 16-byte words, kLoads a thread, of the
// rows s_places[0 .. 63] (row < 0: zeros).
template <int RW>
struct RowLoads {
    static constexpr int kLoads = kKeys * RW / kAttentionThreads;
    u32x4 w[kLoads];
    __device__ __forceinline__ void load(const void* base, int64_t ld, int column, int dim, const WindowPlace* s_places, int vec) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * kAttentionThreads + threadIdx.x, r = id / RW, word = id % RW;
            const int row = s_places[r].row;
            w[i] = row_word(base, (int64_t)row * ld + column + word * W, row < 0 ? 0 : dim - word * W, vec);
        }
    }
    __device__ __forceinline__ void commit(char* tile) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * kAttentionThreads + threadIdx.x;
            *reinterpret_cast<u32x4*>(tile + tile_word<RW>(id / RW, id % RW)) = w[i];
        }
    }
};

// The one-hot rows of a tile (row < 0: zeros).
template <int DT, int RW>
__device__ __forceinline__ void commit_cells(char* tile, const WindowPlace* s_places) {
#pragma unroll
    for (int i = 0; i < kKeys * RW / kAttentionThreads; ++i) {
        const int id = i * kAttentionThreads + threadIdx.x, r = id / RW, word = id % RW;
        const WindowPlace p = s_places[r];
        const u32x4 none = {0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4*>(tile + tile_word<RW>(r, word)) = p.row < 0 ? none : one_hot<DT>(p.cells, word);
    }
}

// WindowPlace `at` of a tile's window, no row beyond its end.
__device__ __forceinline__ WindowPlace place_at(const AttentionArgs& a, int at, int end) {
    return at < end ? a.places[at] : WindowPlace{-1, 0u};
}

// Row and cells of a lane's own query or key.
__device__ __forceinline__ WindowPlace own_place(const AttentionArgs& a, const WindowTile& t, int i) {
    return i < t.count ? a.places[t.first + i] : WindowPlace{-1, 0u};
}

}  // namespace
}  // namespace smc
