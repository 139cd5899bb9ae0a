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
// at x_j; the axes' cells lie side by side in the contraction, each axis at a multiple of 4. Table entries are exact in
// the rows' type, so the sum is float32's. The gradient of B is dS E, by the same tiles.
// (Looking entries up costs three LDS reads and nine vector operations a score, more than
// the rest of the softmax.) Infinities would make 0 x inf: they count as the type's
// largest values, whose exponentials are the same.
#pragma once

#include "mixing.h"
#include "row_words.h"

namespace smc {
namespace {

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

// Elements i .. i + 7 of a row, zeros from `left` on (ALIGNED: all of them or none, and no
// branch that a load would be waited for at).
template <bool ALIGNED>
__device__ __forceinline__ u32x4 row_word(const void* base, int64_t i, int left) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (ALIGNED) {
        if (left > 0) w = *reinterpret_cast<const u32x4*>(p);
    } else if (left > 0) {
        w = left >= W ? load_unaligned(p) : load_tail(p, left);
    }
    return w;
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

// A head's table by distance, 2 `up` entries for an axis of `up` elements (see Cells): entry m is
// T[up - m], or T[m - up] where MIRROR, clamped to the reach. The entries lie twice, the second
// time one further, so that two neighbouring ones are an aligned word whatever the first.
template <int EXT>
constexpr int kTableEntries = 2 * EXT + 2;      // of one copy
template <int DT, int EXT, int THREADS, bool MIRROR>
__device__ __forceinline__ void load_table(const AttentionArgs& a, int head, uint16_t* s_table) {
    const uint16_t* t = static_cast<const uint16_t*>(a.table);
    const Cells cells(a.extent);
#pragma unroll
    for (int k = 0; k < (2 * EXT + THREADS - 1) / THREADS; ++k) {
        const int i = k * THREADS + threadIdx.x, axis = cells.axis_of_entry(i);
        if (i >= 2 * cells.all()) continue;
        const int away = cells.pick(cells.up, axis) - (i - 2 * cells.pick(cells.first, axis));
        const int d = min(max(MIRROR ? -away : away, -a.reach), a.reach);
        uint16_t v = t[(int64_t)(axis * (2 * a.reach + 1) + a.reach + d) * a.heads + head];
        const uint16_t inf = DT == kF16 ? 0x7c00 : 0x7f80;
        if ((v & 0x7fff) == inf) v -= 1;
        s_table[i] = v;
        s_table[kTableEntries<EXT> + i + 1] = v;
    }
}

// The table seen from the cells `own`: elements 32 c + 8 q .. + 7 of the contraction, each chunk c.
// Element e of axis d is entry 2 first + up - own + e; four elements lie on one axis.
template <int EXT>
__device__ __forceinline__ void table_words(const AttentionArgs& a, const uint16_t* s_table, uint32_t own, int q,
                                            u32x4 (&w)[EXT ? EXT / 32 : 1]) {
    const Cells cells(a.extent);
    int at[3];                  // bytes from the table's start to element 0
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int m = 2 * cells.first[d] + cells.up[d] - (int)((own >> (8 * d)) & 255u);
        at[d] = 2 * m + ((m & 1) ? 2 * kTableEntries<EXT> + 2 : 0);
    }
    const char* table = reinterpret_cast<const char*>(s_table);
#pragma unroll
    for (int c = 0; c < EXT / 32; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = 32 * c + 8 * q + 4 * h;
            const bool in = e < cells.all();
            const int from = (e < cells.first[1] ? at[0] : e < cells.first[2] ? at[1] : at[2]) + 2 * e;
            const uint32_t lo = *reinterpret_cast<const uint32_t*>(table + (in ? from : 0));
            const uint32_t hi = *reinterpret_cast<const uint32_t*>(table + (in ? from + 4 : 0));
            w[c][2 * h] = in ? lo : 0u;
            w[c][2 * h + 1] = in ? hi : 0u;
        }
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

__device__ __forceinline__ bool any_lane(bool v) { return __ballot(v) != 0; }

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// acc[d][e]: column 16 d + 4 q + e of the lane's row, times f, into the row at `to` of `dim` elements.
template <int DT, int DP, bool ALIGNED>
__device__ __forceinline__ void store_row(const f32x4 (&acc)[DP / 16], float f, void* to, int64_t i, int dim, int lane) {
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
        if (ALIGNED) {
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
template <int RW, int THREADS, bool ALIGNED>
struct RowLoads {
    static constexpr int kLoads = kKeys * RW / THREADS;
    u32x4 w[kLoads];
    __device__ __forceinline__ void load(const void* base, int64_t ld, int column, int dim, const WindowPlace* s_places) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + threadIdx.x, r = id / RW, word = id % RW;
            const int row = s_places[r].row;
            w[i] = row_word<ALIGNED>(base, (int64_t)row * ld + column + word * W, row < 0 ? 0 : dim - word * W);
        }
    }
    __device__ __forceinline__ void commit(char* tile) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + threadIdx.x;
            *reinterpret_cast<u32x4*>(tile + tile_word<RW>(id / RW, id % RW)) = w[i];
        }
    }
};

// The one-hot rows of a tile (row < 0: zeros).
template <int DT, int RW, int THREADS>
__device__ __forceinline__ void commit_cells(char* tile, const WindowPlace* s_places) {
#pragma unroll
    for (int i = 0; i < kKeys * RW / THREADS; ++i) {
        const int id = i * THREADS + threadIdx.x, r = id / RW, word = id % RW;
        const WindowPlace p = s_places[r];
        const u32x4 none = {0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4*>(tile + tile_word<RW>(r, word)) = p.row < 0 ? none : one_hot<DT>(p.cells, word);
    }
}

// Waves and columns a wave of a block. Short windows: 32 queries by one wave (a block's latency is
// what they cost, and smaller blocks leave fewer waves without queries); long ones: 128, so that
// what is read from LDS serves two columns.
template <int WAVES_, int COLUMNS_>
struct Block {
    static constexpr int kWaves = WAVES_, kColumns = COLUMNS_, kThreads = 64 * WAVES_;
    static constexpr int kRows = 16 * WAVES_ * COLUMNS_;        // queries (or keys)
    static constexpr bool kSkips = WAVES_ <= 2;                 // 16 keys past a window's end are left out
};
template <int DP>
using BlockShort = Block<DP <= 64 ? 1 : 2, DP <= 64 ? 2 : 1>;
typedef Block<4, 1> BlockMid;
typedef Block<4, 2> BlockLong;

// Place `at` of a tile's window, no row beyond its end.
__device__ __forceinline__ WindowPlace place_at(const AttentionArgs& a, int at, int end) {
    return at < end ? a.places[at] : WindowPlace{-1, 0u};
}

// Two tiles of a window's rows (keys and values, or queries and dout) and their one-hot cells, 64 rows
// a step: a step's rows are loaded while the one before is worked on, and go to LDS after it, with two
// buffers without waiting for the other waves' reads of it.
template <int DT, int DP, int EXT, bool A, class B, int NB>
struct Walk {
    static constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, TH = B::kThreads;
    struct Memory {
        char x[NB][kKeys * DP * 2], y[NB][kKeys * DP * 2], e[NB][EXT ? kKeys * EXT * 2 : 16];
        WindowPlace places[2][kKeys];
    };
    RowLoads<RW, TH, A> lx, ly;
    WindowPlace next;
    // The first step's loads. (Every thread calls these.)
    __device__ __forceinline__ void start(const AttentionArgs& a, Memory& m, const WindowTile& t, const void* x, int64_t ldx,
                                          const void* y, int64_t ldy, int column) {
        const int i = threadIdx.x & (kKeys - 1);
        if (threadIdx.x < kKeys) m.places[0][i] = place_at(a, t.begin + i, t.end);
        if (TH == kKeys || (threadIdx.x >= kKeys && threadIdx.x < 2 * kKeys)) m.places[1][i] = place_at(a, t.begin + kKeys + i, t.end);
        next = place_at(a, t.begin + 2 * kKeys + i, t.end);
        __syncthreads();
        load(a, m, 0, x, ldx, y, ldy, column);
    }
    __device__ __forceinline__ void load(const AttentionArgs& a, const Memory& m, int step, const void* x, int64_t ldx,
                                         const void* y, int64_t ldy, int column) {
        lx.load(x, ldx, column, a.dim, m.places[step & 1]);
        ly.load(y, ldy, column, a.dim, m.places[step & 1]);
    }
    // The loaded step to LDS; `step` is its number.
    __device__ __forceinline__ void commit(const AttentionArgs& a, Memory& m, int step, const WindowTile& t) {
        const int buf = NB == 2 ? step & 1 : 0;
        if (NB == 1) __syncthreads();
        lx.commit(m.x[buf]);
        ly.commit(m.y[buf]);
        if (EXT) commit_cells<DT, RE, TH>(m.e[buf], m.places[step & 1]);
        if (step > 0) {
            const int i = threadIdx.x & (kKeys - 1);
            if (threadIdx.x < kKeys) m.places[(step + 1) & 1][i] = next;        // of the step before
            next = place_at(a, t.begin + (step + 2) * kKeys + i, t.end);
        }
        __syncthreads();
    }
};

// Row and cells of a lane's own query or key (the lowest cells where there is none).
__device__ __forceinline__ WindowPlace own_place(const AttentionArgs& a, const WindowTile& t, int i) {
    return i < t.count ? a.places[t.first + i] : WindowPlace{-1, Cells(a.extent).lowest()};
}

}  // namespace
}  // namespace smc
