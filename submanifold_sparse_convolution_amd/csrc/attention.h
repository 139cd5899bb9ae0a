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
// the rest of the softmax.) Entries count as at most 2^14 in size: infinities
// would make 0 x inf, and where a mask of such entries leaves a row nothing, log sum exp of
// far larger scores would lose the sum, and the gradients' probabilities with it (at 3 2^14 a
// float's step is 2^-8). Scores below the largest by that much have no share either way.
#pragma once

#include <algorithm>

#include "mixing.h"
#include "row_words.h"

namespace smc {
namespace {

// for loads and stores through pointers that are picked by a condition, which the compiler else takes for
// pointers to any memory
#define SMC_GLOBAL __attribute__((address_space(1)))

constexpr int kKeys = 64;               // rows of a tile in LDS
constexpr float kLog2e = 1.44269504088896340736f;

// A tile: rows of RW 16-byte words, 32-byte pieces of a row permuted by its number so that what is read at
// a time lies in different banks of the 64 (256 bytes): by 16-byte reads, lanes 0 .. 3, 12 .. 15 of one word
// and 4 .. 11 of the next (or the other way round), each lane a row; by transposing reads, 8 rows' pieces.
template <int RW>
__device__ __forceinline__ int tile_word(int row, int word) {
    const int f = RW == 16 ? row & 7 : RW == 8 ? (row >> 1) & 3 : (row >> 2) & 1;
    return (row * RW + (word ^ (2 * f))) * 16;
}
// A lane's places in a tile, which do not depend on the step: word 4 c + lane / 16 of the row lane % 16 (rows
// 16 b + that are a constant further), and its 8 bytes of a transposing read of the columns 16 piece ..
// + 15 of the rows 4 (lane / 16) .. + 3.
template <int RW>
struct TileLane {
    int row[(RW + 3) / 4], column[RW / 2];
    __device__ __forceinline__ explicit TileLane(int lane) {
#pragma unroll
        for (int c = 0; c < RW / 4; ++c) row[c] = tile_word<RW>(lane & 15, 4 * c + (lane >> 4));
#pragma unroll
        for (int d = 0; d < RW / 2; ++d)
            column[d] = tile_word<RW>(4 * (lane >> 4) + ((lane & 15) >> 2), 2 * d + ((lane >> 1) & 1)) + (lane & 1) * 8;
    }
    __device__ __forceinline__ u32x4 along(const char* tile, int row16, int c) const {
        return *reinterpret_cast<const u32x4*>(tile + row[c] + row16 * (RW * 16));
    }
    // (rows r .. of the lanes' first four, and 16 further)
    __device__ __forceinline__ u32x4 across(const char* tile, int piece, int r) const {
        const char* p = tile + column[piece] + r * (RW * 16);
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SMC_LDS s16x4*)(p)));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SMC_LDS s16x4*)(p + 16 * RW * 16)));
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
    }
};

// Elements i .. i + 7 of a row, zeros from `left` on (ALIGNED: all of them or none, and no
// branch that a load would be waited for at).
template <bool ALIGNED>
__device__ __forceinline__ u32x4 row_word(const void* base, int64_t i, int left) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (ALIGNED) {
        if (left > 0) w = *(const SMC_GLOBAL u32x4*)(p);
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
struct TableLoads {
    static constexpr int kLoads = EXT ? (2 * EXT + THREADS - 1) / THREADS : 1;
    uint16_t v[kLoads];
    __device__ __forceinline__ void load(const AttentionArgs& a, int head) {
        const uint16_t* t = static_cast<const uint16_t*>(a.table);
        const Cells cells(a.extent);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int i = k * THREADS + threadIdx.x, axis = cells.axis_of_entry(i);
            const int away = cells.pick(cells.up, axis) - (i - 2 * cells.pick(cells.first, axis));
            const int d = min(max(MIRROR ? -away : away, -a.reach), a.reach);
            v[k] = 0;
            if (i < 2 * cells.all()) v[k] = t[(int64_t)(axis * (2 * a.reach + 1) + a.reach + d) * a.heads + head];
        }
    }
    __device__ __forceinline__ void commit(const AttentionArgs& a, uint16_t* s_table) const {
        const uint16_t inf = DT == kF16 ? 0x7c00 : 0x7f80, most = DT == kF16 ? 0x7400 : 0x4680;    // 2^14
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int i = k * THREADS + threadIdx.x;
            if (i >= 2 * EXT) continue;
            const uint16_t size = v[k] & 0x7fff;
            const uint16_t e = size > most && size <= inf ? (v[k] & 0x8000) | most : v[k];
            s_table[i] = e;
            s_table[kTableEntries<EXT> + i + 1] = e;
        }
    }
};

// The tables of up to HEADS heads, every load before the first is waited for.
template <int DT, int EXT, int THREADS, int HEADS>
__device__ __forceinline__ void load_tables(const AttentionArgs& a, int head, int heads,
                                            uint16_t (&s_table)[HEADS][EXT ? 2 * kTableEntries<EXT> : 2]) {
    TableLoads<DT, EXT, THREADS, false> t[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
        if (h < heads) t[h].load(a, head + h);
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
        if (h < heads) t[h].commit(a, s_table[h]);
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

// The block's tile and heads, `each` of them from `head` on: consecutive blocks lie on one XCD, whose L2
// then holds the other heads' columns of the rows that are read (blocks go round the 8 XCDs in turn).
__device__ __forceinline__ bool tile_and_head(int n_tiles, int heads, int each, int& tile, int& head) {
    const uint32_t groups = (uint32_t)(heads + each - 1) / (uint32_t)each;
    const uint32_t b = (uint32_t)block_number(), total = (uint32_t)n_tiles * groups, an_xcd = (total + 7) / 8;
    const uint32_t i = (b & 7) * an_xcd + (b >> 3);
    if ((b >> 3) >= an_xcd || i >= total) return false;
    tile = (int)(i / groups);
    head = (int)(i % groups) * each;
    return true;
}
inline dim3 attention_grid(int64_t n_tiles, int heads, int each) {
    return grid_of((n_tiles * ((heads + each - 1) / each) + 7) / 8 * 8);
}

// Heads a block: two where one would make more than 16 blocks a CU. Forward / backward in us, one, two and
// four: 91,000 rows, 14,208 blocks 53.6, 47.3, 50.1 / 200.8, 187.6, 200.0; 40,000 in windows of 24, 6,668
// 20.3, 17.2, 17.0 / 85.1, 80.4, 81.7; of 60, 2,668 13.7, 15.2, 15.2 / 47.2, 51.2, 48.9.
inline int heads_a_block(int64_t n_tiles, int heads, int most) {
    return n_tiles * heads >= 16 * device_cus() ? std::min(heads, most) : 1;
}

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
            *(SMC_GLOBAL u32x4*)(p) = u;
        } else if (left >= W) {
            store_unaligned(p, u);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e < left) p[e] = (uint16_t)(u[e >> 1] >> ((e & 1) * 16));
        }
    }
}

// Waves, columns a wave and heads a block. Short windows: 32 queries and several heads, so that what
// does not depend on the head (places, cells, addresses), half of the work, is done once, and the
// next head's rows are on their way while one is worked on; long ones: 128 queries, so that what is
// read from LDS serves two columns.
template <int WAVES_, int COLUMNS_, int HEADS_>
struct Block {
    static constexpr int kWaves = WAVES_, kColumns = COLUMNS_, kThreads = 64 * WAVES_;
    static constexpr int kRows = 16 * WAVES_ * COLUMNS_;        // queries (or keys)
    static constexpr int kHeads = HEADS_;                       // at most
    static constexpr bool kSkips = WAVES_ <= 2;                 // 16 keys past a window's end are left out
    static constexpr bool kHalves = COLUMNS_ == 1;              // 32 keys at a time, none past a window's end
};
typedef Block<2, 1, 2> BlockShort;
typedef Block<4, 1, 2> BlockMid;
typedef Block<4, 2, 1> BlockLong;

// Place `at` of a tile's window, no row beyond its end (and cells that are none).
__device__ __forceinline__ WindowPlace place_at(const AttentionArgs& a, int at, int end) {
    WindowPlace p = {-1, 0xffffffffu};
    if (at < end) p = a.places[at];
    return p;
}

// Two tiles of a window's rows (keys and values, or queries and dout) and their one-hot cells, 64 rows
// a step: a step's rows are loaded while the one before is worked on, and go to LDS after it, with two
// buffers without waiting for the other waves' reads of it. Places past the window's end are zeros; where REPEATS
// the first tile has the window's last row there, so that its products with infinities are no others than the window's.
template <int DT, int DP, int EXT, bool A, class B, int NB, bool REPEATS = false>
struct Walk {
    static constexpr int RW = DP / 8, RE = EXT ? EXT / 8 : 4, TH = B::kThreads;
    static constexpr int kWords = kKeys * RW / TH, kCells = EXT ? kKeys * RE / TH : 1;      // a thread's
    struct Memory {
        char x[NB][kKeys * DP * 2], y[NB][kKeys * DP * 2], e[NB][EXT ? kKeys * EXT * 2 : 16];
    };
    u32x4 wx[kWords], wy[kWords];
    const char *px, *py;        // this thread's word of row 0, of the head whose rows are loaded
    int rows[kWords];           // of the step to load; negative past the end (REPEATS: ~ of the last row)
    uint32_t cells[kCells], held[kCells];       // of that step, and of the step loaded
    bool whole;                 // the step to load has 64 rows, of DP elements

    __device__ static int word() { return (int)threadIdx.x % RW * W; }
    __device__ __forceinline__ void point(const void* x, const void* y, int column) {
        px = static_cast<const char*>(x) + 2 * (int64_t)(column + word());
        py = static_cast<const char*>(y) + 2 * (int64_t)(column + word());
    }
    __device__ __forceinline__ void places(const AttentionArgs& a, const WindowTile& t, int step) {
        const int first = t.begin + step * kKeys;
        whole = A && first + kKeys <= t.end && a.dim == DP;
        if (whole) {
            const SMC_GLOBAL WindowPlace* p = (const SMC_GLOBAL WindowPlace*)a.places + first;
#pragma unroll
            for (int i = 0; i < kWords; ++i) rows[i] = p[(i * TH + (int)threadIdx.x) / RW].row;
            if (EXT)
#pragma unroll
                for (int i = 0; i < kCells; ++i) cells[i] = p[(i * TH + (int)threadIdx.x) / RE].cells;
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int at = first + (i * TH + (int)threadIdx.x) / RW;
            if (REPEATS) {
                const int row = a.places[max(min(at, t.end - 1), 0)].row;
                rows[i] = at < t.end ? row : ~row;
            } else {
                rows[i] = place_at(a, at, t.end).row;
            }
        }
        if (EXT)
#pragma unroll
            for (int i = 0; i < kCells; ++i) cells[i] = place_at(a, first + (i * TH + (int)threadIdx.x) / RE, t.end).cells;
    }
    __device__ __forceinline__ void load(const AttentionArgs& a, int64_t ldx, int64_t ldy) {
        const uint32_t bx = (uint32_t)ldx * 2, by = (uint32_t)ldy * 2;
        if (whole) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                wx[i] = *(const SMC_GLOBAL u32x4*)(px + (uint64_t)(uint32_t)rows[i] * bx);
                wy[i] = *(const SMC_GLOBAL u32x4*)(py + (uint64_t)(uint32_t)rows[i] * by);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int left = rows[i] < 0 ? 0 : a.dim - word();
                const int x = REPEATS && rows[i] < 0 ? ~rows[i] : rows[i];
                wx[i] = row_word<A>(px + (uint64_t)(uint32_t)x * bx, 0, REPEATS ? a.dim - word() : left);
                wy[i] = row_word<A>(py + (uint64_t)(uint32_t)rows[i] * by, 0, left);
            }
        }
        if (EXT)
#pragma unroll
            for (int i = 0; i < kCells; ++i) held[i] = cells[i];
    }
    // The loaded step to LDS.
    __device__ __forceinline__ void commit(Memory& m, int buf, bool with_cells) {
        if (NB == 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int id = i * TH + threadIdx.x, at = tile_word<RW>(id / RW, id % RW);
            *reinterpret_cast<u32x4*>(m.x[buf] + at) = wx[i];
            *reinterpret_cast<u32x4*>(m.y[buf] + at) = wy[i];
        }
        if (EXT && with_cells)
#pragma unroll
            for (int i = 0; i < kCells; ++i) {
                const int id = i * TH + threadIdx.x;
                *reinterpret_cast<u32x4*>(m.e[buf] + tile_word<RE>(id / RE, id % RE)) = one_hot<DT>(held[i], id % RE);
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
