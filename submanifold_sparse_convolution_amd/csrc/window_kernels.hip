// The index of windows that attention walks: for every place of the window order
// its row and cell, and the tiles of 32, 64 and 128 places, none of which has rows of
// two windows (so nothing of one window, not a NaN either, reaches another).
// Made once for all layers on the same windows.
#include <algorithm>

#include "mixing.h"

namespace smc {
namespace {

__device__ __forceinline__ WindowHeader* header_of(const WindowArgs& a) {
    return reinterpret_cast<WindowHeader*>(a.plan);
}

// Window w's first place; the places before the first window and after the last are
// windows -1 and `windows`. Offsets outside [0, n] are cut to it.
__device__ __forceinline__ int window_start(const WindowArgs& a, int64_t w) {
    if (w < 0) return 0;
    if (w > a.windows) return (int)a.n;
    return min(max(a.offsets[w], 0), (int)a.n);
}
__device__ __forceinline__ int window_end(const WindowArgs& a, int64_t w) {
    return max(window_start(a, w), window_start(a, w + 1));
}

__global__ __launch_bounds__(256) void k_windows_clear(WindowArgs a, uint32_t* seen, int64_t words) {
    const int64_t i = block_number() * 256 + threadIdx.x;
    if (i < words) seen[i] = 0;
    if (i == 0) *header_of(a) = WindowHeader{0, {0, 0, 0}, 0, 0};
}

// Rows of the places: within [0, n), none twice.
__global__ __launch_bounds__(256) void k_windows_rows(WindowArgs a, WindowPlace* places, uint32_t* seen) {
    const int64_t i = block_number() * 256 + threadIdx.x;
    if (i >= a.n) return;
    int row = a.order ? a.order[i] : (int)i;
    uint32_t status = 0;
    if (row < 0 || row >= a.n) {
        status = kStRange;
        row = (int)i;
    } else if (atomicOr(seen + (row >> 5), 1u << (row & 31)) >> (row & 31) & 1u) {
        status = kStDuplicate;
    }
    places[i] = WindowPlace{row, Cells(a.extent).lowest()};
    if (status) atomicOr(&header_of(a)->status, status);
}

// Cells of a window's rows, counted from its lowest; a block a window.
__global__ __launch_bounds__(256) void k_windows_cells(WindowArgs a, WindowPlace* places) {
    __shared__ int s_low[3][4];
    for (int64_t w = block_number(); w < a.windows; w += (int64_t)gridDim.x * gridDim.y) {
        const int begin = window_start(a, w), end = window_end(a, w);
        int low[3] = {INT_MAX, INT_MAX, INT_MAX};
        for (int i = begin + threadIdx.x; i < end; i += 256)
#pragma unroll
            for (int d = 0; d < 3; ++d) low[d] = min(low[d], a.coords[(int64_t)places[i].row * a.cols + a.cols - 3 + d]);
#pragma unroll
        for (int d = 0; d < 3; ++d)
            for (int o = 32; o > 0; o >>= 1) low[d] = min(low[d], __shfl_xor(low[d], o));
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            for (int d = 0; d < 3; ++d) s_low[d][threadIdx.x >> 6] = low[d];
        __syncthreads();
        uint32_t status = 0;
        for (int i = begin + threadIdx.x; i < end; i += 256) {
            uint32_t cells = 0;
            const Cells at(a.extent);
#pragma unroll
            for (int d = 0; d < 3; ++d) {
                const int lowest = min(min(s_low[d][0], s_low[d][1]), min(s_low[d][2], s_low[d][3]));
                // (a difference of any two coordinates fits 32 bits without a sign)
                uint32_t cell = (uint32_t)a.coords[(int64_t)places[i].row * a.cols + a.cols - 3 + d] - (uint32_t)lowest;
                if (cell >= (uint32_t)a.extent[d]) {
                    status = kStRange;
                    cell = 0;
                }
                cells |= (cell + at.first[d]) << (8 * d);
            }
            places[i].cells = cells;
        }
        if (status) atomicOr(&header_of(a)->status, status);
    }
}

// The tiles, window by window, by one block: counts of 1,024 windows at a time
// and their running sum. Offsets out of order are told by the way.
__global__ __launch_bounds__(1024) void k_windows_tiles(WindowArgs a, WindowTile* tiles32, WindowTile* tiles64,
                                                        WindowTile* tiles128) {
    __shared__ long long s_sum[3][1024];        // (offsets out of order could pass 32 bits)
    __shared__ int s_longest, s_bad;
    __shared__ unsigned long long s_pairs;
    if (threadIdx.x == 0) {
        s_longest = s_bad = 0;
        s_pairs = 0;
    }
    __syncthreads();
    int done[3] = {0, 0, 0};
    for (int64_t w0 = -1; w0 <= a.windows; w0 += 1024) {
        const int64_t w = w0 + threadIdx.x;
        int begin = 0, end = 0;
        if (w <= a.windows) {
            begin = window_start(a, w);
            end = window_end(a, w);
            if (w >= 0) {
                const int raw = a.offsets[w];
                if (raw != begin || (w < a.windows && a.offsets[w + 1] < raw)) atomicOr(&s_bad, 1);
                if (w < a.windows) {
                    atomicMax(&s_longest, end - begin);
                    atomicAdd(&s_pairs, (unsigned long long)(end - begin) * (unsigned long long)(end - begin));
                }
            }
        }
        int count[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int size = 32 << k;
            count[k] = (int)(((int64_t)end - begin + size - 1) / size);
            s_sum[k][threadIdx.x] = count[k];
        }
        __syncthreads();
        for (int o = 1; o < 1024; o <<= 1) {
            long long before[3] = {0, 0, 0};
            if (threadIdx.x >= o)
                for (int k = 0; k < 3; ++k) before[k] = s_sum[k][threadIdx.x - o];
            __syncthreads();
            for (int k = 0; k < 3; ++k) s_sum[k][threadIdx.x] += before[k];
            __syncthreads();
        }
        const bool inside = w >= 0 && w < a.windows;
        const int first64 = (int)min((int64_t)done[1] + s_sum[1][threadIdx.x] - count[1], a.n / 64 + a.windows + 1);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int size = 32 << k;
            // offsets out of order could make more tiles than there is room for
            const int64_t most = a.n / size + a.windows + 2;
            WindowTile* to = k == 0 ? tiles32 : k == 1 ? tiles64 : tiles128;
            int64_t at = (int64_t)done[k] + s_sum[k][threadIdx.x] - count[k];
            for (int i = 0; i < count[k] && at + i < most; ++i) {
                const int first = begin + i * size;
                to[at + i] = WindowTile{first, min(size, end - first), inside ? begin : 0, inside ? end : 0, first64, {0, 0, 0}};
            }
            done[k] = (int)min((int64_t)done[k] + s_sum[k][1023], most);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        WindowHeader* h = header_of(a);
        for (int k = 0; k < 3; ++k) h->tiles[k] = done[k];
        h->longest = s_longest;
        h->pairs = s_pairs;
        if (s_bad) atomicOr(&h->status, (uint32_t)kStRange);
    }
}

}  // namespace

hipError_t launch_windows(const WindowArgs& a, hipStream_t s) {
    const WindowLayout at(a.n, a.windows);
    WindowPlace* const places = reinterpret_cast<WindowPlace*>(a.plan + at.places);
    uint32_t* const seen = reinterpret_cast<uint32_t*>(a.plan + at.seen);
    const int64_t words = (a.n + 31) / 32;
    launch(k_windows_clear, grid_of(std::max<int64_t>(1, (words + 255) / 256)), dim3(256), 0, s, a, seen, words);
    if (a.n > 0) launch(k_windows_rows, grid_of((a.n + 255) / 256), dim3(256), 0, s, a, places, seen);
    if (a.n > 0 && a.coords && a.windows > 0)
        launch(k_windows_cells, dim3((unsigned)std::min<int64_t>(a.windows, 1 << 16)), dim3(256), 0, s, a, places);
    WindowTile* tiles[3];
    for (int k = 0; k < 3; ++k) tiles[k] = reinterpret_cast<WindowTile*>(a.plan + at.tiles[k]);
    launch(k_windows_tiles, dim3(1), dim3(1024), 0, s, a, tiles[0], tiles[1], tiles[2]);
    return hipGetLastError();
}

}  // namespace smc
