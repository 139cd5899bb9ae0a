// Internal declarations of the operators that mix rows: group norm over the rows
// of a sample and attention inside windows of rows. The C entries are in
// mixing_api.hip.
#pragma once

#include "pointwise.h"

namespace smc {

// ---- group norm (group_norm_kernels.hip) ----
struct GroupArgs {
    int64_t n = 0;
    int c = 0, groups = 0, samples = 0;
    int act = 0;
    float eps = 0.f;
    const int* offsets = nullptr;   // [samples + 1] or null: every row is of the one sample
    const void* x = nullptr;
    int64_t ldx = 0;
    const void* weight = nullptr;
    const void* bias = nullptr;
    void* y = nullptr;              // backward: dx
    int64_t ldy = 0;
    float* stats = nullptr;         // [samples][groups][2]: mean, 1 / sqrt(var + eps)
    const void* dy = nullptr;
    int64_t lddy = 0;
    void* dweight = nullptr;
    void* dbias = nullptr;
    // by group_plan
    int rows_each = 1;              // rows of a piece
    int pieces = 0;                 // see Piece
    bool whole = false;             // forward: one launch
    float* by_group = nullptr;      // [pieces][groups][2]
    float* by_channel = nullptr;    // backward: [pieces][2][c]
    int vec = 0;                    // 16-byte loads and stores are possible
};
constexpr int kMaxGroupChannels = 8192;         // a block's threads hold a row
constexpr int kMaxGroupsOfNorm = 4096;         // their statistics lie in LDS
constexpr int kMaxSamples = 1 << 16;
void group_plan(GroupArgs& a);                  // rows_each and pieces, from n, c, samples and offsets
hipError_t launch_group_norm(const GroupArgs& a, int dt, hipStream_t s);
hipError_t launch_group_norm_backward(const GroupArgs& a, int dt, hipStream_t s);

// ---- windows (window_kernels.hip) ----
// A place is a position in the window order. Header, places and tiles of 32, 64 and 128
// places lie behind each other in the plan.
struct WindowPlace {
    int row;            // row of the tensors
    uint32_t cells;     // of the row in its window, x, y and z as elements of Cells, 8 bits each
};
// The axes' cells side by side, each axis at a multiple of 4.
struct Cells {
    int up[3], first[3];        // elements of an axis, the first of them
    __host__ __device__ explicit Cells(const int (&extent)[3]) {
        int at = 0;
        for (int d = 0; d < 3; ++d) {
            up[d] = (extent[d] + 3) & ~3;
            first[d] = at;
            at += up[d];
        }
    }
    __host__ __device__ int all() const { return first[2] + up[2]; }
    // twice as many entries by distance (see TableLoads)
    __host__ __device__ int axis_of_entry(int i) const { return (i >= 2 * first[1]) + (i >= 2 * first[2]); }
    __host__ __device__ static int pick(const int (&v)[3], int axis) { return axis == 0 ? v[0] : axis == 1 ? v[1] : v[2]; }
    __host__ __device__ uint32_t lowest() const { return (uint32_t)first[1] << 8 | (uint32_t)first[2] << 16; }
};
struct WindowTile {
    int first, count;   // places
    int begin, end;     // of the window; equal: the rows are in no window
    int first64;        // the window's first tile of 64 places
    int unused[3];
};
struct WindowHeader {
    uint32_t status;    // kSt* bits
    int tiles[3];       // of 32, 64 and 128 places
    int longest;        // rows of the longest window
    unsigned long long pairs;   // sum of the squares of the windows' rows
};
constexpr int kMaxCells = 128;                  // elements of Cells
constexpr int kMaxReach = 127;                  // cells lie no further apart
constexpr int64_t kMaxWindows = 1 << 24;
struct WindowLayout {
    size_t places, tiles[3], seen, bytes;       // offsets; seen: a bit a row, scratch of the build
    WindowLayout(int64_t n, int64_t windows) {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        places = 256;
        size_t at = places + up((size_t)n * sizeof(WindowPlace));
        for (int k = 0; k < 3; ++k) {
            tiles[k] = at;
            at += up((size_t)(n / (32 << k) + windows + 2) * sizeof(WindowTile));
        }
        seen = at;
        bytes = seen + up((size_t)(n + 31) / 32 * 4);
    }
};
struct WindowArgs {
    int64_t n = 0, windows = 0;
    const int* offsets = nullptr;   // [windows + 1]
    const int* order = nullptr;     // [n] or null
    const int* coords = nullptr;    // [n, cols] or null, x, y, z last
    int cols = 0;
    int extent[3] = {0, 0, 0};
    char* plan = nullptr;
};
hipError_t launch_windows(const WindowArgs& a, hipStream_t s);

// ---- window attention (attention_*.hip) ----
struct AttentionArgs {
    int64_t n = 0;
    int heads = 0, kv_heads = 0, dim = 0;
    int heads_each = 1;             // of a block
    float scale = 0.f;
    const void *q = nullptr, *k = nullptr, *v = nullptr;
    int64_t ldq = 0, ldk = 0, ldv = 0;
    const WindowPlace* places = nullptr;
    const WindowTile* tiles = nullptr;
    int n_tiles = 0;
    int extent[3] = {0, 0, 0};
    const void* table = nullptr;    // [3][2 reach + 1][heads] or null
    int reach = 0;
    void* out = nullptr;            // backward: read
    int64_t ldo = 0;
    float* lse = nullptr;           // [heads][n] by place; forward: or null
    const void* dout = nullptr;
    int64_t ld_dout = 0;
    void *dq = nullptr, *dk = nullptr, *dv = nullptr;
    int64_t ld_dq = 0, ld_dk = 0, ld_dv = 0;
    void* dtable = nullptr;
    float* delta = nullptr;         // [heads][n] by place: sums of dout out
    float* part = nullptr;          // [tiles][heads][3 (2 reach + 1)] sums of dS
    float* range = nullptr;         // f16: [tiles of 64][heads + kv_heads] largest |dout| and |v|
    const WindowTile* tiles64 = nullptr;
    int n_tiles64 = 0;
    int vec = 0;                    // every row is made of aligned 16-byte words
};
// By the windows' mean length, which a launch's blocks fit; the tiles are of 32, 64 and 128 places.
enum : int { kShortWindows = 0, kMidWindows = 1, kLongWindows = 2 };
hipError_t launch_attention_bf16(const AttentionArgs& a, int lengths, hipStream_t s);
hipError_t launch_attention_f16(const AttentionArgs& a, int lengths, hipStream_t s);
hipError_t launch_attention_backward_bf16(const AttentionArgs& a, int lengths, hipStream_t s);
hipError_t launch_attention_backward_f16(const AttentionArgs& a, int lengths, hipStream_t s);

}  // namespace smc
