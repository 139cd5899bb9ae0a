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
    int rows_log = 0;               // rows of a piece (log2)
    int pieces = 0;                 // see k_group_sums
    float* by_group = nullptr;      // [pieces][groups][2]
    float* by_channel = nullptr;    // backward: [pieces][2][c]
    int vec = 0;                    // 16-byte loads and stores are possible
};
constexpr int kMaxGroupChannels = 8192;         // a block's threads hold a row
constexpr int kMaxGroupsOfNorm = 4096;         // their statistics lie in LDS
constexpr int kMaxSamples = 1 << 16;
void group_plan(GroupArgs& a);                  // rows_log and pieces, from n, c, samples and offsets
hipError_t launch_group_norm(const GroupArgs& a, int dt, hipStream_t s);
hipError_t launch_group_norm_backward(const GroupArgs& a, int dt, hipStream_t s);

}  // namespace smc
