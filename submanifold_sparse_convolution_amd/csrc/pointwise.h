// Internal declarations of the row operators (RMS norm, linear and gated
// layers): the operands their kernels take and the host functions that launch
// them. The C entries are in pointwise_api.hip.
#pragma once

#include "smc_internal.h"

namespace smc {

// Element types (the C interface's SMC_DTYPE_* values).
enum Dtype : int { kBF16 = 0, kF16 = 1, kE4M3 = 2 };
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// What a product kernel does with its float32 accumulators.
enum Epilogue : int {
    kEpiStore = 0,      // y = act(z + bias) + residual
    kEpiGated = 1,      // h = act(z_gate + bias) * (z_up + bias)
    kEpiSlope = 2,      // dz = dy act'(z + bias)
    kEpiGatedSlope = 3, // dz_gate = dh u act'(g), dz_up = dh act(g)
    kEpiPartial = 4,    // the float32 sums of one range of the contraction
};

// How an operand lies in memory, seen from the product: its contraction index
// is the contiguous one (kAlongK: rows of x, or W^T), or the other one is
// (kAcrossK: W itself as [k, n], or both operands of x^T dz).
enum Layout : int { kAlongK = 0, kAcrossK = 1 };

// out[m, n] = sum over k of a(m, k) b(n, k), then the epilogue.
struct ProductArgs {
    const void* a = nullptr;    // rows of the output
    const void* b = nullptr;    // columns of the output
    int64_t lda = 0, ldb = 0;   // elements from one memory row to the next
    int m = 0, k = 0;
    int n = 0;                  // columns of b (gated: both halves)
    int half = 0;               // gated: columns of one half of b
    int half_out = 0;           // gated: columns of out and of a half of the bias (0: half)
    const void* bias = nullptr; // [n]
    const float* a_scale = nullptr;   // e4m3: one a row of a, of b
    const float* b_scale = nullptr;
    const void* extra = nullptr;      // residual, dy or dh: [m, n] ([m, half] gated)
    int64_t ld_extra = 0;
    int extra_width = 0;        // columns of extra (0: as many as out)
    void* out = nullptr;        // [m, n] ([m, half] for kEpiGated)
    int64_t ldo = 0;
    float* part = nullptr;      // kEpiPartial: [splits][m + colsum][n]
    int k_split = 0;            // contraction length of a split (all of k: one split; none is empty)
    int splits = 1;
    int colsum = 0;             // kEpiPartial: row m of a split's sums is the sum of b over k
    // f16 slopes, whose rows are written times a power of two (see range_scale):
    float* dz_max = nullptr;          // one a block, the largest finite |dz|: written by the first
                                      // launch, read by the second, which
    float* dz_unscale = nullptr;      // writes the inverse scale here (null: the first launch)
    const float* unscale = nullptr;   // f16 input gradient: its sums are multiplied by this
    int act = 0;
    int vec_a = 0, vec_b = 0;   // 16-byte loads are possible
    int vec_x = 0;              // a row of extra has a whole 16-byte word
    // the tile walk
    int tiles_m = 0, tiles_n = 0;
    int group_log = 0;          // row tiles walked together (log2)
    int xcds = 8;
};

// The grid of `blocks` blocks of 256 threads. A dimension's threads are counted in
// 32 bits (beyond them the launch succeeds with the blocks that are left), so many
// blocks lie in two dimensions; block_number() tells them apart, the last few of
// them past `blocks`.
constexpr int kGridLog = 23;
inline dim3 grid_of(int64_t blocks) {
    const int64_t most = 1 << kGridLog;
    return dim3((unsigned)(blocks < most ? blocks : most), (unsigned)((blocks + most - 1) >> kGridLog));
}
__device__ __forceinline__ int64_t block_number() { return ((int64_t)blockIdx.y << kGridLog) + blockIdx.x; }

// Compute units of the current device (looked up once per device).
int device_cus();

// out = product (see ProductArgs); dt: type of out, bias and extra, and of a
// and b unless e4m3 (whose b lies along k or across it). Fills in the tile walk.
constexpr int kMaxBlocksPerCu = 3;      // blocks of a product kernel, at most, for each CU
constexpr int kFewRows = 16;    // forward 16-bit products of up to as many rows may take a kernel of their own
bool few_rows_pay(const ProductArgs& p, Epilogue epi);      // (kEpiStore or kEpiGated, 16-bit operands)
hipError_t launch_forward(ProductArgs p, Epilogue epi, int dt, bool e4m3, bool w_along, hipStream_t s);
// dx = dz W^T: both operands along k.
hipError_t launch_input_gradient(ProductArgs p, int dt, hipStream_t s);
// dW = x^T dz (both operands across k) and, with colsum, db: float32 sums of
// `splits` ranges of k_split rows, added and rounded by launch_sum_parts.
int weight_gradient_range(int64_t rows, int c_in, int n);      // rows of a range (0 for no rows)
hipError_t launch_weight_gradient(ProductArgs p, int dt, hipStream_t s);
// The sums have n = halves half_p columns; column c < c_out of half h goes to
// column h c_out + c of dw (and db).
struct SumArgs {
    const float* part = nullptr;
    int splits = 0;
    int64_t m = 0;              // rows of dw
    int n = 0, half_p = 0, c_out = 0;
    void* dw = nullptr;
    int64_t ldw = 0;
    void* db = nullptr;         // or null
    const float* unscale = nullptr;     // factor of the sums (or null)
};
hipError_t launch_sum_parts(const SumArgs& a, int dt, hipStream_t s);
// dst [rows_p, ldd] = src [rows, halves c] with each half at a multiple of half_p
// columns, zeros elsewhere; rows of dst are whole 16-byte words. esize: bytes an
// element (1 or 2).
hipError_t launch_pad_rows(int esize, const void* src, int64_t lds, int64_t rows, int halves, int c, void* dst,
                           int64_t ldd, int64_t rows_p, int half_p, hipStream_t s);

// ---- norm (norm_kernels.hip) ----
struct NormArgs {
    int64_t n = 0;
    int c = 0;
    float eps = 0.f;
    const void* x = nullptr;        // backward: s, the rows that were normalised
    int64_t ldx = 0;
    const void* residual = nullptr; // backward: the gradient that reaches s by other paths
    int64_t ldr = 0;
    const void* weight = nullptr;
    void* y = nullptr;              // backward: dx
    int64_t ldy = 0;
    void* s = nullptr;
    int64_t lds = 0;
    float* y_scale = nullptr;       // e4m3 output
    const void* dy = nullptr;
    int64_t lddy = 0;
    void* dweight = nullptr;
    float* part = nullptr;          // backward: [blocks][c] sums of dy x_hat
    int vec = 0;                    // 16-byte loads and stores are possible
};
hipError_t launch_norm(const NormArgs& a, int dt, hipStream_t s);
int norm_backward_blocks(int64_t n, int c);
hipError_t launch_norm_backward(const NormArgs& a, int dt, hipStream_t s);
hipError_t launch_quantize_weight(const void* w, int64_t ldw, int c_in, int c_out, void* q,
                                  int64_t ldq, float* scale, int dt, hipStream_t s);

}  // namespace smc
