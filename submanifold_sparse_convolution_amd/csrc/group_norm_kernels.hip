// Group norm of rows, channels last, with an activation, and its gradients.
//
//   mean, var over the rows of a sample and the channels of a group
//   x_hat = (x - mean) rstd, rstd = 1 / sqrt(var + eps), z = x_hat w + b, y = act(z)
//
//   dz = dy act'(z), a = dz w
//   dx = rstd (a - mean(a) - x_hat mean(a x_hat)), dw = sum of dz x_hat, db = sum of dz
//
// Two passes over the rows, one kernel each: sums of pieces, then outputs, whose
// blocks add up the pieces of their sample first (a kernel between the two for that would
// cost its launch). x (and dy) are read twice, the second time largely from the caches.
//
// 91,000 x 128 bf16 in six samples: 10.8 us of sums and 13.2 of outputs, 22.4 us a call (70 MB:
// 9.1 at the rate of a large copy, x counted once); backward, 95,000 x 128 in two: 15.0 and 18.3,
// 32.5 a call. A thread's rows are few there (192 x 16 words on 512 threads: 6), and what bounds
// the kernels is latency: the loads', the tree's over a block's rows, the joining of pieces.
// Without gain: six rows of a thread fetched before the pieces are joined (23.1 us); columns
// summed by a thread each in place of the tree (25.7 for 24.2).
//
// Variances do not suffer from large means, nor from rows far off: a thread keeps the mean of its rows so
// far and the sum of squared deviations from it (as Welford, of differences from the piece's first row,
// which keep the mean's digits), and threads, channels and pieces are joined by theirs (as Chan, Golub and
// LeVeque). (Sums of the differences and of their squares, whose parts from that row to the mean are taken off
// at the end, lose digits where it lies far off: 1,000,000 rows of mean 1,000 and spread 1 behind a row of zeros
// 6 % of the variance; so 10^-7.)
#include <algorithm>

#include "mixing.h"
#include "row_words.h"

namespace smc {
namespace {

// Threads of a block: a row is held by one, 8 channels a thread.
constexpr int kThreads = 512, kThreadsWide = 1024;
static_assert(kMaxGroupChannels == kThreadsWide * W, "a row is held by a block");

// ---- pieces --------------------------------------------------------------------
// The rows are cut at every multiple of `rows_each` and at the samples' borders.
// Runs: the rows before the first sample, each sample, the rows after the last
// (without offsets, one run). Piece number = run + multiples passed: it grows
// with the rows, run r owns the numbers from begin / rows_each + r on, one at least, and
// what a piece holds follows from the offsets alone, however uneven they are.

struct Piece {
    int run;            // 0: before the samples, samples + 1: after them
    int begin, end;     // rows
    int run_begin, run_end;
};

// Offsets outside [0, n] or out of order make wrong, but valid, row ranges.
__device__ __forceinline__ int run_start(const GroupArgs& a, int run) {
    if (run <= 0) return 0;
    if (run > a.samples + 1) return (int)a.n;
    return min(max(a.offsets[run - 1], 0), (int)a.n);
}

__device__ __forceinline__ int multiples(const GroupArgs& a, int row) {
    return (int)((uint32_t)row / (uint32_t)a.rows_each);
}

__device__ __forceinline__ Piece piece_of(const GroupArgs& a, int number) {
    Piece p;
    if (!a.offsets) {
        p.run = 1;
        p.run_begin = 0;
        p.run_end = (int)a.n;
        p.begin = (int)min((int64_t)number * a.rows_each, a.n);
        p.end = (int)min((int64_t)(number + 1) * a.rows_each, a.n);
        return p;
    }
    // the last run that owns a number up to this one
    int run = -1;
    const int lane = threadIdx.x & 63;
    for (int r0 = 0; r0 < a.samples + 2; r0 += 64) {
        const int r = r0 + lane;
        const bool in = r < a.samples + 2 && multiples(a, run_start(a, r)) + r <= number;
        run += __popcll(__ballot(in));
    }
    run = __builtin_amdgcn_readfirstlane(max(run, 0));
    p.run = run;
    p.run_begin = run_start(a, run);
    p.run_end = max(p.run_begin, run_start(a, run + 1));
    const int64_t cut = (int64_t)max(number - run, 0) * a.rows_each;
    p.begin = (int)min(max((int64_t)p.run_begin, cut), (int64_t)p.run_end);
    p.end = (int)max((int64_t)p.begin, min((int64_t)p.run_end, cut + a.rows_each));
    return p;
}

// First number of a run, and of the run's last row.
__device__ __forceinline__ int first_piece(const GroupArgs& a, const Piece& p) {
    return multiples(a, p.run_begin) + (a.offsets ? p.run : 0);
}
__device__ __forceinline__ int last_piece(const GroupArgs& a, const Piece& p) {
    const int row = max(p.run_begin, p.run_end - 1);
    return multiples(a, row) + (a.offsets ? p.run : 0);
}
__device__ __forceinline__ bool is_sample(const GroupArgs& a, const Piece& p) {
    return !a.offsets || (p.run >= 1 && p.run <= a.samples);
}

// ---- sums over a block ------------------------------------------------------------

// How a block's threads lie over rows of c channels.
template <int T>
struct Lay {
    int words, rows, word, row;
    bool ok;
    __device__ explicit Lay(int c) {
        words = (c + W - 1) / W;
        rows = T / words;
        row = threadIdx.x / words;
        word = threadIdx.x - row * words;
        ok = row < rows;
    }
};

// The threads' values added over the rows of the block: in row 0 of them at the end. Halves are
// joined in a fixed order. s: N x T / 2 floats.
template <int T, int N>
__device__ __forceinline__ void sum_rows(float (&v)[N], const Lay<T>& l, float* s) {
    for (int rows = l.rows; rows > 1;) {
        const int half = (rows + 1) >> 1;
        __syncthreads();
        if (l.row >= half && l.row < rows)
#pragma unroll
            for (int e = 0; e < N; ++e) s[e * (T / 2) + (l.row - half) * l.words + l.word] = v[e];
        __syncthreads();
        if (l.row + half < rows)
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += s[e * (T / 2) + l.row * l.words + l.word];
        rows = half;
    }
    __syncthreads();
}

// Floats of dynamic LDS: join_rows of 2 W + 1 values, or two values a channel.
template <int T>
__host__ __device__ inline int sum_floats(int c) { return std::max((2 * W + 1) * T / 2, 2 * c); }

// ---- forward -------------------------------------------------------------------------

// `rows` values' mean and sum of squared deviations, `times` values a row.
struct Moments {
    float rows, mean, m2;
    // with those of other rows (times: values a row); a NaN or infinity in either stays
    __device__ __forceinline__ void join(const Moments& o, float times) {
        const float all = rows + o.rows, share = o.rows * __builtin_amdgcn_rcpf(fmaxf(all, 1.f)), d = o.mean - mean;
        m2 += o.m2 + d * (d * (rows * share * times));
        mean += d * share;
        rows = all;
    }
};

// The threads' means and sums of squared deviations joined over the rows of the block: in row 0 of them at the
// end, as sum_rows. s: (2 W + 1) T / 2 floats.
template <int T>
__device__ __forceinline__ void join_rows(float& rows, float (&mean)[W], float (&m2)[W], const Lay<T>& l, float* s) {
    for (int left = l.rows; left > 1;) {
        const int half = (left + 1) >> 1;
        __syncthreads();
        if (l.row >= half && l.row < left) {
            float* to = s + (l.row - half) * l.words + l.word;
            to[W * T] = rows;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                to[e * (T / 2)] = mean[e];
                to[(W + e) * (T / 2)] = m2[e];
            }
        }
        __syncthreads();
        if (l.row + half < left) {
            const float* from = s + l.row * l.words + l.word;
            const float other = from[W * T], share = other * __builtin_amdgcn_rcpf(fmaxf(rows + other, 1.f)), weight = rows * share;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float d = from[e * (T / 2)] - mean[e];
                m2[e] += from[(W + e) * (T / 2)] + d * (d * weight);
                mean[e] += d * share;
            }
            rows += other;
        }
        left = half;
    }
    __syncthreads();
}

// Mean and sum of squared deviations of each group over a piece's rows, into out [groups][2] (memory or LDS).
template <int DT, bool A, int T>
__device__ __forceinline__ void piece_sums(const GroupArgs& a, const Piece& p, const Lay<T>& l, float* s, float* out) {
    const int c = l.word * W, left = a.c - c;
    float base[W], mean[W], m2[W], count = 0.f;
#pragma unroll
    for (int e = 0; e < W; ++e) base[e] = mean[e] = m2[e] = 0.f;
    if (l.ok) {
        load_f32<DT, A>(a.x, (int64_t)p.begin * a.ldx + c, left, base);
#pragma unroll 4
        for (int r = p.begin + l.row; r < p.end; r += l.rows) {
            float v[W];
            load_f32<DT, A>(a.x, (int64_t)r * a.ldx + c, left, v);
            count += 1.f;
            const float share = __builtin_amdgcn_rcpf(count);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float d = v[e] - base[e], off = d - mean[e];
                mean[e] += off * share;
                m2[e] += off * (d - mean[e]);
            }
        }
    }
    join_rows<T>(count, mean, m2, l, s);
    const float rows = (float)(p.end - p.begin);
    float* const s_squares = s + a.c;
    if (l.ok && l.row == 0)
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < left) {
                s[c + e] = base[e] + mean[e];
                s_squares[c + e] = m2[e];
            }
    __syncthreads();
    const int per = a.c / a.groups, lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < a.groups; g += T / 64) {
        const float* mean_of = s + g * per;
        const float* squares_of = s_squares + g * per;
        const float first = mean_of[0];
        float m = 0.f;
        for (int k = lane; k < per; k += 64) m += mean_of[k] - first;
        const float mean = first + lane_sum<64>(m) / (float)per;
        float m2 = 0.f;
        for (int k = lane; k < per; k += 64) {
            const float d = mean_of[k] - mean;
            m2 += squares_of[k] + rows * (d * d);
        }
        m2 = lane_sum<64>(m2);
        if (lane == 0) {
            out[2 * g] = mean;
            out[2 * g + 1] = m2;
        }
    }
}

template <int DT, bool A, int T>
__global__ __launch_bounds__(T) void k_group_sums(GroupArgs a) {
    extern __shared__ float s[];
    const int number = (int)blockIdx.x;
    const Piece p = piece_of(a, number);
    if (!is_sample(a, p) || p.begin >= p.end) return;
    piece_sums<DT, A>(a, p, Lay<T>(a.c), s, a.by_group + (int64_t)number * a.groups * 2);
}

// Mean and rstd of each group of a piece's sample, from its pieces, into s_stats
// [groups][2]. s: 2 T floats.
template <int T>
__device__ void join_pieces(const GroupArgs& a, const Piece& p, float* s, float* s_stats) {
    const int first = first_piece(a, p), count = p.run_end > p.run_begin ? last_piece(a, p) - first + 1 : 0;
    const int cuts = multiples(a, p.run_begin);
    const float per = (float)(a.c / a.groups);
    for (int g0 = 0; g0 < a.groups; g0 += T) {
        const int wide = min(a.groups - g0, T);
        const int parts = T / wide, part = threadIdx.x / wide, g = threadIdx.x - part * wide;
        Moments m = {0.f, 0.f, 0.f};            // (means from the first piece's)
        float base = 0.f;
        if (part < parts && count > 0) {
            const float* from = a.by_group + ((int64_t)first * a.groups + g0 + g) * 2;
            base = from[0];
#pragma unroll 4
            for (int k = part; k < count; k += parts) {
                // rows of the piece: the run's, from one multiple to the next
                const int64_t cut = (int64_t)(cuts + k) * a.rows_each;
                const float rows = (float)(min((int64_t)p.run_end, cut + a.rows_each) -
                                           max((int64_t)p.run_begin, cut));
                m.join({rows, from[(int64_t)k * a.groups * 2] - base, from[(int64_t)k * a.groups * 2 + 1]}, per);
            }
        }
        int rows = min(parts, max(count, 1));
        while (rows > 1) {
            const int half = (rows + 1) >> 1;
            __syncthreads();
            if (part >= half && part < rows) {
                float* to = s + (part - half) * wide + g;
                to[0] = m.rows;
                to[T / 2] = m.mean;
                to[T] = m.m2;
            }
            __syncthreads();
            if (part + half < rows) {
                const float* from = s + part * wide + g;
                m.join({from[0], from[T / 2], from[T]}, per);
            }
            rows = half;
        }
        if (part == 0) {
            s_stats[(g0 + g) * 2] = base + m.mean;
            s_stats[(g0 + g) * 2 + 1] = count > 0 ? inverse_root(m.m2 / ((float)(p.run_end - p.run_begin) * per) + a.eps) : 0.f;
        }
        __syncthreads();
    }
}

template <int DT, bool A, int ACT, int T>
__device__ __forceinline__ void write_rows(const GroupArgs& a, const Piece& p, const Lay<T>& l, const float* s_stats) {
    if (!l.ok) return;
    const int c = l.word * W, left = a.c - c, per = a.c / a.groups;
    float mean[W], scale[W], shift[W];
    load_f32<DT, A>(a.weight, c, left, scale);
    load_f32<DT, A>(a.bias, c, left, shift);
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const int g = (A || e < left ? c + e : c) / per;
        mean[e] = s_stats[2 * g];
        scale[e] *= s_stats[2 * g + 1];
    }
#pragma unroll 4
    for (int r = p.begin + l.row; r < p.end; r += l.rows) {
        float v[W];
        load_f32<DT, A>(a.x, (int64_t)r * a.ldx + c, left, v);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = act_value<ACT>((v[e] - mean[e]) * scale[e] + shift[e]);
        store_16<DT, A>(a.y, (int64_t)r * a.ldy + c, left, v);
    }
}

template <int DT, bool A, int T>
__device__ __forceinline__ void write_zeros(const GroupArgs& a, const Piece& p, const Lay<T>& l) {
    if (!l.ok) return;
    const float v[W] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int r = p.begin + l.row; r < p.end; r += l.rows)
        store_16<DT, A>(a.y, (int64_t)r * a.ldy + l.word * W, a.c - l.word * W, v);
}

template <int DT, bool A, int T>
__global__ __launch_bounds__(T) void k_group_write(GroupArgs a) {
    extern __shared__ float s[];
    const int number = (int)blockIdx.x;
    const Piece p = piece_of(a, number);
    const Lay<T> l(a.c);
    if (!is_sample(a, p)) return write_zeros<DT, A, T>(a, p, l);
    float* const s_stats = s + 2 * T;
    join_pieces<T>(a, p, s, s_stats);
    if (a.stats && number == first_piece(a, p)) {
        float* o = a.stats + (int64_t)(a.offsets ? p.run - 1 : 0) * a.groups * 2;
        for (int i = threadIdx.x; i < 2 * a.groups; i += T) o[i] = s_stats[i];
    }
    with_act(a.act, [&](auto act) SMC_INLINE { write_rows<DT, A, decltype(act)::value, T>(a, p, l, s_stats); });
}

// The whole of a small norm: a block for each run.
template <int DT, bool A, int T>
__global__ __launch_bounds__(T) void k_group_whole(GroupArgs a) {
    extern __shared__ float s[];
    Piece p;
    p.run = a.offsets ? (int)blockIdx.x : 1;
    p.begin = p.run_begin = a.offsets ? run_start(a, p.run) : 0;
    p.end = p.run_end = a.offsets ? max(p.begin, run_start(a, p.run + 1)) : (int)a.n;
    const Lay<T> l(a.c);
    if (!is_sample(a, p)) return write_zeros<DT, A, T>(a, p, l);
    float* const s_stats = s + sum_floats<T>(a.c);
    if (p.begin < p.end) piece_sums<DT, A>(a, p, l, s, s_stats);
    __syncthreads();
    const float n = (float)(p.end - p.begin) * (float)(a.c / a.groups);
    for (int g = threadIdx.x; g < a.groups; g += T) {
        const float mean = p.begin < p.end ? s_stats[2 * g] : 0.f;
        const float rstd = p.begin < p.end ? inverse_root(s_stats[2 * g + 1] / n + a.eps) : 0.f;
        s_stats[2 * g] = mean;
        s_stats[2 * g + 1] = rstd;
        if (a.stats) {
            float* o = a.stats + ((int64_t)(p.run - 1) * a.groups + g) * 2;
            o[0] = mean;
            o[1] = rstd;
        }
    }
    __syncthreads();
    with_act(a.act, [&](auto act) SMC_INLINE { write_rows<DT, A, decltype(act)::value, T>(a, p, l, s_stats); });
}

// ---- backward ----------------------------------------------------------------------

// What a thread needs of its channels.
struct Channels {
    float w[W], b[W], mean[W], rstd[W];
    template <int DT, bool A>
    __device__ __forceinline__ void load(const GroupArgs& a, const Piece& p, int c, int left) {
        load_f32<DT, A>(a.weight, c, left, w);
        load_f32<DT, A>(a.bias, c, left, b);
        const float* stats = a.stats + (int64_t)(a.offsets ? p.run - 1 : 0) * a.groups * 2;
        const int per = a.c / a.groups;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const int g = (A || e < left ? c + e : c) / per;
            mean[e] = stats[2 * g];
            rstd[e] = stats[2 * g + 1];
        }
    }
};

// x_hat and dz of an element. The same bits in both passes, and in gradient_rows a - mean(a) is
// exactly zero in a sample of one element: no fused multiply-adds.
template <int ACT>
__device__ __forceinline__ void slope_of(float v, float dy, const Channels& ch, int e, float& xh, float& dz) {
#pragma clang fp contract(off)
    xh = (v - ch.mean[e]) * ch.rstd[e];
    dz = dy * act_slope<ACT>(xh * ch.w[e] + ch.b[e]);
}

// A piece's sums of dz and dz x_hat, each channel; and of a and a x_hat, each group.
template <int DT, bool A, int ACT, int T>
__device__ __forceinline__ void gradient_sums(const GroupArgs& a, const Piece& p, const Lay<T>& l, float (&sum)[2 * W]) {
    const int c = l.word * W, left = a.c - c;
    Channels ch;
    ch.load<DT, A>(a, p, c, left);
#pragma unroll 2
    for (int r = p.begin + l.row; r < p.end; r += l.rows) {
        float v[W], dy[W];
        load_f32<DT, A>(a.x, (int64_t)r * a.ldx + c, left, v);
        load_f32<DT, A>(a.dy, (int64_t)r * a.lddy + c, left, dy);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            float xh, dz;
            slope_of<ACT>(v[e], dy[e], ch, e, xh, dz);
            sum[e] += dz;
            sum[W + e] += dz * xh;
        }
    }
}

template <int DT, bool A, int T>
__global__ __launch_bounds__(T) void k_group_gradient_sums(GroupArgs a) {
    extern __shared__ float s[];
    const int number = (int)blockIdx.x;
    const Piece p = piece_of(a, number);
    const Lay<T> l(a.c);
    const int c = l.word * W, left = a.c - c;
    float sum[2 * W];
#pragma unroll
    for (int e = 0; e < 2 * W; ++e) sum[e] = 0.f;
    if (l.ok && is_sample(a, p) && p.begin < p.end)
        with_act(a.act, [&](auto act) SMC_INLINE { gradient_sums<DT, A, decltype(act)::value, T>(a, p, l, sum); });
    sum_rows<T>(sum, l, s);
    if (l.ok && l.row == 0)
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < left) {
                s[c + e] = sum[e];
                s[a.c + c + e] = sum[W + e];
            }
    __syncthreads();
    float* o = a.by_channel + (int64_t)number * 2 * a.c;
    for (int i = threadIdx.x; i < 2 * a.c; i += T) o[i] = s[i];
    const int per = a.c / a.groups, lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < a.groups; g += T / 64) {
        float m1 = 0.f, m2 = 0.f;
        for (int k = lane; k < per; k += 64) {
            const float w = to_f32<DT>(static_cast<const uint16_t*>(a.weight)[g * per + k]);
            m1 += w * s[g * per + k];
            m2 += w * s[a.c + g * per + k];
        }
        m1 = lane_sum<64>(m1);
        m2 = lane_sum<64>(m2);
        if (lane == 0) {
            a.by_group[((int64_t)number * a.groups + g) * 2] = m1;
            a.by_group[((int64_t)number * a.groups + g) * 2 + 1] = m2;
        }
    }
}

// The means of a and a x_hat over a piece's sample, each group.
template <int T>
__device__ void join_gradient_pieces(const GroupArgs& a, const Piece& p, float* s, float* s_means) {
    const int first = first_piece(a, p), count = p.run_end > p.run_begin ? last_piece(a, p) - first + 1 : 0;
    for (int g0 = 0; g0 < a.groups; g0 += T) {
        const int wide = min(a.groups - g0, T);
        const int parts = T / wide, part = threadIdx.x / wide, g = threadIdx.x - part * wide;
        float v[2] = {0.f, 0.f};
        if (part < parts) {
            const float* from = a.by_group + ((int64_t)first * a.groups + g0 + g) * 2;
#pragma unroll 4
            for (int k = part; k < count; k += parts) {
                v[0] += from[(int64_t)k * a.groups * 2];
                v[1] += from[(int64_t)k * a.groups * 2 + 1];
            }
        }
        int rows = min(parts, max(count, 1));
        while (rows > 1) {
            const int half = (rows + 1) >> 1;
            __syncthreads();
            if (part >= half && part < rows) {
                s[(part - half) * wide + g] = v[0];
                s[T + (part - half) * wide + g] = v[1];
            }
            __syncthreads();
            if (part + half < rows) {
                v[0] += s[part * wide + g];
                v[1] += s[T + part * wide + g];
            }
            rows = half;
        }
        if (part == 0) {
            const float n = (float)max(p.run_end - p.run_begin, 1) * (float)(a.c / a.groups);
            s_means[(g0 + g) * 2] = v[0] / n;
            s_means[(g0 + g) * 2 + 1] = v[1] / n;
        }
        __syncthreads();
    }
}

template <int DT, bool A, int ACT, int T>
__device__ __forceinline__ void gradient_rows(const GroupArgs& a, const Piece& p, const Lay<T>& l, const float* s_means) {
#pragma clang fp contract(off)
    if (!l.ok) return;
    const int c = l.word * W, left = a.c - c, per = a.c / a.groups;
    Channels ch;
    ch.load<DT, A>(a, p, c, left);
    float m1[W], m2[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const int g = (A || e < left ? c + e : c) / per;
        m1[e] = s_means[2 * g];
        m2[e] = s_means[2 * g + 1];
    }
#pragma unroll 2
    for (int r = p.begin + l.row; r < p.end; r += l.rows) {
        float v[W], dy[W];
        load_f32<DT, A>(a.x, (int64_t)r * a.ldx + c, left, v);
        load_f32<DT, A>(a.dy, (int64_t)r * a.lddy + c, left, dy);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            float xh, dz;
            slope_of<ACT>(v[e], dy[e], ch, e, xh, dz);
            v[e] = ch.rstd[e] * ((dz * ch.w[e] - m1[e]) - xh * m2[e]);
        }
        store_16<DT, A>(a.y, (int64_t)r * a.ldy + c, left, v);
    }
}

// dw and db of 8 channels: every piece's sums, in T / 16 strided runs joined by a tree.
template <int DT, int T>
__device__ __forceinline__ void sum_channels(const GroupArgs& a, int block, float* s) {
    const int x = threadIdx.x & 15, run = threadIdx.x >> 4;        // 8 channels of db, then of dw
    const int c = block * 8 + (x & 7);
    float v = 0.f;
    if (c < a.c) {
        const float* from = a.by_channel + (x >> 3) * a.c + c;
#pragma unroll 8
        for (int k = run; k < a.pieces; k += T / 16) v += from[(int64_t)k * 2 * a.c];
    }
    s[run * 17 + x] = v;
    __syncthreads();
    for (int o = T / 32; o > 0; o >>= 1) {
        if (run < o) s[run * 17 + x] += s[(run + o) * 17 + x];
        __syncthreads();
    }
    if (run == 0 && c < a.c) static_cast<uint16_t*>(x >> 3 ? a.dweight : a.dbias)[c] = (uint16_t)from_f32<DT>(s[x]);
}

// dx of a piece; the blocks after the pieces' add up dw and db.
template <int DT, bool A, int T>
__global__ __launch_bounds__(T) void k_group_gradient_write(GroupArgs a) {
    extern __shared__ float s[];
    const int number = (int)blockIdx.x;
    if (number >= a.pieces) return sum_channels<DT, T>(a, number - a.pieces, s);
    const Piece p = piece_of(a, number);
    const Lay<T> l(a.c);
    if (!is_sample(a, p)) return write_zeros<DT, A, T>(a, p, l);
    if (p.begin >= p.end) return;
    float* const s_means = s + 2 * T;
    join_gradient_pieces<T>(a, p, s, s_means);
    with_act(a.act, [&](auto act) SMC_INLINE { gradient_rows<DT, A, decltype(act)::value, T>(a, p, l, s_means); });
}

template <int DT, bool A, int T>
void group_norm_t(const GroupArgs& a, hipStream_t s) {
    if (a.whole)
        return launch(k_group_whole<DT, A, T>, dim3((unsigned)(a.offsets ? a.samples + 2 : 1)), dim3(T),
                      (size_t)(sum_floats<T>(a.c) + 2 * a.groups) * 4, s, a);
    launch(k_group_sums<DT, A, T>, dim3((unsigned)a.pieces), dim3(T), (size_t)sum_floats<T>(a.c) * 4, s, a);
    launch(k_group_write<DT, A, T>, dim3((unsigned)a.pieces), dim3(T), (2 * T + 2 * (size_t)a.groups) * 4, s, a);
}

template <int DT, bool A, int T>
void group_norm_backward_t(const GroupArgs& a, hipStream_t s) {
    launch(k_group_gradient_sums<DT, A, T>, dim3((unsigned)a.pieces), dim3(T), (size_t)sum_floats<T>(a.c) * 4, s, a);
    launch(k_group_gradient_write<DT, A, T>, dim3((unsigned)(a.pieces + (a.c + 7) / 8)), dim3(T),
           (2 * T + 2 * (size_t)a.groups) * 4, s, a);
}

template <int DT>
hipError_t group_norm_of(const GroupArgs& a, bool backward, hipStream_t s) {
    const bool wide = a.c > kThreads * W;
#define SMC_GO(A, T) backward ? group_norm_backward_t<DT, A, T>(a, s) : group_norm_t<DT, A, T>(a, s)
    if (a.vec) wide ? (SMC_GO(true, kThreadsWide)) : (SMC_GO(true, kThreads));
    else wide ? (SMC_GO(false, kThreadsWide)) : (SMC_GO(false, kThreads));
#undef SMC_GO
    return hipGetLastError();
}

}  // namespace

// Rows of a piece: two pieces a compute unit, but no fewer rows than give each thread 4 words; the same in both passes.
// (One or four pieces a compute unit: 40,000 x 512 in four samples 30.2 or 40.6 us for 30.5, its backward 49.7 or 53.7
// for 46.1; 91,000 x 128 in one sample 23.0 or 30.5 for 25.3, its backward 34.9 or 37.3 for 32.1.) Whole steps of a
// block: 91,000 x 128 in six samples 22.4 us for 25.3.
//
// One launch up to 4 words a thread: a single row 12.0 us a call for 14.6; the rows of 64 words a
// thread would take 43 for 14.7, one block's loads waiting for each other.
void group_plan(GroupArgs& a) {
    const int64_t words = (a.c + W - 1) / W, blocks = 2 * (int64_t)device_cus();
    a.rows_each = (int)std::max<int64_t>((a.n + blocks - 1) / blocks, std::max<int64_t>(1, 4 * kThreads / words));
    const int64_t step = std::max<int64_t>(1, kThreads / words);
    a.rows_each = (int)((a.rows_each + step - 1) / step * step);
    a.pieces = (int)((a.n + a.rows_each - 1) / a.rows_each);
    if (a.offsets) a.pieces += a.samples + 2;
    a.pieces = std::max(a.pieces, 1);
    a.whole = a.n * words <= (int64_t)4 * kThreads;
}

hipError_t launch_group_norm(const GroupArgs& a, int dt, hipStream_t s) {
    return dt == kF16 ? group_norm_of<kF16>(a, false, s) : group_norm_of<kBF16>(a, false, s);
}

hipError_t launch_group_norm_backward(const GroupArgs& a, int dt, hipStream_t s) {
    return dt == kF16 ? group_norm_of<kF16>(a, true, s) : group_norm_of<kBF16>(a, true, s);
}

}  // namespace smc
