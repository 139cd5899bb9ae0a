// C entries of the operators that mix rows: argument checks, scratch layout and
// launches. See include/smconv.h for the contract of each call.
#include "api_checks.h"
#include "mixing.h"

using namespace smc;

namespace {

bool odd(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

// Arguments that may not share memory.
struct Rows {
    const char* name;
    const void* p;
    int64_t ld, cols;
};
struct Vector {
    const char* name;
    const void* p;
    size_t bytes;
};
int apart(const Vector& v, const Rows& r, int64_t n) {
    return over_rows(v.p, v.bytes, r.p, r.ld, n, r.cols) ? bad(SMC_ERR_ARG, "%s shares memory with %s", v.name, r.name) : SMC_OK;
}
int apart(const Vector& v, const Vector& w) {
    return over_bytes(v.p, v.bytes, w.p, w.bytes) ? bad(SMC_ERR_ARG, "%s shares memory with %s", v.name, w.name) : SMC_OK;
}

// ---- group norm --------------------------------------------------------------------

int check_group(const smc_group_norm_t* a, bool backward) {
    if (!a) return bad(SMC_ERR_ARG, "args is NULL");
    CHECK(check_common(a->n, a->c, "c", a->dtype));
    if (a->groups < 1 || a->c % a->groups) return bad(SMC_ERR_ARG, "%d channels in %d groups", a->c, a->groups);
    if (a->c > kMaxGroupChannels || a->groups > kMaxGroupsOfNorm)
        return bad(SMC_ERR_UNSUPPORTED, "%d channels in %d groups, more than %d or %d", a->c, a->groups,
                   kMaxGroupChannels, kMaxGroupsOfNorm);
    if (a->samples < 1 || (!a->offsets && a->samples != 1))
        return bad(SMC_ERR_ARG, "samples = %d%s", a->samples, a->offsets ? "" : " without offsets");
    if (a->samples > kMaxSamples) return bad(SMC_ERR_UNSUPPORTED, "%d samples, more than %d", a->samples, kMaxSamples);
    if (odd(a->offsets, 4)) return bad(SMC_ERR_ARG, "offsets is not aligned to its elements");
    if (a->activation < SMC_ACT_NONE || a->activation > SMC_ACT_GELU)
        return bad(SMC_ERR_ARG, "activation %d", a->activation);
    if (!(a->eps >= 0.f)) return bad(SMC_ERR_ARG, "eps = %g", (double)a->eps);
    if (!a->weight || odd(a->weight, 2)) return bad(SMC_ERR_ARG, "weight is NULL or misaligned");
    if (!a->bias || odd(a->bias, 2)) return bad(SMC_ERR_ARG, "bias is NULL or misaligned");
    if (odd(a->stats, 4)) return bad(SMC_ERR_ARG, "stats is not aligned to its elements");
    CHECK(check_rows("x", a->x, a->n, a->c, a->ldx));
    // an output row is written by the threads that have read that row, and by no others
    auto over = [&](const void* p, int64_t ldp, const void* q, int64_t ldq) {
        return (p != q || ldp != ldq) && share_memory(p, ldp, 2, q, ldq, 2, a->n, a->c, a->c);
    };
    // and some blocks write theirs while others still read the vectors and statistics
    const size_t row = (size_t)a->c * 2, kept = (size_t)a->samples * a->groups * 8;
    const Vector in[] = {{"weight", a->weight, row}, {"bias", a->bias, row}, {"offsets", a->offsets, ((size_t)a->samples + 1) * 4}};
    const Vector stats = {"stats", a->stats, kept};
    if (!backward) {
        CHECK(check_rows("y", a->y, a->n, a->c, a->ldy));
        if (over(a->y, a->ldy, a->x, a->ldx)) return bad(SMC_ERR_ARG, "y shares memory with x");
        const Rows x = {"x", a->x, a->ldx, a->c}, y = {"y", a->y, a->ldy, a->c};
        for (const Vector& v : in) {
            CHECK(apart(v, y, a->n));
            CHECK(apart(stats, v));
        }
        CHECK(apart(stats, x, a->n));
        return apart(stats, y, a->n);
    }
    if (!a->stats) return bad(SMC_ERR_ARG, "stats is NULL");
    CHECK(check_rows("dy", a->dy, a->n, a->c, a->ld_dy));
    CHECK(check_rows("dx", a->dx, a->n, a->c, a->ld_dx));
    if (!a->dweight || odd(a->dweight, 2)) return bad(SMC_ERR_ARG, "dweight is NULL or misaligned");
    if (!a->dbias || odd(a->dbias, 2)) return bad(SMC_ERR_ARG, "dbias is NULL or misaligned");
    if (over(a->dx, a->ld_dx, a->x, a->ldx)) return bad(SMC_ERR_ARG, "dx shares memory with x");
    if (over(a->dx, a->ld_dx, a->dy, a->ld_dy)) return bad(SMC_ERR_ARG, "dx shares memory with dy");
    const Rows rows[] = {{"x", a->x, a->ldx, a->c}, {"dy", a->dy, a->ld_dy, a->c}, {"dx", a->dx, a->ld_dx, a->c}};
    const Vector to[] = {{"dweight", a->dweight, row}, {"dbias", a->dbias, row}};
    for (const Vector& t : to) {
        for (const Vector& v : in) CHECK(apart(t, v));
        CHECK(apart(t, stats));
        for (const Rows& r : rows) CHECK(apart(t, r, a->n));
    }
    for (const Vector& v : in) CHECK(apart(v, rows[2], a->n));
    CHECK(apart(stats, rows[2], a->n));
    return apart(to[0], to[1]);
}

GroupArgs group_args(const smc_group_norm_t* a) {
    GroupArgs p;
    p.n = a->n;
    p.c = a->c;
    p.groups = a->groups;
    p.samples = a->samples;
    p.offsets = a->offsets;
    group_plan(p);
    return p;
}

size_t group_bytes(const GroupArgs& p) { return round_up((size_t)p.pieces * p.groups * 8); }

size_t group_workspace(const smc_group_norm_t* a, bool backward) {
    if (!a || a->n < 0 || a->n > kMaxRows || a->c < 1 || a->c > kMaxGroupChannels || a->groups < 1 ||
        a->groups > kMaxGroupsOfNorm || a->samples < 1 || a->samples > kMaxSamples)
        return 0;
    const GroupArgs p = group_args(a);
    return group_bytes(p) + (backward ? round_up((size_t)p.pieces * p.c * 8) : 0);
}

int group(const smc_group_norm_t* a, bool backward, void* stream) {
    CHECK(check_group(a, backward));
    const size_t need = group_workspace(a, backward);
    if (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need)
        return bad(SMC_ERR_ARG, "workspace: %zu bytes at %p, %zu needed, 16-byte aligned", a->workspace_bytes,
                   a->workspace, need);
    GroupArgs p = group_args(a);
    p.act = a->activation;
    p.eps = a->eps;
    p.x = a->x;
    p.ldx = a->ldx;
    p.weight = a->weight;
    p.bias = a->bias;
    p.stats = a->stats;
    p.by_group = static_cast<float*>(a->workspace);
    p.vec = a->c % 8 == 0 && words16(a->x, a->ldx) && aligned16(a->weight) && aligned16(a->bias);
    if (!backward) {
        p.y = a->y;
        p.ldy = a->ldy;
        p.vec = p.vec && words16(p.y, p.ldy);
        return hip_status(launch_group_norm(p, a->dtype, (hipStream_t)stream), "smc_group_norm");
    }
    p.y = a->dx;
    p.ldy = a->ld_dx;
    p.dy = a->dy;
    p.lddy = a->ld_dy;
    p.dweight = a->dweight;
    p.dbias = a->dbias;
    p.by_channel = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + group_bytes(p));
    p.vec = p.vec && words16(p.y, p.ldy) && words16(p.dy, p.lddy);
    return hip_status(launch_group_norm_backward(p, a->dtype, (hipStream_t)stream), "smc_group_norm_backward");
}

// ---- windows -----------------------------------------------------------------------

int check_windows(const smc_windows_t* w) {
    if (!w) return bad(SMC_ERR_ARG, "windows is NULL");
    if (w->n < 0 || w->n > kMaxRows) return bad(SMC_ERR_ARG, "n = %lld", (long long)w->n);
    if (w->windows < 0 || w->windows > kMaxWindows)
        return bad(SMC_ERR_ARG, "windows = %lld outside [0, 2^24]", (long long)w->windows);
    if (!w->plan || !aligned16(w->plan) || w->plan_bytes < WindowLayout(w->n, w->windows).bytes)
        return bad(SMC_ERR_ARG, "plan: %zu bytes at %p, %zu needed, 16-byte aligned", w->plan_bytes, w->plan,
                   WindowLayout(w->n, w->windows).bytes);
    if (w->ex < 0 || w->ey < 0 || w->ez < 0 || ((w->ex | w->ey | w->ez) && (w->ex < 1 || w->ey < 1 || w->ez < 1)))
        return bad(SMC_ERR_ARG, "extent %d x %d x %d", w->ex, w->ey, w->ez);
    const int extent[3] = {w->ex, w->ey, w->ez};
    if (w->ex > kMaxCells || w->ey > kMaxCells || w->ez > kMaxCells || Cells(extent).all() > kMaxCells)
        return bad(SMC_ERR_UNSUPPORTED, "extent %d, %d, %d: more than %d cells in all, each rounded up to a multiple of 4",
                   w->ex, w->ey, w->ez, kMaxCells);
    return SMC_OK;
}

int build_windows(smc_windows_t* w, hipStream_t s) {
    CHECK(check_windows(w));
    if (!w->offsets || odd(w->offsets, 4)) return bad(SMC_ERR_ARG, "offsets is NULL or misaligned");
    if (odd(w->order, 4) || odd(w->coords, 4)) return bad(SMC_ERR_ARG, "order or coords is not aligned to its elements");
    if (w->coords && w->coord_cols != 3 && w->coord_cols != 4)
        return bad(SMC_ERR_ARG, "coord_cols = %d", w->coord_cols);
    if (!w->coords && w->ex > 0 && w->n > 0) return bad(SMC_ERR_ARG, "an extent needs coords");
    if (w->coords && w->ex < 1) return bad(SMC_ERR_ARG, "coords need an extent");
    w->tiles32 = w->tiles64 = w->tiles128 = w->longest = 0;
    w->pairs = 0;
    WindowArgs p;
    p.n = w->n;
    p.windows = w->windows;
    p.offsets = w->offsets;
    p.order = w->order;
    p.coords = w->coords;
    p.cols = w->coord_cols;
    p.extent[0] = w->ex;
    p.extent[1] = w->ey;
    p.extent[2] = w->ez;
    p.plan = static_cast<char*>(w->plan);
    CHECK(hip_status(launch_windows(p, s), "smc_windows_build"));
    WindowHeader h;
    CHECK(hip_status(hipMemcpyAsync(&h, w->plan, sizeof h, hipMemcpyDeviceToHost, s), "smc_windows_build"));
    CHECK(hip_status(hipStreamSynchronize(s), "smc_windows_build"));
    if (h.status & kStRange)
        return bad(SMC_ERR_RANGE, "offsets that do not ascend within [0, n], a row of order outside it, or a window of "
                                  "more cells than its extent");
    if (h.status & kStDuplicate) return bad(SMC_ERR_DUPLICATE, "order has a row twice");
    w->tiles32 = h.tiles[0];
    w->tiles64 = h.tiles[1];
    w->tiles128 = h.tiles[2];
    w->longest = h.longest;
    w->pairs = (int64_t)h.pairs;
    return SMC_OK;
}

// ---- window attention ----------------------------------------------------------------

constexpr int kMaxHeadDim = 128;

int check_attention(const smc_attention_t* a, bool backward) {
    if (!a) return bad(SMC_ERR_ARG, "args is NULL");
    CHECK(check_windows(a->windows));
    const int64_t n = a->windows->n;
    if (n > 0 && a->windows->tiles64 < 1) return bad(SMC_ERR_STATE, "windows is not built");
    if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads)
        return bad(SMC_ERR_ARG, "%d heads, %d of keys and values", a->heads, a->kv_heads);
    if (a->head_dim < 1) return bad(SMC_ERR_ARG, "head_dim = %d", a->head_dim);
    if (a->head_dim > kMaxHeadDim) return bad(SMC_ERR_UNSUPPORTED, "head_dim = %d, more than %d", a->head_dim, kMaxHeadDim);
    const int64_t c = (int64_t)a->heads * a->head_dim, ckv = (int64_t)a->kv_heads * a->head_dim;
    CHECK(check_common(n, c, "heads * head_dim", a->dtype));
    if ((int64_t)a->windows->tiles32 * a->heads >= (int64_t)1 << 31)
        return bad(SMC_ERR_UNSUPPORTED, "%d tiles of %d heads: 2^31 or more", a->windows->tiles32, a->heads);
    if (!(a->scale > 0.f) || a->scale > 0x1p126f)      // (its product with log2 e is finite)
        return bad(SMC_ERR_ARG, "scale = %g", (double)a->scale);
    CHECK(check_rows("q", a->q, n, c, a->ldq));
    CHECK(check_rows("k", a->k, n, ckv, a->ldk));
    CHECK(check_rows("v", a->v, n, ckv, a->ldv));
    CHECK(check_rows("out", a->out, n, c, a->ld_out));
    if (odd(a->lse, 4)) return bad(SMC_ERR_ARG, "lse is not aligned to its elements");
    if (a->bias) {
        if (odd(a->bias, 2)) return bad(SMC_ERR_ARG, "bias is not aligned to its elements");
        if (a->windows->ex < 1) return bad(SMC_ERR_STATE, "a bias needs windows with cells");
        if (a->reach < 1 || a->reach > kMaxReach) return bad(SMC_ERR_ARG, "reach = %d outside [1, %d]", a->reach, kMaxReach);
    }
    const Vector lse = {"lse", a->lse, (size_t)a->heads * n * 4};
    const Vector table = {"bias", a->bias, a->bias ? (size_t)3 * (2 * a->reach + 1) * a->heads * 2 : 0};
    const Rows in[] = {{"q", a->q, a->ldq, c}, {"k", a->k, a->ldk, ckv}, {"v", a->v, a->ldv, ckv},
                       {"out", a->out, a->ld_out, c}, {"dout", a->dout, a->ld_dout, c}};
    if (!backward) {
        CHECK(apart(table, in[3], n));
        CHECK(apart(lse, table));
        for (int i = 0; i < 4; ++i) CHECK(apart(lse, in[i], n));
        // other blocks read the inputs' rows again
        if (share_memory(a->out, a->ld_out, 2, a->q, a->ldq, 2, n, c, c) ||
            share_memory(a->out, a->ld_out, 2, a->k, a->ldk, 2, n, c, ckv) ||
            share_memory(a->out, a->ld_out, 2, a->v, a->ldv, 2, n, c, ckv))
            return bad(SMC_ERR_ARG, "out shares memory with q, k or v");
        return SMC_OK;
    }
    if (!a->lse && n > 0) return bad(SMC_ERR_ARG, "lse is NULL");
    CHECK(check_rows("dout", a->dout, n, c, a->ld_dout));
    CHECK(check_rows("dq", a->dq, n, c, a->ld_dq));
    CHECK(check_rows("dk", a->dk, n, ckv, a->ld_dk));
    CHECK(check_rows("dv", a->dv, n, ckv, a->ld_dv));
    if (a->bias && (!a->dbias || odd(a->dbias, 2))) return bad(SMC_ERR_ARG, "dbias is NULL or misaligned");
    const Rows to[] = {{"dq", a->dq, a->ld_dq, c}, {"dk", a->dk, a->ld_dk, ckv}, {"dv", a->dv, a->ld_dv, ckv}};
    auto shared = [n](const Rows& x, const Rows& y) {
        return share_memory(x.p, x.ld, 2, y.p, y.ld, 2, n, x.cols, y.cols);
    };
    for (int i = 0; i < 3; ++i) {
        for (const Rows& r : in)
            if (shared(to[i], r)) return bad(SMC_ERR_ARG, "%s shares memory with %s", to[i].name, r.name);
        for (int j = 0; j < i; ++j)
            if (shared(to[i], to[j])) return bad(SMC_ERR_ARG, "%s shares memory with %s", to[i].name, to[j].name);
    }
    // (dbias is written by the last kernel: it may be bias)
    const Vector to_table = {"dbias", a->dbias, table.bytes};
    CHECK(apart(to_table, lse));
    for (const Rows& r : in) CHECK(apart(to_table, r, n));
    for (const Rows& r : to) {
        CHECK(apart(table, r, n));
        CHECK(apart(lse, r, n));
        CHECK(apart(to_table, r, n));
    }
    return SMC_OK;
}

bool attention_words(const smc_attention_t* a, bool backward) {
    return a->head_dim % 8 == 0 && words16(a->q, a->ldq) && words16(a->k, a->ldk) && words16(a->v, a->ldv) &&
           words16(a->out, a->ld_out) &&
           (!backward || (words16(a->dout, a->ld_dout) && words16(a->dq, a->ld_dq) && words16(a->dk, a->ld_dk) &&
                          words16(a->dv, a->ld_dv)));
}

bool short_windows(const smc_windows_t* w) { return w->windows > 0 && w->n / w->windows < 40; }

// Blocks by the windows' lengths: short where they are short on average, long where the rows are mostly in
// long ones (pairs / rows) and there are blocks for the device. Forward / backward in us, short, mid and long:
//   40,000 rows x 4 heads of 32, cells, windows of 24   13.8, 17.0, 29.4 / 61.4, 79.9, 114.5
//                                                  60   15.5, 13.4, 16.8 / 56.8, 46.9, 62.4
//                                                 100   25.0, 19.0, 18.2 / 87.3, 67.2, 60.4
//                                                 400   51.5, 37.3, 37.2 / 147.9, 111.7, 104.2
//   16,000 x 8 heads of 64, windows of             24   15.6, 17.1, 26.5 / 44.4, 58.1, 84.6
//                                                  60   16.5, 13.9, 16.3 / 45.7, 41.1, 50.5
//                                                 100   22.2, 18.7, 18.1 / 62.7, 58.8, 54.7
//                                                 400   45.5, 34.1, 31.4 / 135.8, 108.1, 97.5
//   91,000 x 4 of 32, cells, 2,905 windows of 1 .. 160  50.5, 48.9, 67.5 / 172.2, 186.6, 227.4
// (A few long windows among many short ones stay with short blocks, whose starts cost least: 20,000 windows of a row
// and 20 of 1,000, 4 heads of 32: short 256 / 726, long 345 / 841; 2,000 of 10 and 40 of 500, 8 of 64: 204 / 579, 253 / 853.)
// Rows that are no whole 16-byte words have mid blocks only.
int window_lengths(const smc_attention_t* a, bool backward) {
    const smc_windows_t* w = a->windows;
    if (!attention_words(a, backward) || w->windows < 1) return kMidWindows;
    if (short_windows(w)) return kShortWindows;
    return w->pairs / w->n < 96 || (int64_t)w->tiles128 * a->heads < device_cus() ? kMidWindows : kLongWindows;
}

int tiles_of(const smc_windows_t* w, int lengths) {
    return lengths == kShortWindows ? w->tiles32 : lengths == kMidWindows ? w->tiles64 : w->tiles128;
}

AttentionArgs attention_args(const smc_attention_t* a, int lengths, bool backward) {
    AttentionArgs p;
    const smc_windows_t* w = a->windows;
    const WindowLayout at(w->n, w->windows);
    p.n = w->n;
    p.heads = a->heads;
    p.kv_heads = a->kv_heads;
    p.dim = a->head_dim;
    p.scale = a->scale;
    p.q = a->q;
    p.ldq = a->ldq;
    p.k = a->k;
    p.ldk = a->ldk;
    p.v = a->v;
    p.ldv = a->ldv;
    const char* plan = static_cast<const char*>(w->plan);
    p.places = reinterpret_cast<const WindowPlace*>(plan + at.places);
    p.tiles = reinterpret_cast<const WindowTile*>(plan + at.tiles[lengths]);
    p.n_tiles = tiles_of(w, lengths);
    p.tiles64 = reinterpret_cast<const WindowTile*>(plan + at.tiles[1]);
    p.n_tiles64 = w->tiles64;
    p.extent[0] = w->ex;
    p.extent[1] = w->ey;
    p.extent[2] = w->ez;
    p.table = a->bias;
    p.reach = a->reach;
    p.out = a->out;
    p.ldo = a->ld_out;
    p.lse = a->lse;
    p.vec = attention_words(a, backward);
    return p;
}

int attention(const smc_attention_t* a, void* stream) {
    CHECK(check_attention(a, false));
    if (a->windows->n == 0) return SMC_OK;
    const int lengths = window_lengths(a, false);
    const AttentionArgs p = attention_args(a, lengths, false);
    const hipStream_t s = (hipStream_t)stream;
    return hip_status(a->dtype == SMC_DTYPE_F16 ? launch_attention_f16(p, lengths, s) : launch_attention_bf16(p, lengths, s),
                      "smc_window_attention");
}

// Scratch of a backward pass: delta, the blocks' buckets, and f16's maxima. For the more tiles of those that
// window_lengths may choose, whatever the alignment.
struct AttentionScratch {
    size_t delta = 0, part = 0, range = 0, bytes = 0;       // offsets
    explicit AttentionScratch(const smc_attention_t* a) {
        const smc_windows_t* w = a->windows;
        part = round_up((size_t)a->heads * w->n * 4);
        const int64_t tiles = short_windows(w) ? w->tiles32 : w->tiles64;
        range = part + (a->bias ? round_up((size_t)tiles * a->heads * 3 * (2 * a->reach + 1) * 4) : 0);
        bytes = range + (a->dtype == SMC_DTYPE_F16 ? round_up((size_t)w->tiles64 * (a->heads + a->kv_heads) * 4) : 0);
    }
};

size_t attention_workspace(const smc_attention_t* a) {
    if (!a || !a->windows || a->windows->n < 0 || a->windows->n > kMaxRows || a->windows->windows < 0 || a->heads < 1 ||
        a->heads > kMaxDim || a->kv_heads < 1 || a->kv_heads > a->heads || a->reach < 0 || a->reach > kMaxReach ||
        a->windows->tiles32 < 0 || a->windows->tiles64 < 0 || a->windows->tiles128 < 0)
        return 0;
    return AttentionScratch(a).bytes;
}

int attention_backward(const smc_attention_t* a, void* stream) {
    CHECK(check_attention(a, true));
    const AttentionScratch at(a);
    if (a->windows->n > 0 && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < at.bytes))
        return bad(SMC_ERR_ARG, "workspace: %zu bytes at %p, %zu needed, 16-byte aligned", a->workspace_bytes,
                   a->workspace, at.bytes);
    const int lengths = window_lengths(a, true);
    AttentionArgs p = attention_args(a, lengths, true);
    char* const ws = static_cast<char*>(a->workspace);
    p.dout = a->dout;
    p.ld_dout = a->ld_dout;
    p.dq = a->dq;
    p.ld_dq = a->ld_dq;
    p.dk = a->dk;
    p.ld_dk = a->ld_dk;
    p.dv = a->dv;
    p.ld_dv = a->ld_dv;
    p.dtable = a->dbias;
    p.delta = reinterpret_cast<float*>(ws);
    p.part = reinterpret_cast<float*>(ws + at.part);
    p.range = reinterpret_cast<float*>(ws + at.range);
    const hipStream_t s = (hipStream_t)stream;
    return hip_status(a->dtype == SMC_DTYPE_F16 ? launch_attention_backward_f16(p, lengths, s)
                                                : launch_attention_backward_bf16(p, lengths, s),
                      "smc_window_attention_backward");
}

}  // namespace

extern "C" {

int smc_group_norm(const smc_group_norm_t* a, void* stream) { return group(a, false, stream); }
int smc_group_norm_backward(const smc_group_norm_t* a, void* stream) { return group(a, true, stream); }
size_t smc_group_norm_workspace(const smc_group_norm_t* a) { return group_workspace(a, false); }
size_t smc_group_norm_backward_workspace(const smc_group_norm_t* a) { return group_workspace(a, true); }

size_t smc_windows_bytes(int64_t n, int64_t windows) {
    if (n < 0 || n > kMaxRows || windows < 0 || windows > kMaxWindows) return 0;
    return WindowLayout(n, windows).bytes;
}
int smc_windows_build(smc_windows_t* w, void* stream) { return build_windows(w, (hipStream_t)stream); }

int smc_window_attention(const smc_attention_t* a, void* stream) { return attention(a, stream); }
int smc_window_attention_backward(const smc_attention_t* a, void* stream) { return attention_backward(a, stream); }
size_t smc_window_attention_backward_workspace(const smc_attention_t* a) { return attention_workspace(a); }

}  // extern "C"
