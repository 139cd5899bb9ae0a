// C entries of the row operators: argument checks, scratch layout and launches.
// See include/smconv.h for the contract of each call.
#include <cstdarg>
#include <cstdio>

#include "smconv.h"
#include "pointwise.h"

using namespace smc;

namespace {

constexpr int64_t kMaxDim = 1 << 21;           // channels and row distances: tile offsets fit 31 bits
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;   // row numbers are 32-bit
constexpr size_t kAlign = 256;

int bad(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int bad(int status, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(status, buf);
}

int hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return SMC_OK;
    return bad(SMC_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool words16(const void* p, int64_t ld) { return aligned16(p) && (ld & 7) == 0; }   // 16-bit rows
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// A [rows, cols] tensor: present where it has elements, row distance in range.
int check_rows(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (!p && rows > 0) return bad(SMC_ERR_ARG, "%s is NULL", name);
    if (ld < cols || ld > kMaxDim)
        return bad(SMC_ERR_ARG, "row distance of %s is %lld, outside [%lld, 2^21]", name, (long long)ld,
                   (long long)cols);
    if (((uintptr_t)p & 1) != 0) return bad(SMC_ERR_ARG, "%s is not aligned to its elements", name);
    return SMC_OK;
}

// Do the tensors at p and q (rows of cols elements of es bytes, ld elements from
// row to row) share memory? Columns of one buffer, whose ranges overlap with equal
// row distances in bytes, are told apart; other overlapping ranges count as shared.
bool share_memory(const void* p, int64_t ldp, int esp, const void* q, int64_t ldq, int esq, int64_t rows,
                  int64_t colsp, int64_t colsq) {
    if (!p || !q || rows <= 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    const uint64_t pitch = (uint64_t)ldp * esp, wp = (uint64_t)colsp * esp, wq = (uint64_t)colsq * esq;
    if (a + (uint64_t)(rows - 1) * pitch + wp <= b || b + (uint64_t)(rows - 1) * ldq * esq + wq <= a) return false;
    if (pitch != (uint64_t)ldq * esq) return true;
    const uint64_t apart = a > b ? (pitch - (a - b) % pitch) % pitch : (b - a) % pitch;    // q's columns after p's
    return apart < wp || apart + wq > pitch;
}

int check_common(int64_t n, int64_t c, const char* cname, int dtype) {
    if (n < 0 || n > kMaxRows) return bad(SMC_ERR_ARG, "n = %lld", (long long)n);
    if (c < 1 || c > kMaxDim) return bad(SMC_ERR_ARG, "%s = %lld outside [1, 2^21]", cname, (long long)c);
    if (dtype != SMC_DTYPE_BF16 && dtype != SMC_DTYPE_F16)
        return bad(SMC_ERR_ARG, "dtype %d (SMC_DTYPE_BF16 or SMC_DTYPE_F16)", dtype);
    return SMC_OK;
}

#define CHECK(call)              \
    do {                         \
        const int rc_ = (call);  \
        if (rc_) return rc_;     \
    } while (0)

// Checks of smc_linear, smc_gated (halves = 2) and their backward passes.
int check_product(const smc_product_t* a, int halves, bool backward) {
    if (!a) return bad(SMC_ERR_ARG, "args is NULL");
    CHECK(check_common(a->n, a->c_in, "c_in", a->dtype));
    if (a->c_out < 1 || a->c_out > kMaxDim / halves)
        return bad(SMC_ERR_ARG, "c_out = %d outside [1, 2^21%s]", a->c_out, halves == 2 ? " / 2" : "");
    const int64_t wide = (int64_t)a->c_out * halves;
    const bool e4m3 = a->x_dtype == SMC_DTYPE_E4M3;
    if (!e4m3 && a->x_dtype != a->dtype)
        return bad(SMC_ERR_ARG, "x_dtype %d with dtype %d", a->x_dtype, a->dtype);
    if (e4m3 && backward) return bad(SMC_ERR_UNSUPPORTED, "gradients of e4m3 layers");
    if (a->activation < SMC_ACT_NONE || a->activation > SMC_ACT_GELU)
        return bad(SMC_ERR_ARG, "activation %d", a->activation);
    // the weights are addressed by 31-bit byte offsets from their first element
    if (a->w_transposed && !e4m3) return bad(SMC_ERR_UNSUPPORTED, "w_transposed is for e4m3 weights");
    const int64_t w_rows = a->w_transposed ? wide : a->c_in, w_cols = a->w_transposed ? a->c_in : wide;
    if (!a->w) return bad(SMC_ERR_ARG, "w is NULL");
    if (a->ldw < w_cols || a->ldw > kMaxDim)
        return bad(SMC_ERR_ARG, "row distance of w is %lld, outside [%lld, 2^21]", (long long)a->ldw,
                   (long long)w_cols);
    const int per = e4m3 ? 16 : 8;
    const int64_t padded = ((int64_t)a->c_in + per - 1) / per * per * ((a->c_out + per - 1) / per * per) * halves;
    if ((w_rows * a->ldw > padded ? w_rows * a->ldw : padded) * (e4m3 ? 1 : 2) >= ((int64_t)1 << 31))
        return bad(SMC_ERR_UNSUPPORTED, "w spans 2^31 bytes or more");
    if (e4m3) {
        if (!a->w_scale || (!a->x_scale && a->n > 0)) return bad(SMC_ERR_ARG, "e4m3 operands need scales");
        if (!a->x && a->n > 0) return bad(SMC_ERR_ARG, "x is NULL");
        if (a->ldx < a->c_in || a->ldx > kMaxDim)
            return bad(SMC_ERR_ARG, "row distance of x is %lld", (long long)a->ldx);
    } else {
        CHECK(check_rows("x", a->x, a->n, a->c_in, a->ldx));
        if (((uintptr_t)a->w & 1) != 0) return bad(SMC_ERR_ARG, "w is not aligned to its elements");
    }
    if (((uintptr_t)a->bias & 1) != 0) return bad(SMC_ERR_ARG, "bias is not aligned to its elements");
    if (a->residual && (halves == 2 || backward))
        return bad(SMC_ERR_ARG, "residual is an argument of smc_linear only");
    if (!backward) {
        if (a->residual) CHECK(check_rows("residual", a->residual, a->n, a->c_out, a->ld_residual));
        CHECK(check_rows("y", a->y, a->n, a->c_out, a->ldy));
        // (blocks of other column tiles read x again)
        if (share_memory(a->y, a->ldy, 2, a->x, a->ldx, e4m3 ? 1 : 2, a->n, a->c_out, a->c_in))
            return bad(SMC_ERR_ARG, "y shares memory with x");
        return SMC_OK;
    }
    CHECK(check_rows("dy", a->dy, a->n, a->c_out, a->ld_dy));
    CHECK(check_rows("dx", a->dx, a->n, a->c_in, a->ld_dx));
    if (!a->dw) return bad(SMC_ERR_ARG, "dw is NULL");
    CHECK(check_rows("dw", a->dw, a->c_in, wide, a->ld_dw));
    if (((uintptr_t)a->db & 1) != 0) return bad(SMC_ERR_ARG, "db is not aligned to its elements");
    // dW is taken from x after dx, and from dy too where no activation changes it
    if (share_memory(a->dx, a->ld_dx, 2, a->x, a->ldx, 2, a->n, a->c_in, a->c_in))
        return bad(SMC_ERR_ARG, "dx shares memory with x");
    if (halves == 1 && a->activation == SMC_ACT_NONE &&
        share_memory(a->dx, a->ld_dx, 2, a->dy, a->ld_dy, 2, a->n, a->c_in, a->c_out))
        return bad(SMC_ERR_ARG, "dx shares memory with dy");
    return SMC_OK;
}

ProductArgs forward_args(const smc_product_t* a, int halves) {
    ProductArgs p;
    const int es = a->x_dtype == SMC_DTYPE_E4M3 ? 1 : 2;
    p.a = a->x;
    p.lda = a->ldx;
    p.b = a->w;
    p.ldb = a->ldw;
    p.m = (int)a->n;
    p.k = a->c_in;
    p.n = a->c_out * halves;
    p.half = a->c_out;
    p.bias = a->bias;
    p.a_scale = a->x_scale;
    p.b_scale = a->w_scale;
    p.act = a->activation;
    // a row of x, and of w^T, is whole 16-byte words; of w, each half starts at one
    const int per = 16 / es;
    p.vec_a = aligned16(a->x) && a->ldx % per == 0 && a->c_in % per == 0;
    p.vec_b = aligned16(a->w) && a->ldw % per == 0 &&
              (a->w_transposed ? a->c_in % per == 0 : halves == 1 || a->c_out % per == 0);
    return p;
}

// Padded copies of x and w that a forward product takes where their rows are
// not whole 16-byte words: x [n, k] and w [k, halves half], zeros between. They
// cost a pass over x and w and two launches, and spare the product the staging
// of both operands through registers. In place and with copies, us on the GPU:
//   w unaligned:  1,000 x 128 -> 141 11.4, 6.7   91,000 x 128 -> 141 59.4, 27.6
//                 91,000 x 141 -> 141 81.4, 44.4   gated 300 x 702 -> 1365 51.2, 16.4
//                 91,000 x 128 -> 341 gated 61.8, 45.6
//   x alone:      20,000 x 250 -> 128 13.3, 17.6; -> 256 15.8, 21.6; -> 512 29.1, 27.4;
//                 -> 1024 53.9, 34.0   4,000 x 1241 -> 464 38.1, 25.9
//   e4m3, w in [k, n] order: 20 x 1488 -> 106 78.2, 10.3   41,305 x 240 -> 995 93.9, 51.8
//   e4m3, x alone: 20,000 x 250 -> 128 / 512 20.9 / 42.9, 14.9 / 23.1
//   one step:     220 x 46 -> 128 5.9, 7.6   13,654 x 29 -> 65 8.2, 8.9
// so they are made for contractions of more than one step (128 bytes) where w is
// unaligned, or x is and is staged often (more than 256 columns) or long (512).
struct Padded {
    bool copy_x = false, copy_w = false;
    int k = 0, half = 0;
    size_t w = 0, bytes = 0;    // offset of w's; all of them (0: none needed)
};

Padded padded_of(const smc_product_t* a, const ProductArgs& p) {
    Padded pd;
    const int halves = p.n / a->c_out, es = a->x_dtype == SMC_DTYPE_E4M3 ? 1 : 2, per = 16 / es;
    if ((es == 2 && few_rows_pay(p, halves == 2 ? kEpiGated : kEpiStore)) || (p.vec_a && p.vec_b)) return pd;
    if (a->c_in <= 128 / es || (p.vec_b && p.n <= 256 && a->c_in <= 512)) return pd;
    pd.copy_x = !p.vec_a;
    pd.k = (a->c_in + per - 1) / per * per;
    pd.copy_w = !p.vec_b || pd.k != a->c_in;
    // (w^T has its halves in rows)
    pd.half = pd.copy_w && !a->w_transposed ? (a->c_out + per - 1) / per * per : a->c_out;
    if (pd.copy_x) pd.w = round_up((size_t)a->n * pd.k * es);
    pd.bytes = pd.w + (pd.copy_w ? round_up((size_t)pd.k * pd.half * halves * es) : 0);
    return pd;
}

size_t forward_workspace_of(const smc_product_t* a, int halves) {
    if (!a || a->n < 0 || a->n > kMaxRows || a->c_in < 1 || a->c_in > kMaxDim || a->c_out < 1 ||
        a->c_out > kMaxDim / halves)
        return 0;
    return padded_of(a, forward_args(a, halves)).bytes;
}

int forward(const smc_product_t* a, int halves, Epilogue epi, void* stream) {
    CHECK(check_product(a, halves, false));
    if (a->n == 0) return SMC_OK;
    ProductArgs p = forward_args(a, halves);
    p.out = a->y;
    p.ldo = a->ldy;
    p.extra = a->residual;
    p.ld_extra = a->ld_residual;
    const Padded pd = padded_of(a, p);
    if (pd.bytes && a->workspace && aligned16(a->workspace) && a->workspace_bytes >= pd.bytes) {
        const hipStream_t s = (hipStream_t)stream;
        char* const ws = static_cast<char*>(a->workspace);
        const int es = a->x_dtype == SMC_DTYPE_E4M3 ? 1 : 2, wide = pd.half * halves;
        if (pd.copy_x) {
            CHECK(hip_status(launch_pad_rows(es, p.a, p.lda, a->n, 1, a->c_in, ws, pd.k, a->n, pd.k, s), "copy of x"));
            p.a = ws;
            p.lda = pd.k;
        }
        if (pd.copy_w) {
            const hipError_t e =
                a->w_transposed
                    ? launch_pad_rows(es, p.b, p.ldb, p.n, 1, a->c_in, ws + pd.w, pd.k, p.n, pd.k, s)
                    : launch_pad_rows(es, p.b, p.ldb, a->c_in, halves, a->c_out, ws + pd.w, wide, pd.k, pd.half, s);
            CHECK(hip_status(e, "copy of w"));
            p.b = ws + pd.w;
            p.ldb = a->w_transposed ? pd.k : wide;
        }
        p.k = pd.k;
        if (halves == 2) {
            p.half_out = a->c_out;
            p.half = pd.half;
            p.n = wide;
        }
        p.vec_a = p.vec_b = 1;
    }
    p.vec_x = a->c_out >= 8;
    return hip_status(launch_forward(p, epi, a->dtype, a->x_dtype == SMC_DTYPE_E4M3, a->w_transposed != 0,
                                     (hipStream_t)stream),
                      halves == 2 ? "smc_gated" : "smc_linear");
}

// Scratch of a backward pass. Its products read x, w, dz or dy as 16-byte words;
// where their rows are not made of such, padded copies take their place: xp
// [n, c_in_p], wp [c_in_p, halves half_p] and the bias alike, zeros between; dz has
// wp's columns; f16: the slopes' maxima and their scale. (Through registers instead, us on the GPU: gated 144 -> 734 with 8 /
// 256 / 4,818 rows 45.7 / 49.3 / 92.6, with the copies 24.6 / 27.0 / 43.0.) Then the
// weight gradient's float32 sums.
struct Scratch {
    bool slope = false;         // dz is made (else it is dy, or its copy)
    bool copy_x = false, copy_w = false, copy_dy = false;
    int half_p = 0, c_in_p = 0; // columns of a half of dz, w; of x
    int wide_p = 0;
    size_t xp = 0, wp = 0, bp = 0, dz = 0, range = 0, part = 0, bytes = 0;      // offsets
    int range_rows = 0, splits = 1;     // ranges of the rows that dW is summed over
};

Scratch scratch_of(const smc_product_t* a, int halves) {
    Scratch s;
    s.slope = halves == 2 || a->activation != SMC_ACT_NONE;
    s.c_in_p = a->c_in;
    const bool w_words = words16(a->w, a->ldw) && a->c_out % 8 == 0;
    const bool x_words = words16(a->x, a->ldx) && (!s.slope || a->c_in % 8 == 0);
    s.half_p = (a->c_out + 7) / 8 * 8;
    if (a->n > 0) {
        s.copy_x = !x_words;
        if (s.copy_x) s.c_in_p = (a->c_in + 7) / 8 * 8;
        s.copy_w = !w_words || s.c_in_p != a->c_in;
        s.copy_dy = !s.slope && !(words16(a->dy, a->ld_dy) && a->c_out % 8 == 0);
    }
    s.wide_p = s.half_p * halves;
    auto take = [&](size_t bytes) {
        const size_t at = s.bytes;
        s.bytes += round_up(bytes);
        return at;
    };
    if (s.copy_x) s.xp = take((size_t)a->n * s.c_in_p * 2);
    if (s.copy_w) s.wp = take((size_t)s.c_in_p * s.wide_p * 2);
    if (s.copy_w && a->bias) s.bp = take((size_t)s.wide_p * 2);
    if (s.slope || s.copy_dy) s.dz = take((size_t)a->n * ((s.wide_p + 7) / 8 * 8) * 2);
    if (s.slope && a->dtype == SMC_DTYPE_F16) s.range = take((size_t)(1 + kMaxBlocksPerCu * device_cus()) * 4);
    s.range_rows = weight_gradient_range(a->n, a->c_in, s.wide_p);
    if (a->n > 0) s.splits = (int)((a->n + s.range_rows - 1) / s.range_rows);
    s.part = take((size_t)s.splits * (a->c_in + (a->db ? 1 : 0)) * s.wide_p * 4);
    return s;
}

size_t workspace_of(const smc_product_t* a, int halves) {
    if (!a || a->n < 0 || a->n > kMaxRows || a->c_in < 1 || a->c_in > kMaxDim || a->c_out < 1 ||
        a->c_out > kMaxDim / halves)
        return 0;
    return scratch_of(a, halves).bytes;
}

int backward(const smc_product_t* a, int halves, void* stream) {
    const char* name = halves == 2 ? "smc_gated_backward" : "smc_linear_backward";
    CHECK(check_product(a, halves, true));
    const Scratch sc = scratch_of(a, halves);
    if (a->n > 0 && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < sc.bytes))
        return bad(SMC_ERR_ARG, "workspace: %zu bytes at %p, %zu needed, 16-byte aligned",
                   a->workspace_bytes, a->workspace, sc.bytes);
    const hipStream_t s = (hipStream_t)stream;
    char* const ws = static_cast<char*>(a->workspace);
    SumArgs sum;
    sum.m = a->c_in;
    sum.n = sc.wide_p;
    sum.half_p = sc.half_p;
    sum.c_out = a->c_out;
    sum.dw = a->dw;
    sum.ldw = a->ld_dw;
    sum.db = a->db;
    if (a->n == 0) return hip_status(launch_sum_parts(sum, a->dtype, s), name);

    const void *x = a->x, *w = a->w, *bias = a->bias, *dz = a->dy;
    const float* unscale = nullptr;
    int64_t ldx = a->ldx, ldw = a->ldw, ld_dz = a->ld_dy;
    if (sc.copy_x) {
        CHECK(hip_status(launch_pad_rows(2, x, ldx, a->n, 1, a->c_in, ws + sc.xp, sc.c_in_p, a->n, sc.c_in_p, s), name));
        x = ws + sc.xp;
        ldx = sc.c_in_p;
    }
    if (sc.copy_w) {
        CHECK(hip_status(launch_pad_rows(2, w, ldw, a->c_in, halves, a->c_out, ws + sc.wp, sc.wide_p, sc.c_in_p,
                                         sc.half_p, s), name));
        w = ws + sc.wp;
        ldw = sc.wide_p;
        if (bias && sc.slope) {
            CHECK(hip_status(launch_pad_rows(2, bias, (int64_t)a->c_out * halves, 1, halves, a->c_out, ws + sc.bp,
                                             sc.wide_p, 1, sc.half_p, s), name));
            bias = ws + sc.bp;
        }
    }
    if (sc.slope) {
        ProductArgs p;
        p.a = x;
        p.lda = ldx;
        p.b = w;
        p.ldb = ldw;
        p.m = (int)a->n;
        p.k = sc.c_in_p;
        p.n = sc.wide_p;
        p.half = sc.half_p;
        p.bias = bias;
        p.act = a->activation;
        p.extra = a->dy;
        p.ld_extra = a->ld_dy;
        p.extra_width = a->c_out;
        p.out = ws + sc.dz;
        p.ldo = (sc.wide_p + 7) / 8 * 8;
        p.vec_a = words16(x, ldx) && sc.c_in_p % 8 == 0;
        p.vec_b = words16(w, ldw) && (halves == 1 || sc.half_p % 8 == 0);
        p.vec_x = a->c_out >= 8;
        const Epilogue epi = halves == 2 ? kEpiGatedSlope : kEpiSlope;
        const bool f16 = a->dtype == SMC_DTYPE_F16;
        float* const range = reinterpret_cast<float*>(ws + sc.range);
        if (f16) p.dz_max = range + 1;
        CHECK(hip_status(launch_forward(p, epi, a->dtype, false, false, s), name));
        if (f16) {
            p.dz_unscale = range;
            CHECK(hip_status(launch_forward(p, epi, a->dtype, false, false, s), name));
            unscale = range;
        }
        dz = p.out;
        ld_dz = p.ldo;
    } else if (sc.copy_dy) {
        CHECK(hip_status(launch_pad_rows(2, dz, ld_dz, a->n, 1, a->c_out, ws + sc.dz, sc.half_p, a->n, sc.half_p, s), name));
        dz = ws + sc.dz;
        ld_dz = sc.half_p;
    }
    {
        ProductArgs p;                          // dx = dz W^T
        p.a = dz;
        p.lda = ld_dz;
        p.b = w;
        p.ldb = ldw;
        p.m = (int)a->n;
        p.k = sc.wide_p;
        p.n = a->c_in;
        p.unscale = unscale;
        p.out = a->dx;
        p.ldo = a->ld_dx;
        p.vec_a = words16(dz, ld_dz) && sc.wide_p % 8 == 0;
        p.vec_b = words16(w, ldw) && sc.wide_p % 8 == 0;
        CHECK(hip_status(launch_input_gradient(p, a->dtype, s), name));
    }
    ProductArgs p;                              // dW = x^T dz
    p.a = x;
    p.lda = ldx;
    p.b = dz;
    p.ldb = ld_dz;
    p.m = a->c_in;
    p.k = (int)a->n;
    p.n = sc.wide_p;
    p.part = reinterpret_cast<float*>(ws + sc.part);
    p.k_split = sc.range_rows;
    p.splits = sc.splits;
    p.colsum = a->db != nullptr;
    p.vec_a = words16(x, ldx);
    p.vec_b = words16(dz, ld_dz);
    CHECK(hip_status(launch_weight_gradient(p, a->dtype, s), name));
    sum.part = p.part;
    sum.splits = sc.splits;
    sum.unscale = unscale;
    return hip_status(launch_sum_parts(sum, a->dtype, s), name);
}

}  // namespace

extern "C" {

int smc_rms_norm(const smc_norm_t* a, void* stream) {
    if (!a) return bad(SMC_ERR_ARG, "args is NULL");
    CHECK(check_common(a->n, a->c, "c", a->dtype));
    if (!(a->eps >= 0.f)) return bad(SMC_ERR_ARG, "eps = %g", (double)a->eps);
    if (!a->weight || ((uintptr_t)a->weight & 1)) return bad(SMC_ERR_ARG, "weight is NULL or misaligned");
    CHECK(check_rows("x", a->x, a->n, a->c, a->ldx));
    if (a->residual) CHECK(check_rows("residual", a->residual, a->n, a->c, a->ld_residual));
    if (a->s) CHECK(check_rows("s", a->s, a->n, a->c, a->lds));
    if (!a->y && a->n > 0) return bad(SMC_ERR_ARG, "y is NULL");
    if (a->ldy < a->c || a->ldy > kMaxDim)
        return bad(SMC_ERR_ARG, "row distance of y is %lld, outside [%d, 2^21]", (long long)a->ldy, a->c);
    if (!a->y_scale && ((uintptr_t)a->y & 1)) return bad(SMC_ERR_ARG, "y is not aligned to its elements");
    // e4m3 rows over 16-bit ones: a row of y would lie in other rows' bytes, which
    // another wave may not have read
    if (a->y_scale && (share_memory(a->y, a->ldy, 1, a->x, a->ldx, 2, a->n, a->c, a->c) ||
                       share_memory(a->y, a->ldy, 1, a->residual, a->ld_residual, 2, a->n, a->c, a->c) ||
                       share_memory(a->y, a->ldy, 1, a->s, a->lds, 2, a->n, a->c, a->c)))
        return bad(SMC_ERR_ARG, "e4m3 y shares memory with x, residual or s");
    NormArgs p;
    p.n = a->n;
    p.c = a->c;
    p.eps = a->eps;
    p.x = a->x;
    p.ldx = a->ldx;
    p.residual = a->residual;
    p.ldr = a->ld_residual;
    p.weight = a->weight;
    p.y = a->y;
    p.ldy = a->ldy;
    p.y_scale = a->y_scale;
    p.s = a->s;
    p.lds = a->lds;
    const bool y_ok = a->y_scale ? ((uintptr_t)a->y & 7) == 0 && a->ldy % 8 == 0 : words16(a->y, a->ldy);
    p.vec = a->c % 8 == 0 && words16(a->x, a->ldx) && (!a->residual || words16(a->residual, a->ld_residual)) &&
            (!a->s || words16(a->s, a->lds)) && aligned16(a->weight) && y_ok;
    return hip_status(launch_norm(p, a->dtype, (hipStream_t)stream), "smc_rms_norm");
}

size_t smc_rms_norm_backward_workspace(int64_t n, int c) {
    if (n < 0 || n > kMaxRows || c < 1 || c > kMaxDim) return 0;
    return round_up((size_t)norm_backward_blocks(n, c) * c * 4);
}

int smc_rms_norm_backward(const smc_norm_backward_t* a, void* stream) {
    if (!a) return bad(SMC_ERR_ARG, "args is NULL");
    CHECK(check_common(a->n, a->c, "c", a->dtype));
    if (!(a->eps >= 0.f)) return bad(SMC_ERR_ARG, "eps = %g", (double)a->eps);
    if (!a->weight || ((uintptr_t)a->weight & 1)) return bad(SMC_ERR_ARG, "weight is NULL or misaligned");
    if (!a->dweight || ((uintptr_t)a->dweight & 1)) return bad(SMC_ERR_ARG, "dweight is NULL or misaligned");
    CHECK(check_rows("dy", a->dy, a->n, a->c, a->ld_dy));
    CHECK(check_rows("s", a->s, a->n, a->c, a->lds));
    if (a->ds) CHECK(check_rows("ds", a->ds, a->n, a->c, a->ld_ds));
    CHECK(check_rows("dx", a->dx, a->n, a->c, a->ld_dx));
    const size_t need = smc_rms_norm_backward_workspace(a->n, a->c);
    if (a->n > 0 && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need))
        return bad(SMC_ERR_ARG, "workspace: %zu bytes at %p, %zu needed, 16-byte aligned",
                   a->workspace_bytes, a->workspace, need);
    NormArgs p;
    p.n = a->n;
    p.c = a->c;
    p.eps = a->eps;
    p.x = a->s;
    p.ldx = a->lds;
    p.residual = a->ds;
    p.ldr = a->ld_ds;
    p.weight = a->weight;
    p.y = a->dx;
    p.ldy = a->ld_dx;
    p.dy = a->dy;
    p.lddy = a->ld_dy;
    p.dweight = a->dweight;
    p.part = static_cast<float*>(a->workspace);
    p.vec = a->c % 8 == 0 && words16(a->s, a->lds) && words16(a->dy, a->ld_dy) &&
            (!a->ds || words16(a->ds, a->ld_ds)) && words16(a->dx, a->ld_dx) && aligned16(a->weight);
    return hip_status(launch_norm_backward(p, a->dtype, (hipStream_t)stream), "smc_rms_norm_backward");
}

int smc_linear(const smc_product_t* a, void* stream) { return forward(a, 1, kEpiStore, stream); }
int smc_gated(const smc_product_t* a, void* stream) { return forward(a, 2, kEpiGated, stream); }
int smc_linear_backward(const smc_product_t* a, void* stream) { return backward(a, 1, stream); }
int smc_gated_backward(const smc_product_t* a, void* stream) { return backward(a, 2, stream); }
size_t smc_linear_workspace(const smc_product_t* a) { return forward_workspace_of(a, 1); }
size_t smc_gated_workspace(const smc_product_t* a) { return forward_workspace_of(a, 2); }
size_t smc_linear_backward_workspace(const smc_product_t* a) { return workspace_of(a, 1); }
size_t smc_gated_backward_workspace(const smc_product_t* a) { return workspace_of(a, 2); }

int smc_weight_quantize(const void* w, int64_t ldw, int c_in, int c_out, int dtype, void* q,
                        int64_t ldq, float* scale, void* stream) {
    CHECK(check_common(0, c_in, "c_in", dtype));
    if (c_out < 1 || c_out > kMaxDim) return bad(SMC_ERR_ARG, "c_out = %d outside [1, 2^21]", c_out);
    CHECK(check_rows("w", w, c_in, c_out, ldw));
    if (!q || !scale) return bad(SMC_ERR_ARG, "NULL pointer");
    if (ldq < c_in || ldq > kMaxDim) return bad(SMC_ERR_ARG, "row distance of q is %lld", (long long)ldq);
    return hip_status(launch_quantize_weight(w, ldw, c_in, c_out, q, ldq, scale, dtype, (hipStream_t)stream),
                      "smc_weight_quantize");
}

}  // extern "C"
