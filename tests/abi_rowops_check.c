/*
 * Host-side check of the row operators' C entries under AddressSanitizer and
 * UndefinedBehaviorSanitizer (built and run by tests/test_rowops_abi_cpu.py, no
 * GPU needed): every call here is refused or reports static information before
 * any GPU work. Exits 0 when every status is the one the header documents.
 */
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "smconv.h"

static int failures = 0;

#define EXPECT(expr, want)                                                                \
    do {                                                                                  \
        long long got_ = (long long)(expr);                                               \
        if (got_ != (long long)(want)) {                                                  \
            fprintf(stderr, "%s:%d: %s = %lld, want %lld (%s)\n", __FILE__, __LINE__,     \
                    #expr, got_, (long long)(want), smc_last_error());                    \
            ++failures;                                                                   \
        }                                                                                 \
    } while (0)

/* a refused call with one field changed */
#define REFUSED(call, good, field, value, want) \
    do {                                        \
        __typeof__(good) a_ = good;             \
        a_.field = value;                       \
        EXPECT(call(&a_, NULL), want);          \
    } while (0)

int main(void) {
    static unsigned short buf[4096];
    static float f32[64];
    void* const p = buf;
    void* const odd = (char*)buf + 1;
    const int64_t far = ((int64_t)1 << 21) + 1;

    smc_norm_t n;
    memset(&n, 0, sizeof n);
    n.n = 4; n.c = 16; n.eps = 1e-6f;
    n.x = p; n.ldx = 16; n.weight = p; n.y = p; n.ldy = 16;
    EXPECT(smc_rms_norm(NULL, NULL), SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, n, -1, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, n, (int64_t)1 << 31, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, c, 0, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, c, (1 << 21) + 1, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, dtype, SMC_DTYPE_E4M3, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, eps, -1.f, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, eps, NAN, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, x, NULL, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, x, odd, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, ldx, 15, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, ldx, far, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, weight, NULL, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, y, NULL, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, ldy, 15, SMC_ERR_ARG);
    REFUSED(smc_rms_norm, n, residual, p, SMC_ERR_ARG);     /* ld_residual is 0 */
    REFUSED(smc_rms_norm, n, s, p, SMC_ERR_ARG);

    smc_norm_backward_t nb;
    memset(&nb, 0, sizeof nb);
    nb.n = 4; nb.c = 16; nb.eps = 1e-6f;
    nb.dy = p; nb.ld_dy = 16; nb.s = p; nb.lds = 16; nb.weight = p;
    nb.dx = p; nb.ld_dx = 16; nb.dweight = p; nb.workspace = f32; nb.workspace_bytes = 0;
    EXPECT(smc_rms_norm_backward(NULL, NULL), SMC_ERR_ARG);
    EXPECT(smc_rms_norm_backward(&nb, NULL), SMC_ERR_ARG);          /* no workspace */
    REFUSED(smc_rms_norm_backward, nb, dweight, NULL, SMC_ERR_ARG);
    REFUSED(smc_rms_norm_backward, nb, dy, NULL, SMC_ERR_ARG);
    REFUSED(smc_rms_norm_backward, nb, ld_dx, 8, SMC_ERR_ARG);
    EXPECT(smc_rms_norm_backward_workspace(4, 16) >= 4 * 16 * 4, 1);
    EXPECT(smc_rms_norm_backward_workspace(0, 16), 0);
    EXPECT(smc_rms_norm_backward_workspace(-1, 16), 0);
    EXPECT(smc_rms_norm_backward_workspace(4, 0), 0);

    smc_product_t a;
    memset(&a, 0, sizeof a);
    a.n = 4; a.c_in = 16; a.c_out = 8;
    a.x = p; a.ldx = 16; a.w = p; a.ldw = 16; a.y = p; a.ldy = 8;
    int (*forward[2])(const smc_product_t*, void*) = {smc_linear, smc_gated};
    for (int i = 0; i < 2; ++i) {
        EXPECT(forward[i](NULL, NULL), SMC_ERR_ARG);
        REFUSED(forward[i], a, n, -1, SMC_ERR_ARG);
        REFUSED(forward[i], a, c_in, 0, SMC_ERR_ARG);
        REFUSED(forward[i], a, c_out, 0, SMC_ERR_ARG);
        REFUSED(forward[i], a, c_out, (1 << 21) + 1, SMC_ERR_ARG);
        REFUSED(forward[i], a, dtype, 7, SMC_ERR_ARG);
        REFUSED(forward[i], a, x_dtype, SMC_DTYPE_F16, SMC_ERR_ARG);
        REFUSED(forward[i], a, x_dtype, SMC_DTYPE_E4M3, SMC_ERR_ARG);      /* no scales */
        REFUSED(forward[i], a, w_transposed, 1, SMC_ERR_UNSUPPORTED);
        REFUSED(forward[i], a, activation, 4, SMC_ERR_ARG);
        REFUSED(forward[i], a, x, NULL, SMC_ERR_ARG);
        REFUSED(forward[i], a, ldx, 8, SMC_ERR_ARG);
        REFUSED(forward[i], a, w, NULL, SMC_ERR_ARG);
        REFUSED(forward[i], a, w, odd, SMC_ERR_ARG);
        REFUSED(forward[i], a, ldw, 7, SMC_ERR_ARG);
        REFUSED(forward[i], a, bias, odd, SMC_ERR_ARG);
        REFUSED(forward[i], a, y, NULL, SMC_ERR_ARG);
        REFUSED(forward[i], a, ldy, 7, SMC_ERR_ARG);
    }
    REFUSED(smc_linear, a, residual, p, SMC_ERR_ARG);               /* ld_residual is 0 */
    REFUSED(smc_gated, a, residual, p, SMC_ERR_ARG);
    REFUSED(smc_gated, a, ldw, 15, SMC_ERR_ARG);                    /* two halves of 8 */
    {
        smc_product_t big = a;
        big.c_in = 1 << 12;
        big.ldx = 1 << 12;
        big.ldw = (int64_t)1 << 19;
        EXPECT(smc_linear(&big, NULL), SMC_ERR_UNSUPPORTED);        /* w spans 2^32 bytes */
        EXPECT(strstr(smc_last_error(), "2^31") != NULL, 1);
    }

    a.dy = p; a.ld_dy = 8; a.dx = p; a.ld_dx = 16; a.dw = p; a.ld_dw = 16;
    int (*back[2])(const smc_product_t*, void*) = {smc_linear_backward, smc_gated_backward};
    size_t (*need[2])(const smc_product_t*) = {smc_linear_backward_workspace, smc_gated_backward_workspace};
    for (int i = 0; i < 2; ++i) {
        EXPECT(back[i](NULL, NULL), SMC_ERR_ARG);
        EXPECT(back[i](&a, NULL), SMC_ERR_ARG);                     /* no workspace */
        REFUSED(back[i], a, dy, NULL, SMC_ERR_ARG);
        REFUSED(back[i], a, dx, NULL, SMC_ERR_ARG);
        REFUSED(back[i], a, dw, NULL, SMC_ERR_ARG);
        REFUSED(back[i], a, ld_dw, 7, SMC_ERR_ARG);
        REFUSED(back[i], a, residual, p, SMC_ERR_ARG);
        REFUSED(back[i], a, x_dtype, SMC_DTYPE_E4M3, SMC_ERR_UNSUPPORTED);
        EXPECT(need[i](NULL), 0);
        EXPECT(need[i](&a) >= (size_t)16 * 8 * 4, 1);
        size_t (*room[2])(const smc_product_t*) = {smc_linear_workspace, smc_gated_workspace};
        EXPECT(room[i](NULL), 0);
    }

    EXPECT(smc_weight_quantize(NULL, 8, 16, 8, SMC_DTYPE_BF16, p, 16, f32, NULL), SMC_ERR_ARG);
    EXPECT(smc_weight_quantize(p, 7, 16, 8, SMC_DTYPE_BF16, p, 16, f32, NULL), SMC_ERR_ARG);
    EXPECT(smc_weight_quantize(p, 8, 16, 8, SMC_DTYPE_E4M3, p, 16, f32, NULL), SMC_ERR_ARG);
    EXPECT(smc_weight_quantize(p, 8, 16, 8, SMC_DTYPE_BF16, p, 15, f32, NULL), SMC_ERR_ARG);
    EXPECT(smc_weight_quantize(p, 8, 16, 8, SMC_DTYPE_BF16, NULL, 16, f32, NULL), SMC_ERR_ARG);

    if (failures) {
        fprintf(stderr, "%d check(s) failed\n", failures);
        return 1;
    }
    printf("row operators abi check ok\n");
    return 0;
}
