/*
 * Host-side check of group norm's, the windows' and window attention's C entries
 * under AddressSanitizer and UndefinedBehaviorSanitizer (built and run by
 * tests/test_mixing_cpu.py, no GPU needed): every call here is refused or reports
 * static information before any GPU work. Exits 0 when every status is the one
 * the header documents.
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

static _Alignas(256) unsigned short buf[1 << 16];

static void group_norm(void) {
    void* const x = buf, * const y = buf + 4096, * const w = buf + 8192, * const dy = buf + 12288, * const odd = (char*)buf + 1;
    smc_group_norm_t n;
    memset(&n, 0, sizeof n);
    n.n = 4; n.c = 16; n.groups = 4; n.samples = 1; n.eps = 1e-5f;
    n.x = x; n.ldx = 16; n.weight = w; n.bias = w; n.y = y; n.ldy = 16;
    EXPECT(smc_group_norm_workspace(NULL), 0);
    EXPECT(smc_group_norm_workspace(&n) > 0, 1);
    EXPECT(smc_group_norm_backward_workspace(&n) >= smc_group_norm_workspace(&n) + 16 * 8, 1);
    n.workspace = buf + 16384; n.workspace_bytes = sizeof buf - 32768;
    EXPECT(smc_group_norm(NULL, NULL), SMC_ERR_ARG);
    EXPECT(smc_group_norm_backward(NULL, NULL), SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, n, -1, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, n, (int64_t)1 << 31, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, c, 0, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, dtype, SMC_DTYPE_E4M3, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, groups, 0, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, groups, 5, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, groups, -4, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, samples, 0, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, samples, 2, SMC_ERR_ARG);            /* without offsets */
    REFUSED(smc_group_norm, n, offsets, odd, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, activation, 7, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, eps, -1.f, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, eps, NAN, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, weight, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, bias, odd, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, stats, (float*)((char*)buf + 2), SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, x, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, x, odd, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, ldx, 15, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, ldx, ((int64_t)1 << 21) + 1, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, y, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, y, (char*)x + 32, SMC_ERR_ARG);      /* row r over row r + 1 */
    REFUSED(smc_group_norm, n, workspace, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, workspace, (char*)buf + 8, SMC_ERR_ARG);
    REFUSED(smc_group_norm, n, workspace_bytes, 8, SMC_ERR_ARG);
    smc_group_norm_t wide = n;
    wide.c = wide.ldx = wide.ldy = 8200;
    EXPECT(smc_group_norm(&wide, NULL), SMC_ERR_UNSUPPORTED);
    wide.c = wide.groups = wide.ldx = wide.ldy = 4099;
    EXPECT(smc_group_norm(&wide, NULL), SMC_ERR_UNSUPPORTED);
    EXPECT(smc_group_norm_workspace(&wide), 0);

    n.dy = dy; n.ld_dy = 16; n.dx = y; n.ld_dx = 16; n.dweight = n.dbias = buf + 4000; n.stats = (float*)(buf + 3000);
    REFUSED(smc_group_norm_backward, n, stats, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dy, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dx, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dx, (char*)x + 2, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dx, (char*)dy + 32, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, ld_dx, 15, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dweight, NULL, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, dbias, odd, SMC_ERR_ARG);
    REFUSED(smc_group_norm_backward, n, workspace_bytes, 64, SMC_ERR_ARG);
}

static smc_windows_t windows(void) {
    smc_windows_t w;
    memset(&w, 0, sizeof w);
    w.n = 8; w.windows = 2; w.offsets = (const int32_t*)buf;
    w.plan = buf + 32768; w.plan_bytes = smc_windows_bytes(8, 2);
    return w;
}

static void windows_build(void) {
    EXPECT(smc_windows_bytes(-1, 0), 0);
    EXPECT(smc_windows_bytes(0, -1), 0);
    EXPECT(smc_windows_bytes((int64_t)1 << 31, 1), 0);
    EXPECT(smc_windows_bytes(1, (int64_t)1 << 25), 0);
    EXPECT(smc_windows_bytes(0, 0) > 0, 1);
    EXPECT(smc_windows_bytes(1000, 10) > smc_windows_bytes(1000, 0), 1);
    smc_windows_t w = windows();
    EXPECT(smc_windows_build(NULL, NULL), SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, n, -1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, n, ((int64_t)1 << 31) - 1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, windows, -1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, windows, (1 << 24) + 1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, offsets, NULL, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, offsets, (const int32_t*)((char*)buf + 2), SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, order, (const int32_t*)((char*)buf + 2), SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, coords, (const int32_t*)((char*)buf + 2), SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, plan, NULL, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, plan, (char*)buf + 8, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, plan_bytes, w.plan_bytes - 1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, w, ex, 4, SMC_ERR_ARG);               /* one axis alone */
    smc_windows_t c = w;
    c.ex = c.ey = c.ez = 4;
    EXPECT(smc_windows_build(&c, NULL), SMC_ERR_ARG);                /* no coords */
    c.coords = (const int32_t*)buf;
    EXPECT(smc_windows_build(&c, NULL), SMC_ERR_ARG);                /* of no columns */
    c.coord_cols = 4;
    REFUSED(smc_windows_build, c, ex, 0, SMC_ERR_ARG);
    REFUSED(smc_windows_build, c, ey, -1, SMC_ERR_ARG);
    REFUSED(smc_windows_build, c, ez, 121, SMC_ERR_UNSUPPORTED);     /* 124 and 4 and 4 */
    REFUSED(smc_windows_build, c, ex, 0x7fffffff, SMC_ERR_UNSUPPORTED);
    c.ex = c.ey = c.ez = 0;
    EXPECT(smc_windows_build(&c, NULL), SMC_ERR_ARG);                /* coords without an extent */
}

static void attention(void) {
    smc_windows_t w = windows();
    smc_attention_t a;
    memset(&a, 0, sizeof a);
    a.windows = &w; a.heads = 4; a.kv_heads = 2; a.head_dim = 16; a.scale = 0.25f;
    a.q = buf; a.ldq = 128; a.k = buf + 64; a.ldk = 128; a.v = buf + 96; a.ldv = 128;
    a.out = buf + 2048; a.ld_out = 64;
    EXPECT(smc_window_attention(NULL, NULL), SMC_ERR_ARG);
    EXPECT(smc_window_attention(&a, NULL), SMC_ERR_STATE);           /* not built */
    w.tiles32 = w.tiles64 = w.tiles128 = 2; w.longest = 4; w.pairs = 32;
    REFUSED(smc_window_attention, a, windows, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, heads, 0, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, kv_heads, 0, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, kv_heads, 3, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, head_dim, 0, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, head_dim, 129, SMC_ERR_UNSUPPORTED);
    REFUSED(smc_window_attention, a, dtype, SMC_DTYPE_E4M3, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, scale, 0.f, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, scale, NAN, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, scale, INFINITY, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, q, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, ldq, 63, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, k, (char*)buf + 1, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, ldk, 31, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, v, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, out, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, out, buf, SMC_ERR_ARG);         /* over q */
    REFUSED(smc_window_attention, a, out, buf + 70, SMC_ERR_ARG);    /* over k */
    REFUSED(smc_window_attention, a, lse, (float*)((char*)buf + 2), SMC_ERR_ARG);
    REFUSED(smc_window_attention, a, bias, buf, SMC_ERR_STATE);      /* windows without cells */
    w.ex = w.ey = w.ez = 4;
    smc_attention_t b = a;
    b.bias = buf + 20000;
    EXPECT(smc_window_attention(&b, NULL), SMC_ERR_ARG);             /* reach 0 */
    REFUSED(smc_window_attention, b, reach, 128, SMC_ERR_ARG);
    b.reach = 2;
    REFUSED(smc_window_attention, b, bias, (char*)buf + 1, SMC_ERR_ARG);
    w.tiles32 = 0x7fffffff;
    EXPECT(smc_window_attention(&b, NULL), SMC_ERR_UNSUPPORTED);
    w.tiles32 = 2;

    b.lse = (float*)(buf + 22000); b.dout = buf + 4096; b.ld_dout = 64;
    b.dq = buf + 8192; b.ld_dq = 128; b.dk = buf + 8192 + 64; b.ld_dk = 128; b.dv = buf + 8192 + 96; b.ld_dv = 128;
    b.dbias = buf + 24000;
    EXPECT(smc_window_attention_backward_workspace(NULL), 0);
    b.workspace_bytes = smc_window_attention_backward_workspace(&b);
    EXPECT(b.workspace_bytes >= 4 * 8 * 4 + 2 * 4 * 15 * 4, 1);
    b.workspace = buf + 26000;
    REFUSED(smc_window_attention_backward, b, lse, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dout, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dq, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dk, b.dq, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dv, b.dk, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dq, buf, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dv, buf + 4096, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, ld_dq, 63, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, dbias, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, workspace, NULL, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, workspace, (char*)b.workspace + 8, SMC_ERR_ARG);
    REFUSED(smc_window_attention_backward, b, workspace_bytes, b.workspace_bytes - 1, SMC_ERR_ARG);
    /* the scratch size reads no pointer and no distance */
    smc_attention_t c = b;
    c.q = c.k = c.v = c.out = c.dq = NULL;
    c.ldq = c.ldk = c.head_dim = 0;
    EXPECT(smc_window_attention_backward_workspace(&c), b.workspace_bytes);
}

int main(void) {
    group_norm();
    windows_build();
    attention();
    if (failures) {
        fprintf(stderr, "%d check(s) failed\n", failures);
        return 1;
    }
    printf("mixing operators abi check ok\n");
    return 0;
}
