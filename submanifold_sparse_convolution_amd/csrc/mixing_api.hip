// C entries of the operators that mix rows: argument checks, scratch layout and
// launches. See include/smconv.h for the contract of each call.
#include "api_checks.h"
#include "mixing.h"

using namespace smc;

namespace {

bool odd(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

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
    if (!backward) {
        CHECK(check_rows("y", a->y, a->n, a->c, a->ldy));
        if (over(a->y, a->ldy, a->x, a->ldx)) return bad(SMC_ERR_ARG, "y shares memory with x");
        return SMC_OK;
    }
    if (!a->stats) return bad(SMC_ERR_ARG, "stats is NULL");
    CHECK(check_rows("dy", a->dy, a->n, a->c, a->ld_dy));
    CHECK(check_rows("dx", a->dx, a->n, a->c, a->ld_dx));
    if (!a->dweight || odd(a->dweight, 2)) return bad(SMC_ERR_ARG, "dweight is NULL or misaligned");
    if (!a->dbias || odd(a->dbias, 2)) return bad(SMC_ERR_ARG, "dbias is NULL or misaligned");
    if (over(a->dx, a->ld_dx, a->x, a->ldx)) return bad(SMC_ERR_ARG, "dx shares memory with x");
    if (over(a->dx, a->ld_dx, a->dy, a->ld_dy)) return bad(SMC_ERR_ARG, "dx shares memory with dy");
    return SMC_OK;
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

}  // namespace

extern "C" {

int smc_group_norm(const smc_group_norm_t* a, void* stream) { return group(a, false, stream); }
int smc_group_norm_backward(const smc_group_norm_t* a, void* stream) { return group(a, true, stream); }
size_t smc_group_norm_workspace(const smc_group_norm_t* a) { return group_workspace(a, false); }
size_t smc_group_norm_backward_workspace(const smc_group_norm_t* a) { return group_workspace(a, true); }

}  // extern "C"
