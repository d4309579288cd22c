// mk_linear: the entry points of the linear map (kernels and plans in mk_linear.cuh).
#include "mk_linear.cuh"

using namespace mk;

extern "C" mk_status mk_linear(const mk_linear_args* a, void* stream) {
    mk_status st = linear_check(a);
    if (st != MK_OK || a->rows == 0) return st;
    LinearParams p{};
    LinearChoice<false> c;
    if ((st = linear_plan(a, LinearNamed{}, p, c)) != MK_OK) return st;
    return c.launch(a, p, LinearExtra<false>{}, c.plan, static_cast<cudaStream_t>(stream));
}

extern "C" mk_status mk_linear_plan(const mk_linear_args* a, int32_t* plan) {
    if (!plan) return fail(MK_ERR_ARG, "null argument");
    mk_status st = linear_check(a);
    if (st != MK_OK) return st;
    if (a->rows == 0) return fail(MK_ERR_ARG, "linear: no rows, no plan");
    LinearParams p{};
    LinearChoice<false> c;
    if ((st = linear_plan(a, LinearNamed{}, p, c)) != MK_OK) return st;
    const int32_t out[6] = {c.unit, c.features, c.tokens, c.plan.split, c.plan.tiles_n * c.plan.tiles_m, int32_t(c.plan.clusters)};
    for (int i = 0; i < 6; ++i) plan[i] = out[i];
    return MK_OK;
}
