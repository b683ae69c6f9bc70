// layer_plan.cpp -- host side of the layer norm: plans, sizes and limits.  No
// device calls.
#include <algorithm>
#include <cstring>
#include <new>

#include "layer_plan.hpp"
#include "plan_internal.hpp"

using basp::record;

namespace {

constexpr int64_t kRowLimit = int64_t{1} << 30;     // bytes of a row
constexpr int64_t kIndexLimit = 0x7fffffff - 1;     // rows

}  // namespace

extern "C" basp_norm_plan *basp_norm_plan_create(int64_t T, int64_t D, basp_dtype dtype, basp_dtype weight_dtype)
{
    const int es = basp::float_bytes(dtype), wes = basp::float_bytes(weight_dtype);
    if (T < 0 || D < 1 || !es || !wes) {
        record(BASP_ERR_INVALID);
        return nullptr;
    }
    if (T > kIndexLimit || D >= kRowLimit / 4) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    basp_norm_plan *p = new (std::nothrow) basp_norm_plan;
    if (!p) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    std::memset(static_cast<void *>(p), 0, sizeof(*p));
    p->T = T;
    p->D = D;
    p->dtype = dtype;
    p->weight_dtype = weight_dtype;
    p->es = es;
    p->ws_es = wes;
    p->vw = basp::row_vector(D, es);
    p->vecs = (D * es + p->vw - 1) / p->vw;
    // rows of a work-group in one go: a share of its threads for each
    const int64_t at_once = p->vecs <= 16 ? 16 : p->vecs <= 128 ? 4 : p->vecs <= 256 ? 2 : 1;
    p->grad_groups = int32_t(std::min<int64_t>(basp::kNormGradGroups, (T + at_once - 1) / at_once));
    p->width = (D + 3) / 4 * 4;
    p->workspace_bytes = int64_t{8} * p->grad_groups * p->width;
    record(BASP_OK);
    return p;
}

extern "C" void basp_norm_plan_destroy(basp_norm_plan *plan)
{
    delete plan;
    record(BASP_OK);
}

extern "C" basp_status basp_norm_plan_query(const basp_norm_plan *p, basp_norm_info *info)
{
    if (!p || !info)
        return record(BASP_ERR_INVALID);
    basp_norm_info r;
    std::memset(&r, 0, sizeof(r));
    r.T = p->T;
    r.D = p->D;
    r.dtype = p->dtype;
    r.weight_dtype = p->weight_dtype;
    r.workspace_bytes = p->workspace_bytes;
    *info = r;
    return record(BASP_OK);
}

extern "C" size_t basp_balance_workspace_bytes(const basp_expert_plan *p)
{
    if (!p) {
        record(BASP_ERR_INVALID);
        return 0;
    }
    record(BASP_OK);
    // and how many of the work-groups that join them are done, with their results
    return (size_t(basp::balance_groups(*p)) * 2 * basp::balance_stride(*p) + 1 + basp::balance_joins(*p)) * 4;
}
