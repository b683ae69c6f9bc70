// index_plan.cpp -- host side of the index-driven re-layouts: plans, sizes,
// limits and pointer checks.  No device calls.
#include <algorithm>
#include <cstring>
#include <new>

#include "index_plan.hpp"
#include "plan_internal.hpp"

using basp::record;

namespace {

constexpr int64_t kRowLimit = int64_t{1} << 30;     // bytes of a row
constexpr int64_t kIndexLimit = 0x7fffffff - 1;     // slots, rows, tokens: int32 with -1, and 31-bit division
constexpr int64_t kVocabLimit = int64_t{1} << 30;
constexpr int64_t kSumGroups = 1024;                // four work-groups a compute unit
constexpr int64_t kSumLimit = int64_t{1} << 23;     // work-groups of a launch's 32-bit extent

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

// Items per work-group of a sort: at least kSortItems, and more where the call
// would otherwise take over kBlocks groups (each reads the counts of all the
// others).  A multiple of the group's threads, so that waves take whole
// multiples of 64.
void split_sort(int64_t n, int32_t &blocks, int64_t &items)
{
    constexpr int64_t kBlocks = 256;
    items = round_up(std::max<int64_t>(basp::kSortItems, ceil_div(n, kBlocks)), basp::kSortBlock);
    blocks = int32_t(std::max<int64_t>(1, ceil_div(n, items)));
}

}  // namespace

namespace basp {

basp_status check_call(const CallBuf *in, int nin, const CallBuf *out, int nout)
{
    const auto at = [](const CallBuf &b) { return reinterpret_cast<uint64_t>(b.ptr); };
    const auto meet = [&](const CallBuf &a, const CallBuf &b) {
        return a.bytes && b.bytes && at(a) < at(b) + uint64_t(b.bytes) && at(b) < at(a) + uint64_t(a.bytes);
    };
    for (int i = 0; i < nin + nout; ++i) {
        const CallBuf &b = i < nin ? in[i] : out[i - nin];
        if (b.bytes && !b.ptr)
            return BASP_ERR_INVALID;
        if (at(b) % uint64_t(b.align))
            return BASP_ERR_ALIGN;
    }
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i)
            if (meet(out[o], in[i]))
                return BASP_ERR_ALIAS;
        for (int j = 0; j < o; ++j)
            if (meet(out[o], out[j]))
                return BASP_ERR_ALIAS;
    }
    return BASP_OK;
}

}  // namespace basp

extern "C" basp_expert_plan *basp_expert_plan_create(int64_t T, int K, int E, int64_t D, int align, int id_bytes,
                                                     basp_dtype dtype, basp_dtype weight_dtype)
{
    const int es = basp::float_bytes(dtype), wes = basp::float_bytes(weight_dtype);
    if (T < 0 || K < 1 || E < 1 || D < 1 || align < 1 || (id_bytes != 4 && id_bytes != 8) || !es || !wes) {
        record(BASP_ERR_INVALID);
        return nullptr;
    }
    if (E > basp::kMaxExperts || align > 65536 || D >= kRowLimit / es || T > kIndexLimit / K) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    const int64_t slots = T * K;
    const int64_t rows = (slots + std::min<int64_t>(E, slots) * (align - 1)) / align * align;
    if (rows > kIndexLimit) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    basp_expert_plan *p = new (std::nothrow) basp_expert_plan;
    if (!p) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    std::memset(static_cast<void *>(p), 0, sizeof(*p));
    p->T = T;
    p->K = K;
    p->E = E;
    p->D = D;
    p->align = align;
    p->id_bytes = id_bytes;
    p->dtype = dtype;
    p->weight_dtype = weight_dtype;
    p->es = es;
    p->ws_es = wes;
    p->slots = slots;
    p->max_rows = rows;
    split_sort(slots, p->sort_blocks, p->block_items);
    // the counts of every work-group
    p->workspace_bytes = p->sort_blocks > 1 ? int64_t{4} * E * p->sort_blocks : 0;
    record(BASP_OK);
    return p;
}

extern "C" void basp_expert_plan_destroy(basp_expert_plan *plan)
{
    delete plan;
    record(BASP_OK);
}

extern "C" basp_status basp_expert_plan_query(const basp_expert_plan *p, basp_expert_info *info)
{
    if (!p || !info)
        return record(BASP_ERR_INVALID);
    basp_expert_info r;
    std::memset(&r, 0, sizeof(r));
    r.T = p->T;
    r.D = p->D;
    r.K = p->K;
    r.E = p->E;
    r.align = p->align;
    r.id_bytes = p->id_bytes;
    r.dtype = p->dtype;
    r.weight_dtype = p->weight_dtype;
    r.slots = p->slots;
    r.max_rows = p->max_rows;
    r.workspace_bytes = p->workspace_bytes;
    *info = r;
    return record(BASP_OK);
}

extern "C" basp_embed_plan *basp_embed_plan_create(const basp_plan *layout, int64_t T, int64_t V, int64_t D,
                                                   int64_t padding, int id_bytes, basp_dtype dtype,
                                                   basp_dtype grad_dtype)
{
    const int es = basp::float_bytes(dtype), ges = basp::float_bytes(grad_dtype);
    if (T < 0 || V < 1 || D < 1 || padding < -1 || padding >= V || (id_bytes != 4 && id_bytes != 8) || !es || !ges ||
        (layout && T != int64_t{layout->B} * layout->S)) {
        record(BASP_ERR_INVALID);
        return nullptr;
    }
    if (T > kIndexLimit || V > kVocabLimit || D >= kRowLimit / 4) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    // the gradient's sums are one launch of 256-thread work-groups: a team of
    // up to 64 lanes takes one vector of channels each and `chunk` sorted
    // tokens, and the teams of a work-group follow each other.  Short chunks
    // where long ones would leave compute units without a few waves each.
    const int epv = basp::row_vector(D, es) / es;
    const int64_t vecs = ceil_div(D, epv);
    int lanes_log2 = 0;
    while (lanes_log2 < 6 && (int64_t{1} << lanes_log2) < vecs)
        ++lanes_log2;
    const int64_t teams = basp::kSumThreads >> lanes_log2, cols = ceil_div(vecs, int64_t{1} << lanes_log2);
    int chunk = 32;
    while (chunk > 8 && ceil_div(T, chunk * teams) * cols < kSumGroups)
        chunk /= 2;
    const int64_t groups = ceil_div(T, chunk * teams);
    if (groups > kSumLimit / cols) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    basp_embed_plan *p = new (std::nothrow) basp_embed_plan;
    if (!p) {
        record(BASP_ERR_UNSUPPORTED);
        return nullptr;
    }
    std::memset(static_cast<void *>(p), 0, sizeof(*p));
    p->T = T;
    p->V = V;
    p->D = D;
    p->padding = padding;
    p->id_bytes = id_bytes;
    p->dtype = dtype;
    p->grad_dtype = grad_dtype;
    p->es = es;
    p->grad_es = ges;
    basp_seq_order &o = p->order;
    o.same = !layout || T == 0 || layout->P == 1 || layout->Bl == 1;
    o.P = layout ? uint32_t(layout->P) : 1;
    o.Bl = layout ? uint32_t(layout->Bl) : 1;
    o.S = layout && T ? uint32_t(layout->S) : 1;
    o.St = layout && T ? uint32_t(layout->St) : 1;
    o.by_S = basp::make_fastdiv(o.S);
    o.by_Bl = basp::make_fastdiv(o.Bl);
    o.by_St = basp::make_fastdiv(o.St);

    // sort by id, least significant digit first, ignored ids as V: as few
    // passes of at most kDigitBits as the ids need, of equal width
    int bits = 1;
    while ((V >> bits) != 0)
        ++bits;
    p->passes = (bits + basp::kDigitBits - 1) / basp::kDigitBits;
    p->digit_bits = (bits + p->passes - 1) / p->passes;
    split_sort(T, p->sort_blocks, p->block_items);
    if (T <= (basp::fits_narrow(T, V) ? basp::kRankNarrow : basp::kRankWide))
        p->sort_blocks = 0;
    p->lanes_log2 = lanes_log2;
    p->chunk = chunk;
    p->blocks = ceil_div(T, int64_t{chunk} * basp::merged_teams(lanes_log2));
    p->col_groups = int32_t(cols);
    p->sum_groups = groups * cols;
    p->width = vecs * epv;
    int64_t at = 0;
    const auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at = round_up(at + bytes, 256);
        return here;
    };
    if (T) {
        for (int i = 0; i < 2; ++i) {
            p->keys[i] = take(4 * T);
            p->tokens[i] = take(4 * T);
        }
        p->tags = take(4 * V);
        p->hist = take((int64_t{4} << p->digit_bits) * p->sort_blocks);
        p->partials = take(p->blocks * 2 * p->width * 4);
    }
    p->workspace_bytes = at;
    record(BASP_OK);
    return p;
}

extern "C" void basp_embed_plan_destroy(basp_embed_plan *plan)
{
    delete plan;
    record(BASP_OK);
}

extern "C" basp_status basp_embed_plan_query(const basp_embed_plan *p, basp_embed_info *info)
{
    if (!p || !info)
        return record(BASP_ERR_INVALID);
    basp_embed_info r;
    std::memset(&r, 0, sizeof(r));
    r.T = p->T;
    r.V = p->V;
    r.D = p->D;
    r.padding = p->padding;
    r.id_bytes = p->id_bytes;
    r.dtype = p->dtype;
    r.grad_dtype = p->grad_dtype;
    r.workspace_bytes = p->workspace_bytes;
    *info = r;
    return record(BASP_OK);
}
