// attention_plan.cpp -- host side of attention on head shards: plans, sizes,
// limits, and how the work is split.  No device calls.
#include <algorithm>
#include <cstring>
#include <new>

#include "attention_plan.hpp"
#include "plan_internal.hpp"

using basp::record;

namespace {

constexpr int64_t kGroups = (int64_t{1} << 24) - 1;     // work-groups of one launch: 32-bit global size
constexpr int kWanted = 512;                            // work-groups that fill the device twice

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

basp_attention_plan *refuse(basp_status s)
{
    record(s);
    return nullptr;
}

}  // namespace

extern "C" basp_attention_plan *basp_attention_plan_create(const basp_plan *layout, int64_t queries, int64_t window,
                                                           int64_t sinks)
{
    if (!layout || window < 1 || sinks < 0 || queries < (layout->S ? 1 : 0) || queries > layout->S)
        return refuse(BASP_ERR_INVALID);
    if (layout->Hq % layout->Hkv)
        return refuse(BASP_ERR_INDIVISIBLE);
    if (layout->dtype == BASP_INT32 || layout->d > 128 || layout->S >= int64_t{1} << 29)
        return refuse(BASP_ERR_UNSUPPORTED);
    const int64_t ratio = layout->Hl_q / layout->Hl_kv, shards = int64_t{layout->N} * layout->Bl;
    const int64_t pairs = shards * layout->Hl_kv, token = int64_t{layout->Hl_q} * layout->d * layout->es;
    // in token order a tile's rows are within 31 bits of its first; one limit for both orders
    if (ratio * queries >= int64_t{1} << 30 || pairs > kGroups || token > int64_t{1} << 24)
        return refuse(BASP_ERR_UNSUPPORTED);

    basp_attention_plan r;
    std::memset(static_cast<void *>(&r), 0, sizeof(r));
    r.B = layout->B;
    r.P = layout->P;
    r.Bl = layout->Bl;
    r.Hl_q = layout->Hl_q;
    r.Hl_kv = layout->Hl_kv;
    r.d = layout->d;
    r.S = layout->S;
    r.layout = layout->layout;
    r.dtype = layout->dtype;
    r.es = layout->es;
    r.shards = int32_t(shards);
    r.ratio = int32_t(ratio);
    r.queries = queries;
    r.window = window;
    r.sinks = int32_t(std::min<int64_t>(sinks, INT32_MAX));
    // window and sinks that cover the cache: all earlier keys
    const bool all = window >= r.S || sinks >= r.S - window;
    r.reach = int32_t(all ? std::max<int64_t>(1, r.S) : window);
    r.firsts = int32_t(all ? 0 : sinks);
    r.q_elems = shards * r.Hl_q * queries * r.d;
    r.kv_elems = shards * r.Hl_kv * r.S * r.d;
    r.lse_elems = shards * r.Hl_q * queries;
    const int64_t row = int64_t{r.d} * r.es;
    const bool heads_first = r.layout == BASP_LAYOUT_HEAD_MAJOR;
    r.q_token = heads_first ? row : r.Hl_q * row;
    r.q_head = heads_first ? queries * row : row;
    r.q_shard = r.Hl_q * queries * row;
    r.kv_token = heads_first ? row : r.Hl_kv * row;
    r.kv_head = heads_first ? r.S * row : row;
    r.kv_shard = r.Hl_kv * r.S * row;
    r.by_ratio = basp::make_fastdiv(uint32_t(ratio));

    // Forward pass.  Keys that a block of queries sees, at most.
    const int64_t cols = ratio * queries;
    const int64_t seen = std::min(r.S, int64_t{r.reach} + r.firsts + std::min(queries, ceil_div(basp::kTileColumns, ratio)));
    const int64_t tile_blocks = std::max<int64_t>(1, ceil_div(cols, basp::kTileColumns));
    r.columns = basp::kTileColumns;
    r.splits = 1;
    // Few columns, or few work-groups for the keys that there are: the waves of a
    // work-group share a block of 32 columns, and work-groups share its keys.  In 16
    // bits that pays from about 1024 keys on (two sequences of 900, 128 channels: 25
    // us, 30 us this way), in fp32 always (5 queries of 8 heads, 305 keys: 52 us, 20).
    const bool slow = r.es == 4;    // 32 keys take as long as 512 in 16 bits
    if (cols <= basp::kStepColumns || (pairs * tile_blocks < kWanted / 4 && seen >= (slow ? 64 : 1024))) {
        r.columns = basp::kStepColumns;
        const int64_t groups = pairs * std::max<int64_t>(1, ceil_div(cols, basp::kStepColumns));
        // at least 256 keys a work-group: two tiles a wave; in fp32 one
        r.splits = int32_t(std::max<int64_t>(1, std::min({ceil_div(kWanted, groups), ceil_div(seen, slow ? 128 : 256), int64_t{256}})));
    }
    const int64_t blocks = std::max<int64_t>(1, ceil_div(cols, r.columns));
    if (blocks * r.splits > kGroups / pairs)
        return refuse(BASP_ERR_UNSUPPORTED);
    r.blocks = int32_t(blocks);
    if (r.splits > 1)
        r.workspace_bytes = pairs * blocks * r.splits * basp::step_partial(basp::padded_channels(r.d)) * 4;

    // Gradient.  A block of keys takes the queries that see one of them: those of
    // the window, or all after it where it holds sinks.  Queries are cut into
    // chunks where the blocks alone would not fill the device, and those of a
    // block with sinks so that it takes no longer than the others.  A chunk's sums
    // go through memory, which pays for 256 queries, in fp32 (a sixteenth of the
    // rate) for 64, and with twice the work-groups.  Two whole sequences of 2048 in
    // bf16: 296 us; 339 us with half as many chunks, 307 us with twice as many.
    const int64_t key_blocks = ceil_div(std::max<int64_t>(1, r.S), basp::kKeyBlock);
    const int64_t sink_blocks = ceil_div(r.firsts, basp::kKeyBlock);
    const int64_t in_window = std::max<int64_t>(1, std::min(queries, int64_t{r.reach} + basp::kKeyBlock));
    const int64_t least = r.es == 4 ? 64 : 256;
    const auto cut = [&](int64_t n, int64_t parts) { return std::max(least, ceil_div(ceil_div(n, parts), 64) * 64); };
    const int64_t chunk = cut(in_window, std::max<int64_t>(1, (r.es == 4 ? 2 * kWanted : kWanted) / (pairs * key_blocks)));
    const int64_t sink_chunk = std::max(chunk, cut(queries, ceil_div(2 * kWanted, pairs * std::max<int64_t>(1, sink_blocks))));
    // Where that still leaves few work-groups with long loops, by heads of a group,
    // too: in fp32 those of 64 queries are long (8 queries of 8 heads, 128 channels:
    // 106 us for a gradient, 60 us by heads), in 16 bits those of 256 (a sequence of
    // 1024 of 4 heads a key head: 78 us, 68 us by heads).
    const int64_t whole = sink_blocks * ceil_div(queries, sink_chunk) + (key_blocks - sink_blocks) * ceil_div(in_window, chunk);
    const int64_t rows = std::min(queries, sink_blocks ? sink_chunk : chunk), much = r.es == 4 ? 64 : 256;
    int64_t parts = 1;
    for (int64_t h = 2; h <= ratio && pairs * whole * parts < kWanted / 2 && ceil_div(rows, 32) * 32 * ratio / parts > much; ++h)
        if (ratio % h == 0 && pairs * whole * h <= 4 * kWanted)     // the workspace, too
            parts = h;
    r.key_blocks = int32_t(key_blocks);
    r.sink_blocks = int32_t(sink_blocks);
    r.head_parts = int32_t(parts);
    r.chunk = int32_t(chunk);
    r.chunks = int32_t(ceil_div(in_window, chunk) * parts);
    r.sink_chunk = int32_t(sink_chunk);
    r.sink_chunks = int32_t(std::max<int64_t>(1, ceil_div(queries, sink_chunk)) * parts);
    const int64_t items = sink_blocks * r.sink_chunks + (key_blocks - sink_blocks) * r.chunks;
    r.grad_blocks = int32_t(tile_blocks);
    if (items > kGroups / pairs || tile_blocks > kGroups / pairs)
        return refuse(BASP_ERR_UNSUPPORTED);
    r.grad_units = r.dtype == BASP_FP16 ? int32_t(ceil_div(cols, 32)) : 0;
    r.partials_at = ceil_div(r.lse_elems * 8 + pairs * r.grad_units * 8, 256) * 256;
    const int64_t unfinished = (r.sink_chunks > 1 ? sink_blocks * r.sink_chunks : 0) +
                               (r.chunks > 1 ? (key_blocks - sink_blocks) * r.chunks : 0);
    r.grad_workspace_bytes = r.partials_at +
                             pairs * unfinished * 2 * basp::kKeyBlock * basp::padded_channels(r.d) * 4;

    basp_attention_plan *p = new (std::nothrow) basp_attention_plan(r);
    if (!p)
        return refuse(BASP_ERR_UNSUPPORTED);
    record(BASP_OK);
    return p;
}

extern "C" void basp_attention_plan_destroy(basp_attention_plan *plan)
{
    delete plan;
    record(BASP_OK);
}

extern "C" basp_status basp_attention_plan_query(const basp_attention_plan *p, basp_attention_info *info)
{
    if (!p || !info)
        return record(BASP_ERR_INVALID);
    basp_attention_info r;
    std::memset(&r, 0, sizeof(r));
    r.S = p->S;
    r.queries = p->queries;
    r.window = p->window;
    r.sinks = p->sinks;
    r.shards = p->shards;
    r.B = p->B;
    r.Hl_q = p->Hl_q;
    r.Hl_kv = p->Hl_kv;
    r.d = p->d;
    r.layout = p->layout;
    r.dtype = p->dtype;
    r.q_elems = p->q_elems;
    r.kv_elems = p->kv_elems;
    r.lse_elems = p->lse_elems;
    r.workspace_bytes = p->workspace_bytes;
    r.grad_workspace_bytes = p->grad_workspace_bytes;
    *info = r;
    return record(BASP_OK);
}
