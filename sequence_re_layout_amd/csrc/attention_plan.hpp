// attention_plan.hpp -- the plan of attention on head shards, in plain C++.
#pragma once

#include <cstdint>

#ifndef BASP_HD
#define BASP_HD
#endif
#include "basp.h"
#include "fastdiv.hpp"

struct basp_attention_plan {
    // of the layout
    int32_t B, P, Bl, Hl_q, Hl_kv, d;
    int64_t S;
    basp_layout layout;
    basp_dtype dtype;
    int32_t es, shards, ratio;      // ratio: query heads of a key head
    // arguments: window as given, window and sinks as the kernels take them
    int64_t queries, window;
    int32_t sinks, reach, firsts;
    int64_t q_elems, kv_elems, lse_elems;
    // strides in bytes
    int64_t q_token, q_head, q_shard, kv_token, kv_head, kv_shard;
    basp::FastDiv by_ratio;
    // forward pass: columns (query, head of a group) of a work-group, its
    // blocks of a key head, and work-groups that share the keys of a block
    int32_t columns, blocks, splits;
    // gradient of keys and values: key blocks of a key head, the first of them
    // with sinks; parts of a group's heads; of the two kinds of blocks, queries that
    // a work-group takes, and such chunks of all parts
    int32_t key_blocks, sink_blocks, head_parts, sink_chunk, sink_chunks, chunk, chunks;
    int32_t grad_blocks;            // blocks of columns of a key head
    int32_t grad_units;             // waves of them, each of which leaves two numbers in fp16
    int64_t partials_at;            // in the gradient's workspace, after two numbers a row and those
    int64_t workspace_bytes, grad_workspace_bytes;
};

namespace basp {

constexpr int kTileColumns = 128;   // columns of a work-group whose waves share the keys
constexpr int kStepColumns = 32;    // of one whose waves share the columns
constexpr int kKeyBlock = 128;      // keys of a work-group of the gradient of keys and values

// Numbers of one work-group's unfinished result: 32 columns of `channels` sums,
// the running maximum and the sum of each.
inline int padded_channels(int d) { return d <= 64 ? 64 : 128; }
BASP_HD constexpr int64_t step_partial(int channels) { return int64_t{kStepColumns} * (channels + 2); }

}  // namespace basp
