// dg_tree.cuh -- a checked call of dg_tree_attention or dg_sink_attention, and the path for few rows.
#pragma once

#include "dg_paged.cuh"

namespace dghost {

struct TreeCall {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int32_t* cu_q;
    const uint32_t* mask;       // null: causal
    const int32_t* positions;   // null without a window, and when causal
    int64_t total_q;
    int32_t n_seq, max_q_len, Hq, Hkv, mask_words, window, sinks;   // sinks 0 without a window
    float scale;
    dg::PagedKV kv;
};

size_t tree_split_bytes(int32_t max_q_len, int32_t group, int32_t D);
dg_status tree_split(const TreeCall& c, int32_t D, void* workspace, cudaStream_t stream);

}  // namespace dghost
