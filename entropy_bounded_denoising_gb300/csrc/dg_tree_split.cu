// dg_tree_split.cu -- dg_tree_attention and dg_sink_attention for calls of few rows a key head: the kernels of
// dg_paged_split.cuh with the trees' masks and the first tokens that stay visible.
#include <cuda_runtime.h>

#include <math.h>

#include "dg_paged_split.cuh"
#include "dg_tree.cuh"

namespace dghost {

size_t tree_split_bytes(int32_t max_q_len, int32_t group, int32_t D) { return split_bytes(item_rows(max_q_len, group), D); }

dg_status tree_split(const TreeCall& c, int32_t D, void* workspace, cudaStream_t st) {
    TreeSplitArgs a;
    const int rows = item_rows(c.max_q_len, c.Hq / c.Hkv);
    a.q = c.q;
    a.o = c.o;
    a.lse = c.lse;
    a.cu_q = c.cu_q;
    a.causal = nullptr;
    a.total_q = c.total_q;
    a.n_seq = c.n_seq;
    a.max_q_len = c.max_q_len;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.group = c.Hq / c.Hkv;
    a.window = c.window;
    a.scale_log2 = c.scale * kLog2e;
    a.kv = c.kv;
    a.mask = c.mask;
    a.positions = c.positions;
    a.mask_words = c.mask_words;
    a.sinks = c.sinks;
    a.desc = static_cast<int4*>(workspace);
    a.part_o = reinterpret_cast<float*>(a.desc + 2 * kMaxCtas);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + (size_t)kMaxCtas * 2 * rows * D);
    a.status = status_word();
    if (in_pairs(c.max_q_len, a.group, a.Hkv, D)) {
        a.Hkv /= 2;
        a.group *= 2;
        return launch_split<128, 1, true>(a, st);
    }
    if (D == 64) return rows == 8 ? launch_split<64, 1>(a, st) : launch_split<64, 2>(a, st);
    if (D == 128) return rows == 8 ? launch_split<128, 1>(a, st) : launch_split<128, 2>(a, st);
    return rows == 8 ? launch_split<256, 1>(a, st) : launch_split<256, 2>(a, st);
}

}  // namespace dghost
