// dg_paged_attn.cu -- attention of a few query rows a sequence over the paged key / value cache.
//
// With few query rows the keys and values are read once and each value is used for a handful of
// multiplications, so the call is bound by memory.  A row here is one (query, query head); the rows that
// share a key head (Hq / Hkv of every query) make items of 8 NB rows (8, or 16 when a call's do not fit 8),
// and an item visits the key tiles that some query of its sequence may see.  All tiles of all items, in
// order, form one line that is cut into equal runs, one for each of a fixed number of resident CTAs (as many
// as the SMs hold): every CTA streams the same number of keys whatever the lengths are, and a long sequence
// is split over as many CTAs as its share of the line takes.  A run's first and last items may be
// pieces; pieces go to the workspace as (maximum, sums, unnormalised output) and a second kernel joins
// them in the order of the line.
//
// Within a CTA each warp owns 16 or 32 keys of a tile and runs on its own: its own ring of stages filled by
// cp.async (a step's keys and values each, past the end of a piece into the next one), its own running
// maximum and sums; warps meet only at the end of a piece.  The products are taken transposed, S^T = K Q^T
// and O^T = V^T P^T, with keys (or dimensions) as the 16 rows of mma.m16n8k16 and the query rows as its 8
// columns: eight rows fill the instruction, and P^T comes out of the first product's layout by two 8 x 8
// register transposes.  (The warp instruction, not tcgen05: at 8 rows the products need a few percent of
// either -- the tensor pipe is 9 % busy over 8k keys -- and a tile of TMEM would only add a round trip between
// the two products.)
//
// Measured: 64 tokens over up to 8k keys, 8 key heads of 128: 216 to 222 us, 6.7 TB/s, 98 % of the rate of a copy;
// one token over 128k keys, 4 key heads of 256: 88 us, 90 %.  Short of that: one sequence over 1k keys takes
// 8.3 us, two launches and five reads that wait for one another (lengths, pages, keys; list, pieces); 250
// windows of 1000 keys at 8 heads of 64 take 84 us, 88 %, of which start and join are 8; and items of few keys
// cost a CTA their latency: 1288 items of 3 keys, heads of 256, 35 us.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dg_paged_split.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether a call takes this file's path or dg_attention's query tiles over pages (dg_attn.cu).  A tile there (128
// queries of a query head) passes over the keys in the time of an item of 8 rows here, or of two for heads of
// 64, and tiles below the number of CTAs take as long as that number does.  So: whichever has fewer passes.
// Measured (us here / there), 16 query over 8 key heads of 128: 32 requests over 4k keys, 8 queries 90 / 137, 16
// queries 167 / 137; 8 requests over 2.3k keys, 16 queries 32 / 35, 24 queries 40 / 35, 64 queries 86 / 36; one over 2k
// keys, 256 queries 44 / 33.  Heads of 64, 16 queries of 8 heads, 32 requests over 4k keys 55 / 65.  Over 216 shapes
// (heads of 64, 128, 256, 1 to 16 query heads a key head, 1 to 256 queries, the same number in every sequence) the
// rule loses 0.1 % to the better path on average, 24 % at most.  A call that mixes lengths goes by its longest, and
// its single tokens then cost a tile each: 63 tokens over 8k keys beside a prompt of 512 take 484 us, in two calls 331;
// one over 128k beside a canvas 1595, in two calls 128.
bool split_path(int32_t n_seq, int32_t max_q_len, int32_t Hq, int32_t Hkv, int32_t D, int sms) {
    const int64_t tile_ctas = D == 256 ? sms : 2 * sms;
    // passes a sequence, which fit 64 bits for every call that the checks let through
    const int64_t here = Hkv * (((int64_t)max_q_len * (Hq / Hkv) + 7) / 8);
    const int64_t there = Hq * (((int64_t)max_q_len + 127) / 128) * (D == 64 ? 2 : 1);
    return here <= std::max(there, tile_ctas / n_seq);
}

}  // namespace

extern "C" size_t dg_paged_attention_workspace_bytes(int32_t n_seq, int32_t max_q_len, int32_t Hq, int32_t Hkv,
                                                     int32_t D) {
    if (n_seq < 1 || max_q_len < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
    // what either path needs, so that a workspace for a program's largest call serves its smaller ones, whichever
    // way they go
    return std::max(split_bytes(item_rows(max_q_len, Hq / Hkv), D), dghost::attention_pages_bytes(n_seq, max_q_len));
}

extern "C" dg_status dg_paged_attention(const uint16_t* q, const dg_paged_kv* cache, uint16_t* o, float* lse,
                                        const int32_t* cu_q, const uint8_t* causal, int32_t n_seq, int32_t max_q_len,
                                        int64_t total_q, int32_t Hq, int32_t Hkv, int32_t D, int32_t window,
                                        float scale, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
    if (n_seq < 0 || n_seq > 65535 || Hq < 1 || Hq > 65535 || Hkv < 1 || Hq % Hkv != 0 || window < -1 ||
        !(fabsf(scale) <= 0x1p127f))   // (past it log2(e) scale is infinite)
        return DG_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return DG_ERR_UNSUPPORTED;
    if (max_q_len < 1 || max_q_len > (1 << 30) || total_q < 0 || total_q >= (1LL << 31)) return DG_ERR_INVALID_ARG;
    if (n_seq == 0 || total_q == 0) return DG_OK;
    if (!q || !o || !cu_q || !causal) return DG_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !dghost::on_multiple(cu_q, 4) || !dghost::on_multiple(lse, 4))
        return DG_ERR_ALIGNMENT;
    SplitArgs a;
    const dg_status ok = dghost::paged_kv(cache, D, &a.kv);
    if (ok != DG_OK) return ok;
    const int rows = item_rows(max_q_len, Hq / Hkv);
    if (!workspace || workspace_bytes < dg_paged_attention_workspace_bytes(n_seq, max_q_len, Hq, Hkv, D))
        return DG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DG_ERR_ALIGNMENT;
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    if (!split_path(n_seq, max_q_len, Hq, Hkv, D, sms))
        return dghost::attention_pages(q, a.kv, o, lse, cu_q, causal, n_seq, max_q_len, total_q, Hq, Hkv, D, window, scale,
                                       workspace, (cudaStream_t)stream);
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.cu_q = cu_q;
    a.causal = causal;
    a.total_q = total_q;
    a.n_seq = n_seq;
    a.max_q_len = max_q_len;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.window = window;
    a.scale_log2 = scale * kLog2e;
    a.desc = static_cast<int4*>(workspace);
    a.part_o = reinterpret_cast<float*>(a.desc + 2 * kMaxCtas);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + (size_t)kMaxCtas * 2 * rows * D);
    a.status = dghost::status_word();
    cudaStream_t st = (cudaStream_t)stream;
    if (in_pairs(max_q_len, a.group, Hkv, D)) {
        a.Hkv /= 2;
        a.group *= 2;
        return launch_split<128, 1, true>(a, st);
    }
    if (D == 64) return rows == 8 ? launch_split<64, 1>(a, st) : launch_split<64, 2>(a, st);
    if (D == 128) return rows == 8 ? launch_split<128, 1>(a, st) : launch_split<128, 2>(a, st);
    return rows == 8 ? launch_split<256, 1>(a, st) : launch_split<256, 2>(a, st);
}
