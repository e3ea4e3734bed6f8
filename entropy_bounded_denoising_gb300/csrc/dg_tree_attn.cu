// dg_tree_attn.cu -- attention of drafted trees, and through a sliding window with first tokens that stay
// visible, over the paged key / value cache.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dg_paged.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct TreeArgs {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int32_t* cu_q;
    const uint32_t* mask;       // null: causal
    const int32_t* positions;
    int64_t total_q;
    int32_t n_seq, max_q_len, Hq, Hkv, mask_words, window, sinks;
    float scale_log2;
    dg::PagedKV kv;
    unsigned* status;
};

DG_DEVINL float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// A warp owns a query of one head, a lane D / 32 of its dimensions; keys one after another.
template <int D>
__global__ void __launch_bounds__(128) k_tree_simple(const TreeArgs a) {
    constexpr int E = D / 32;
    dg::pdl_wait();
    dg::pdl_release();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w < a.n_seq && lane == 0) {
        const dg::PagedSeq p = dg::paged_seq(a.kv, a.cu_q, a.total_q, (int)w, dg::kMaxKeys);
        if (!p.ok || p.ql > a.max_q_len) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
    }
    const int64_t row = w / a.Hq;
    const int h = (int)(w - row * a.Hq);
    if (row >= a.total_q) return;
    const int s = dg::warp_owner(a.cu_q, a.n_seq, (int)row);
    if (s >= a.n_seq) return;
    const dg::PagedSeq p = dg::paged_seq(a.kv, a.cu_q, a.total_q, s, dg::kMaxKeys);
    if (!p.ok || p.ql > a.max_q_len || row < p.q0 || row - p.q0 >= p.ql) return;
    const int i = (int)row - p.q0, ctx = p.kl > 0 ? p.kl - p.ql : 0;
    const int64_t pos = a.positions ? a.positions[row] : ctx + i;
    const uint16_t* q = a.q + (row * a.Hq + h) * D + lane * E;
    float qf[E], acc[E] = {};
    for (int e = 0; e < E; ++e) qf[e] = bf(q[e]) * a.scale_log2;
    float m = -INFINITY, l = 0.f;
    const int64_t head_at = (h / (a.Hq / a.Hkv)) * a.kv.head_stride + lane * E;
    for (int j = 0; j < p.kl; ++j) {
        bool seen = a.window < 0 || (int64_t)j >= pos - a.window || j < a.sinks;
        if (!a.mask)
            seen = seen && j <= ctx + i;
        else if (j >= ctx)
            seen = a.mask[row * a.mask_words + (j - ctx) / 32] >> ((j - ctx) & 31) & 1u;
        if (!seen) continue;
        const int32_t page = a.kv.page_table[(int64_t)s * a.kv.max_pages + (j >> a.kv.page_shift)];
        if (page < 0 || page >= a.kv.n_pages) {
            if (lane == 0) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            continue;
        }
        const int64_t at = page * a.kv.page_stride + (j & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride + head_at;
        float x = 0.f;
        for (int e = 0; e < E; ++e) x = fmaf(qf[e], bf(a.kv.k[at + e]), x);
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float top = fmaxf(m, x), f = m == -INFINITY ? 0.f : exp2f(m - top), w2 = exp2f(x - top);
        l = l * f + w2;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w2 * bf(a.kv.v[at + e]);
        m = top;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; e += 2) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(acc[e + 1] * inv), "f"(acc[e] * inv));
        *reinterpret_cast<uint32_t*>(a.o + (row * a.Hq + h) * D + lane * E + e) = r;
    }
    if (lane == 0 && a.lse) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

dg_status tree_attention(const uint16_t* q, const dg_paged_kv* cache, uint16_t* o, float* lse, const int32_t* cu_q,
                         bool tree, const uint32_t* mask, int32_t mask_words, const int32_t* positions, int32_t n_seq,
                         int32_t max_q_len, int64_t total_q, int32_t Hq, int32_t Hkv, int32_t D, int32_t window,
                         int32_t sinks, float scale, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
    if (n_seq < 0 || n_seq > 65535 || Hq < 1 || Hq > 65535 || Hkv < 1 || Hq % Hkv != 0 || window < (tree ? -1 : 0) ||
        sinks < 0 || !(fabsf(scale) <= 0x1p127f))   // (past it log2(e) scale is infinite)
        return DG_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return DG_ERR_UNSUPPORTED;
    if (max_q_len < 1 || max_q_len > (tree ? 65536 : 1 << 30) || total_q < 0 || total_q >= (1LL << 31))
        return DG_ERR_INVALID_ARG;
    if (tree && mask_words < (max_q_len + 31) / 32) return DG_ERR_INVALID_ARG;
    if (n_seq == 0 || total_q == 0) return DG_OK;
    if (!q || !o || !cu_q || (tree && (!mask || (window >= 0 && !positions)))) return DG_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !dghost::on_multiple(cu_q, 4) || !dghost::on_multiple(lse, 4) ||
        !dghost::on_multiple(mask, 4) || !dghost::on_multiple(positions, 4))
        return DG_ERR_ALIGNMENT;
    TreeArgs a;
    const dg_status ok = dghost::paged_kv(cache, D, &a.kv);
    if (ok != DG_OK) return ok;
    if (!workspace || workspace_bytes < dg_tree_attention_workspace_bytes(n_seq, max_q_len, Hq, Hkv, D))
        return DG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DG_ERR_ALIGNMENT;
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.cu_q = cu_q;
    a.mask = mask;
    a.positions = positions;
    a.total_q = total_q;
    a.n_seq = n_seq;
    a.max_q_len = max_q_len;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.mask_words = mask_words;
    a.window = window;
    a.sinks = window < 0 ? 0 : sinks;
    a.scale_log2 = scale * kLog2e;
    a.status = dghost::status_word();
    const int64_t blocks = (std::max<int64_t>(total_q * Hq, n_seq) + 3) / 4;
    if (blocks > 0x7fffffffLL) return DG_ERR_INVALID_ARG;
    auto kern = D == 64 ? k_tree_simple<64> : D == 128 ? k_tree_simple<128> : k_tree_simple<256>;
    const cudaError_t e = dghost::launch_pdl(kern, dim3((unsigned)blocks), dim3(128), 0, (cudaStream_t)stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}

}  // namespace

extern "C" size_t dg_tree_attention_workspace_bytes(int32_t n_seq, int32_t max_q_len, int32_t Hq, int32_t Hkv, int32_t D) {
    if (n_seq < 1 || max_q_len < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
    return 16;
}

extern "C" dg_status dg_tree_attention(const uint16_t* q, const dg_paged_kv* cache, uint16_t* o, float* lse,
                                       const int32_t* cu_q, const uint32_t* tree_mask, int32_t mask_words,
                                       const int32_t* positions, int32_t n_seq, int32_t max_q_len, int64_t total_q,
                                       int32_t Hq, int32_t Hkv, int32_t D, int32_t window, int32_t sinks, float scale,
                                       void* workspace, size_t workspace_bytes, dg_stream_t stream) {
    return tree_attention(q, cache, o, lse, cu_q, true, tree_mask, mask_words, positions, n_seq, max_q_len, total_q, Hq, Hkv,
                          D, window, sinks, scale, workspace, workspace_bytes, stream);
}

extern "C" dg_status dg_sink_attention(const uint16_t* q, const dg_paged_kv* cache, uint16_t* o, float* lse,
                                       const int32_t* cu_q, int32_t n_seq, int32_t max_q_len, int64_t total_q, int32_t Hq,
                                       int32_t Hkv, int32_t D, int32_t window, int32_t sinks, float scale,
                                       void* workspace, size_t workspace_bytes, dg_stream_t stream) {
    return tree_attention(q, cache, o, lse, cu_q, false, nullptr, 0, nullptr, n_seq, max_q_len, total_q, Hq, Hkv, D, window,
                          sinks, scale, workspace, workspace_bytes, stream);
}
