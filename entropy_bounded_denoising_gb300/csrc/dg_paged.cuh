// dg_paged.cuh -- the paged key / value cache as kernels see it, shared by the append and the
// attention over pages.
#pragma once

#include "dg_common.cuh"

namespace dg {

// dg_paged_kv with the page size as a shift (a power of two, checked on the host).
struct PagedKV {
    uint16_t* k;
    uint16_t* v;
    const int32_t* page_table;
    const int32_t* kv_len;
    int64_t n_pages, page_stride, slot_stride, head_stride;
    int32_t page_shift, max_pages;

    DG_DEVINL int64_t capacity() const { return (int64_t)max_pages << page_shift; }
};

// Keys of a sequence of an attention call, at most: an index a tile past the last key still fits 32 bits.
constexpr int32_t kMaxKeys = 0x7fff0000;

// A sequence of a paged call: its rows of q and its keys.  `ok` is false where the offsets or
// lengths are out of range (the caller raises DG_DEV_BAD_PARAM and leaves the sequence out).
struct PagedSeq {
    int32_t q0, ql, kl;
    bool ok;
};

DG_DEVINL PagedSeq paged_seq(const PagedKV& c, const int32_t* cu_q, int64_t total_q, int s, int32_t max_keys) {
    PagedSeq r;
    r.q0 = cu_q[s];
    const int32_t q1 = cu_q[s + 1];
    r.kl = c.kv_len[s];
    r.ok = r.q0 >= 0 && q1 >= r.q0 && (int64_t)q1 <= total_q && r.kl >= 0 && r.kl <= max_keys &&
           (int64_t)r.kl <= c.capacity();
    r.ql = r.ok ? q1 - r.q0 : 0;
    if (r.kl > 0 && r.ql > r.kl) r.ok = false;
    return r;
}

// The number of sequences that end at or before row t (cu_q[1 .. n] <= t): the index of the
// sequence that owns row t when the offsets are in order.  A whole warp searches, 32 probes a
// round, so 1024 sequences take two dependent loads.
DG_DEVINL int warp_owner(const int32_t* cu_q, int n, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int e = lo + (lane + 1) * step;
        const int before = __popc(__ballot_sync(0xffffffffu, e <= hi && cu_q[min(e, hi)] <= t));
        lo += before * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

}  // namespace dg

namespace dghost {
// Whether a pointer (null too) lies on a multiple of n bytes, a power of two.
inline bool on_multiple(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks shared by the calls that take a dg_paged_kv; fills `c` when it returns DG_OK.
dg_status paged_kv(const dg_paged_kv* cache, int32_t D, dg::PagedKV* c);

// Attention over pages with the query tiles of dg_attention (dg_attn.cu), and its workspace.
size_t attention_pages_bytes(int32_t n_seq, int32_t max_q_len);
dg_status attention_pages(const uint16_t* q, const dg::PagedKV& kv, uint16_t* o, float* lse, const int32_t* cu_q,
                          const uint8_t* causal, int32_t n_seq, int32_t max_q_len, int64_t total_q, int32_t Hq,
                          int32_t Hkv, int32_t D, int32_t window, float scale, void* workspace, cudaStream_t stream);
}  // namespace dghost
