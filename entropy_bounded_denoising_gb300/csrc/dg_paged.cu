// dg_paged.cu -- the paged key / value cache: appending a pass's rotated keys and its values.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dg_paged.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

DG_DEVINL uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}
DG_DEVINL float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
DG_DEVINL float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// ------------------------------------------------------------------ append
// A task is 32 bytes of one head: two 16-byte chunks half a part away from each other, the part
// being the rotated dimensions, the rest, or a whole value head; neighbouring threads then touch
// neighbouring chunks, and the two chunks are the two halves of eight pairs when the pairs lie
// rot_dim / 2 apart.  A block's threads take consecutive tasks of consecutive rows.
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    int64_t ldk, ldv, ldq;
    const int32_t* cu_q;
    const double* inv_freq;
    int64_t total_q;
    int32_t n_seq, Hq, Hkv, D, rot, tasks;  // tasks: per row
    dg::PagedKV kv;
    unsigned* status;
};

DG_DEVINL void rotate_halves(uint4& x, uint4& y, const float2* cs) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&x);
    uint32_t* b = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 c0 = cs[2 * e], c1 = cs[2 * e + 1];
        const float a0 = lo_f(a[e]), a1 = hi_f(a[e]), b0 = lo_f(b[e]), b1 = hi_f(b[e]);
        a[e] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
        b[e] = pack_bf16x2(a0 * c0.y + b0 * c0.x, a1 * c1.y + b1 * c1.x);
    }
}

DG_DEVINL void rotate_neighbours(uint4& x, const float2* cs) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 c = cs[e];
        const float u = lo_f(a[e]), w = hi_f(a[e]);
        a[e] = pack_bf16x2(u * c.x - w * c.y, u * c.y + w * c.x);
    }
}

template <bool Interleaved>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const AppendArgs a) {
    // rows of the block: where each goes, and the sines and cosines of its angles
    constexpr int kRows = kAppendThreads / 8 + 2;  // at least 8 tasks a row (one key head of 64)
    __shared__ int64_t place[kRows];               // cache offset of the row's slot, -1 = skipped
    __shared__ int32_t position[kRows];
    __shared__ float2 cs[kAppendThreads * 4 + 2 * 128];
    dg::pdl_wait();
    dg::pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = (int64_t)blockIdx.x * kAppendThreads;
    const int64_t row0 = first / a.tasks;
    const int rows = (int)(min(a.total_q - 1, (first + kAppendThreads - 1) / a.tasks) - row0) + 1;
    const int half = a.rot / 2;

    for (int r = warp; r < rows; r += kAppendThreads / 32) {
        const int t = (int)(row0 + r);
        const int s = dg::warp_owner(a.cu_q, a.n_seq, t);
        if (lane == 0) {
            int64_t at = -1;
            int p = 0;
            if (s < a.n_seq && a.cu_q[s] <= t) {
                const dg::PagedSeq q = dg::paged_seq(a.kv, a.cu_q, a.total_q, s);
                if (!q.ok) {
                    dg::raise_status(a.status, DG_DEV_BAD_PARAM);
                } else if (q.kl > 0) {
                    p = q.kl - q.ql + (t - q.q0);
                    const int32_t page = a.kv.page_table[(int64_t)s * a.kv.max_pages + (p >> a.kv.page_shift)];
                    if (page < 0 || page >= a.kv.n_pages)
                        dg::raise_status(a.status, DG_DEV_BAD_PARAM);
                    else
                        at = page * a.kv.page_stride + (p & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride;
                }
            }
            place[r] = at;
            position[r] = p;
        }
    }
    __syncthreads();
    // turns of pair j at position p: p * inv_freq / 2 pi modulo 1, exact in 64-bit fixed point
    // once the frequency is rounded to 2^-64 turns (or to its 53 bits)
    for (int i = tid; i < rows * half; i += kAppendThreads) {
        const double turns = a.inv_freq[i % half] * 0.15915494309189533577;
        const uint64_t f = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
        const int64_t u = (int64_t)(f * (uint64_t)position[i / half]);
        float sn, c;
        sincospif((float)u * 1.0842021724855044e-19f, &sn, &c);  // 2^-63: half turns in [-1, 1]
        cs[i] = make_float2(c, sn);
    }
    __syncthreads();
    const int64_t id = first + tid;
    const int64_t row = id / a.tasks;
    if (row >= a.total_q) return;
    const int r = (int)(row - row0);
    if (place[r] < 0) return;
    const int per_head = a.D / 16;
    const int task = (int)(id - row * a.tasks);
    const int head = task / per_head;
    const int tt = task - head * per_head;
    // heads in order: key heads, value heads, query heads
    const bool is_v = head >= a.Hkv && head < 2 * a.Hkv;
    int e0 = tt * 8, dist = a.D / 2;
    const bool turn = !is_v && tt < a.rot / 16;
    if (!is_v) {
        if (turn) {
            dist = half;
        } else {
            e0 = a.rot + (tt - a.rot / 16) * 8;
            dist = (a.D - a.rot) / 2;
        }
    }
    const uint16_t* src;
    uint16_t* dst;
    if (head < a.Hkv) {
        src = a.k + row * a.ldk + (int64_t)head * a.D;
        dst = a.kv.k + place[r] + head * a.kv.head_stride;
    } else if (is_v) {
        src = a.v + row * a.ldv + (int64_t)(head - a.Hkv) * a.D;
        dst = a.kv.v + place[r] + (head - a.Hkv) * a.kv.head_stride;
    } else {
        src = a.q + row * a.ldq + (int64_t)(head - 2 * a.Hkv) * a.D;
        dst = a.q_out + (row * a.Hq + (head - 2 * a.Hkv)) * a.D;
    }
    uint4 x = *reinterpret_cast<const uint4*>(src + e0);
    uint4 y = *reinterpret_cast<const uint4*>(src + e0 + dist);
    if (turn) {
        const float2* c = cs + r * half;
        if (Interleaved) {
            rotate_neighbours(x, c + tt * 4);
            rotate_neighbours(y, c + half / 2 + tt * 4);
        } else {
            rotate_halves(x, y, c + tt * 8);
        }
    }
    *reinterpret_cast<uint4*>(dst + e0) = x;
    *reinterpret_cast<uint4*>(dst + e0 + dist) = y;
}

}  // namespace

namespace dghost {

dg_status paged_kv(const dg_paged_kv* cache, int32_t D, dg::PagedKV* c) {
    if (!cache) return DG_ERR_INVALID_ARG;
    const int32_t ps = cache->page_size;
    const int64_t strides[3] = {cache->page_stride, cache->slot_stride, cache->head_stride};
    if (!cache->k || !cache->v || !cache->page_table || !cache->kv_len || cache->n_pages < 1 ||
        cache->n_pages > 0x7fffffffLL || cache->max_pages < 1)
        return DG_ERR_INVALID_ARG;
    if (ps < 8 || ps > 65536 || (ps & (ps - 1)) != 0) return DG_ERR_UNSUPPORTED;
    for (int64_t s : strides)
        if (s < D || s >= (1LL << 39)) return DG_ERR_INVALID_ARG;
    if (cache->n_pages > (1LL << 60) / cache->page_stride) return DG_ERR_INVALID_ARG;
    if (!aligned16(cache->k) || !aligned16(cache->v)) return DG_ERR_ALIGNMENT;
    for (int64_t s : strides)
        if (s % 8) return DG_ERR_ALIGNMENT;
    c->k = cache->k;
    c->v = cache->v;
    c->page_table = cache->page_table;
    c->kv_len = cache->kv_len;
    c->n_pages = cache->n_pages;
    c->page_stride = cache->page_stride;
    c->slot_stride = cache->slot_stride;
    c->head_stride = cache->head_stride;
    c->page_shift = 0;
    while ((1 << c->page_shift) < ps) ++c->page_shift;
    c->max_pages = cache->max_pages;
    return DG_OK;
}

}  // namespace dghost

extern "C" dg_status dg_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, const uint16_t* q,
                                  int64_t ldq, uint16_t* q_out, const int32_t* cu_q, int32_t n_seq, int64_t total_q,
                                  int32_t Hq, int32_t Hkv, int32_t D, const double* inv_freq, int32_t rot_dim,
                                  int32_t interleaved, const dg_paged_kv* cache, dg_stream_t stream) {
    if (n_seq < 0 || n_seq > 65535 || total_q < 0 || total_q >= (1LL << 31) || Hq < 1 || Hq > 65535 || Hkv < 1 ||
        Hkv > 65535)
        return DG_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return DG_ERR_UNSUPPORTED;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 || (rot_dim > 0 && !inv_freq)) return DG_ERR_INVALID_ARG;
    if (n_seq == 0 || total_q == 0) return DG_OK;
    if (!k || !v || !cu_q || (q != nullptr) != (q_out != nullptr)) return DG_ERR_INVALID_ARG;
    if (ldk < (int64_t)Hkv * D || ldv < (int64_t)Hkv * D || (q && ldq < (int64_t)Hq * D)) return DG_ERR_INVALID_ARG;
    if (ldk >= (1LL << 31) || ldv >= (1LL << 31) || (q && ldq >= (1LL << 31))) return DG_ERR_INVALID_ARG;
    if (q && q_out == q && ldq != (int64_t)Hq * D) return DG_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) || ldk % 8 || ldv % 8 ||
        (q && ldq % 8))
        return DG_ERR_ALIGNMENT;
    AppendArgs a;
    const dg_status ok = dghost::paged_kv(cache, D, &a.kv);
    if (ok != DG_OK) return ok;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldq = ldq;
    a.cu_q = cu_q;
    a.inv_freq = inv_freq;
    a.total_q = total_q;
    a.n_seq = n_seq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.rot = rot_dim;
    a.tasks = ((q ? Hq : 0) + 2 * Hkv) * (D / 16);
    a.status = dghost::status_word();
    const int64_t blocks = (total_q * a.tasks + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7fffffffLL) return DG_ERR_INVALID_ARG;
    const cudaError_t e = dghost::launch_pdl(interleaved ? k_kv_append<true> : k_kv_append<false>,
                                             dim3((unsigned)blocks), dim3(kAppendThreads), 0, (cudaStream_t)stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}
