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
    int32_t n_seq, Hq, Hkv, D, rot, tasks, head_shift;  // tasks: per row; 2^head_shift of them a head
    bool narrow;        // fewer than 2^31 tasks
    uint32_t row_blocks;   // blocks with rows; those behind them check the sequences
    dg::PagedKV kv;
    unsigned* status;
};

struct Task {
    int row, head;   // row of the unit; heads in order: key heads, value heads, query heads
    int at, dist;    // the first chunk's dimension, and how far behind it the second one lies
    bool turn;       // of the rotated part
};

DG_DEVINL Task task_of(const AppendArgs& a, int i) {
    Task k;
    k.row = i / a.tasks;
    const int t = i - k.row * a.tasks;
    k.head = t >> a.head_shift;
    const int tt = t & ((1 << a.head_shift) - 1);
    const bool value = k.head >= a.Hkv && k.head < 2 * a.Hkv;
    k.turn = !value && tt < a.rot / 16;
    k.at = value || k.turn ? tt * 8 : a.rot + (tt - a.rot / 16) * 8;
    k.dist = value ? a.D / 2 : k.turn ? a.rot / 2 : (a.D - a.rot) / 2;
    return k;
}

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

// w radians as a fraction of a turn in 64-bit fixed point: floor(w / (2 pi) 2^64) mod 2^64, within two units of the
// last place.  In integers: w = m 2^(e - 1075) and 4 / (2 pi) = 2 / pi = 0.A2F9836E4E441529 FC2757D1F534DDC0... in
// base 16, so the turns are m times those bits, shifted.  With the first 64 of them the error is |w| / 4 units and
// one, so from |w| = 4 on 128 are taken, which are enough below 2^53.  Past that, and for infinities and NaN, there
// is no angle to speak of, and 0 is returned.  (The doubles' own operations run at a small fraction of this rate.)
DG_DEVINL int exponent_of(double w) { return (int)(__double2hiint(w) >> 20) & 0x7ff; }
DG_DEVINL bool has_angle(double w) { return exponent_of(w) < 1023 + 53; }

// A call of its own: such frequencies are rare, and in line their instructions cost 64 rows 0.2 us and 30k rows 6.
__device__ __noinline__ uint64_t far_turns(uint64_t m, int e) {   // (top, mid, low) 2^(e - 1205) turns, 66 <= down <= 116
    const uint64_t lo = m * 0xA2F9836E4E441529ull, hi = __umul64hi(m, 0xA2F9836E4E441529ull);
    const uint64_t mid = lo + __umul64hi(m, 0xFC2757D1F534DDC0ull), top = hi + (mid < lo ? 1ull : 0ull);
    const int down = 1141 - e;
    return e < 1023 + 53 ? (mid >> (down - 64)) | (top << (128 - down)) : 0ull;
}

DG_DEVINL uint64_t turns_of(double w) {
    const uint64_t bits = (uint64_t)__double_as_longlong(w);
    const int e = exponent_of(w);
    const uint64_t m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0ull);
    uint64_t f = 0;
    if (e < 1023 + 2) {   // (hi, lo) 2^(e - 1141) turns, down from 53
        const uint64_t lo = m * 0xA2F9836E4E441529ull, hi = __umul64hi(m, 0xA2F9836E4E441529ull);
        const int down = 1077 - max(e, 1);
        if (down >= 64 && down < 128)
            f = hi >> (down - 64);
        else if (down < 64)
            f = (lo >> down) | (hi << (64 - down));
    } else {
        f = far_turns(m, e);
    }
    return bits >> 63 ? 0ull - f : f;
}

// The position of a row in the sequence that a search found for it (-1: none, or one that is refused; the
// search says little when the offsets are not in order).
DG_DEVINL int row_position(const AppendArgs& a, int t, int s) {
    if (s >= a.n_seq) return -1;
    const dg::PagedSeq q = dg::paged_seq(a.kv, a.cu_q, a.total_q, s, 0x7fffffff);
    return q.ok && q.q0 <= t && t - q.q0 < q.ql && q.kl > 0 ? q.kl - q.ql + (t - q.q0) : -1;
}

// A block's rows are looked up and its sines computed while its data is on the way: every thread
// first asks for the 32 bytes a task that it will store.
// Bound by memory from a few thousand rows on: 30k rows of 32 heads of 256 (907 MB to and fro) take 139 us,
// 6.5 TB/s.  Below, by its chain of dependent reads (offsets, lengths, page) and the launch: 64 rows of 32 heads of
// 128 take 3.4 us, 2048 rows 9.1, where a copy of their 34 MB takes 6.6.
// PerThread: a thread's tasks.  One, with the most threads an SM holds, while every task has a
// place at once; four where there are several rounds of blocks (more bytes on the way and fewer lookups
// a byte).  One against four, the same rows again and again: 64 rows 3.4 and 5.1 us, 2048 rows 8.4 and 8.2, the 30k
// rows 154 and 138.
template <bool Interleaved, int PerThread>
__global__ void __launch_bounds__(kAppendThreads, PerThread == 1 ? 8 : 4) k_kv_append(const AppendArgs a) {
    constexpr int kPerThread = PerThread, kUnit = kAppendThreads * PerThread;   // tasks of a block
    constexpr int kRows = kUnit / 8 + 2;       // rows of a unit: at least 8 tasks each (one key head of 64)
    __shared__ int64_t place[kRows];           // cache offset of a row's slot, -1 = skipped
    __shared__ int32_t position[kRows];
    __shared__ float2 cs[kUnit * 4 + 2 * 128]; // cosine and sine of its angles
    dg::pdl_wait();
    dg::pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Every sequence is checked, whether a row finds it or not, and every frequency: a thread each, in blocks of
    // their own (0.05 us of 64 rows' 3.4; in the first block, before its lookups, the sequences alone cost 0.25).
    if (blockIdx.x >= a.row_blocks) {
        const int s = (int)(blockIdx.x - a.row_blocks) * kAppendThreads + tid;
        if ((s < a.n_seq && !dg::paged_seq(a.kv, a.cu_q, a.total_q, s, 0x7fffffff).ok) ||
            (s < a.rot / 2 && !has_angle(a.inv_freq[s])))
            dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        return;
    }
    const int half = a.rot / 2;
    const int64_t first = (int64_t)blockIdx.x * kUnit;
    const int64_t row0 = a.narrow ? (int64_t)((uint32_t)first / (uint32_t)a.tasks) : first / a.tasks;
    const int skip = (int)(first - row0 * a.tasks);   // tasks of row0 before the unit
    const int rows = (int)min(a.total_q - row0, (int64_t)((skip + kUnit - 1) / a.tasks + 1));

    uint4 x[kPerThread], y[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const Task k = task_of(a, skip + u * kAppendThreads + tid);
        if (k.row < rows) {
            const int64_t row = row0 + k.row;
            const uint16_t* src = k.head < a.Hkv       ? a.k + row * a.ldk + (int64_t)k.head * a.D
                                  : k.head < 2 * a.Hkv ? a.v + row * a.ldv + (int64_t)(k.head - a.Hkv) * a.D
                                                       : a.q + row * a.ldq + (int64_t)(k.head - 2 * a.Hkv) * a.D;
            x[u] = *reinterpret_cast<const uint4*>(src + k.at);
            y[u] = *reinterpret_cast<const uint4*>(src + k.at + k.dist);
        }
    }
    const double w0 = tid < rows * half ? a.inv_freq[tid % half] : 0.0;   // of this thread's first angle
    int mine = -1, owner = 0;   // the row this thread looks up
    if (rows <= kAppendThreads / 32) {   // a warp a row: two dependent reads for up to 1024 sequences
        if (warp < rows) {
            owner = dg::warp_owner(a.cu_q, a.n_seq, (int)(row0 + warp));
            if (lane == 0) mine = warp;
        }
    } else if (tid < rows) {             // narrow rows: a thread each, by bisection
        mine = tid;
        int hi = a.n_seq;
        while (owner < hi) {
            const int mid = (owner + hi) / 2;
            if (a.cu_q[mid + 1] <= (int)(row0 + tid))
                owner = mid + 1;
            else
                hi = mid;
        }
    }
    int p = -1;
    if (mine >= 0) {
        p = row_position(a, (int)(row0 + mine), owner);
        position[mine] = p;
    }
    __syncthreads();
    if (mine >= 0) {
        int64_t at = -1;
        if (p >= 0) {
            const int32_t page = a.kv.page_table[(int64_t)owner * a.kv.max_pages + (p >> a.kv.page_shift)];
            if (page < 0 || page >= a.kv.n_pages)
                dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            else
                at = page * a.kv.page_stride + (p & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride;
        }
        place[mine] = at;
    }
    for (int i = tid; i < rows * half; i += kAppendThreads) {
        const int r = i / half;
        const double w = i == tid ? w0 : a.inv_freq[i - r * half];
        const int64_t u = (int64_t)(turns_of(w) * (uint64_t)position[r]);
        float sn, c;
        sincospif((float)u * 1.0842021724855044e-19f, &sn, &c);  // 2^-63: half turns in [-1, 1]
        cs[i] = make_float2(c, sn);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const Task k = task_of(a, skip + u * kAppendThreads + tid);
        if (k.row >= rows || place[k.row] < 0) continue;
        if (k.turn) {
            const float2* c = cs + k.row * half;
            if (Interleaved) {
                rotate_neighbours(x[u], c + k.at / 2);
                rotate_neighbours(y[u], c + half / 2 + k.at / 2);
            } else {
                rotate_halves(x[u], y[u], c + k.at);
            }
        }
        uint16_t* dst = k.head < a.Hkv       ? a.kv.k + place[k.row] + k.head * a.kv.head_stride
                        : k.head < 2 * a.Hkv ? a.kv.v + place[k.row] + (k.head - a.Hkv) * a.kv.head_stride
                                             : a.q_out + ((row0 + k.row) * a.Hq + (k.head - 2 * a.Hkv)) * a.D;
        *reinterpret_cast<uint4*>(dst + k.at) = x[u];
        *reinterpret_cast<uint4*>(dst + k.at + k.dist) = y[u];
    }
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
    if (!aligned16(cache->k) || !aligned16(cache->v) || !on_multiple(cache->page_table, 4) || !on_multiple(cache->kv_len, 4))
        return DG_ERR_ALIGNMENT;
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
        (q && ldq % 8) || !dghost::on_multiple(cu_q, 4) || !dghost::on_multiple(inv_freq, 8))
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
    a.head_shift = D == 64 ? 2 : D == 128 ? 3 : 4;
    a.status = dghost::status_word();
    a.narrow = total_q * a.tasks < (1LL << 31);
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    const bool one = total_q * a.tasks <= (int64_t)sms * 2048;
    const int64_t unit = one ? kAppendThreads : kAppendThreads * 4;
    const int64_t row_blocks = (total_q * a.tasks + unit - 1) / unit;
    const int64_t blocks = row_blocks + (n_seq + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7fffffffLL) return DG_ERR_INVALID_ARG;
    a.row_blocks = (uint32_t)row_blocks;
    const cudaError_t e = dghost::launch_pdl(one ? (interleaved ? k_kv_append<true, 1> : k_kv_append<false, 1>)
                                                 : (interleaved ? k_kv_append<true, 4> : k_kv_append<false, 4>),
                                             dim3((unsigned)blocks), dim3(kAppendThreads), 0, (cudaStream_t)stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}
