// dg_paged.cu -- the paged key / value cache: appending a pass's rotated keys and its values, its queries
// and keys normed before where a call says so.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

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

// ------------------------------------------------------------------ append with norms
// A warp owns up to T groups of 32 / (D / 16) heads of one row: a head's D / 16 lanes hold 32 bytes each, two chunks as in a
// task of the append, and the same dimensions in every group, so that a lane reads its cosines and sines once a
// warp and its weights where it lies in a line with its neighbours.  The data is asked for first; the row's sequence and slot
// are looked up and its sines computed while it is on the way, by the warp itself: nothing waits for a block.
// Values stay in fp32 from the norm through the rotation.
// Bound by memory from a few thousand rows on: ragged prompts of 18k rows, 16 / 8 heads of 128, 594 MB to and fro, take 104.5
// us, 84 % of a copy's rate, by instructions as much (62 % of all issue slots); in registers, without shared memory, they
// took 114.  64 rows take 3.4 us, a launch and the reads that wait for one another; 32 trees of 64 rows 10.8.
struct NormArgs : AppendArgs {
    const float* norm[2];      // of keys and of queries; null: not normed
    const int32_t* positions;  // null: the slots' numbers
    float eps;
    int32_t groups, chunks;    // groups of heads in a row, and warps that they take
};
constexpr int kNormWarps = 4;

// The sixteen values of a task as floats, and back.
DG_DEVINL void unpack16(const uint4& x, const uint4& y, float (&f)[16]) {
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[2 * e] = lo_f(w[e]);
        f[2 * e + 1] = hi_f(w[e]);
    }
}
DG_DEVINL void pack16(const float (&f)[16], uint4& x, uint4& y) {
    x = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    y = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
}

// The sum over a head's lanes, which lie side by side.
template <int Lanes>
DG_DEVINL float head_sum(float v) {
#pragma unroll
    for (int o = 1; o < Lanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean f^2 + eps) over a head.  A sum of squares past fp32 (values from 2^60 on) is taken of values 2^-70 as large,
// beside which eps is nothing unless it is as large (then for its own sake: the two might pass fp32 together); f is then
// scaled.  (Whole warp; squares below fp32 are below eps, at least 2^-126.)
template <int D>
DG_DEVINL float norm_of(float (&f)[16], float eps) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        s0 = fmaf(f[e], f[e], s0);
        s1 = fmaf(f[e + 1], f[e + 1], s1);
    }
    float ss = head_sum<D / 16>(s0 + s1);
    const bool large = !(ss <= 0x1p120f) || eps > 0x1p120f;   // (or a NaN, which stays one)
    if (__any_sync(0xffffffffu, large)) {
        if (large) {
            eps *= 0x1p-140f;
            ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                f[e] *= 0x1p-70f;
                ss = fmaf(f[e], f[e], ss);
            }
        }
        const float again = head_sum<D / 16>(ss);
        ss = large ? again : ss;
    }
    return rsqrtf(fmaf(ss, 1.f / D, eps));
}

DG_DEVINL void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dg::smem_u32(dst)), "l"(src) : "memory");
}

template <bool Interleaved, int D, int T>
__global__ void __launch_bounds__(kNormWarps * 32, T == 1 ? 8 : 6) k_kv_append_norm(const __grid_constant__ NormArgs a) {
    constexpr int G = D / 16, Heads = 32 / G;   // lanes of a head, heads of a group
    extern __shared__ uint4 norm_data[];        // [warp][group][chunk][lane]: the data on its way (in registers: 16 warps an SM for 24)
    __shared__ float4 weight[2][4][G];          // [keys, queries][quarter of a lane's values][lane of the head]
    __shared__ float4 turns[kNormWarps][4][G];  // a row's cosines and sines: [pairs 2 e, 2 e + 1 of a lane][lane]
    dg::pdl_wait();
    dg::pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // every sequence and frequency is checked by blocks of their own, as in the append
    if (blockIdx.x >= a.row_blocks) {
        const int s = (int)(blockIdx.x - a.row_blocks) * (kNormWarps * 32) + tid;
        if ((s < a.n_seq && !dg::paged_seq(a.kv, a.cu_q, a.total_q, s, 0x7fffffff).ok) ||
            (s < a.rot / 2 && !has_angle(a.inv_freq[s])))
            dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        return;
    }
    const int64_t task = (int64_t)blockIdx.x * kNormWarps + warp;
    int64_t row;
    int g0 = 0;       // the first group
    if (a.chunks == 1) {
        row = task;
    } else {
        row = a.narrow ? (int64_t)((uint32_t)task / (uint32_t)a.chunks) : task / a.chunks;
        g0 = (int)(task - row * a.chunks) * T;
    }
    const bool real = row < a.total_q;
    const int tt = lane % G, sub = lane / G, half = a.rot / 2, heads = 2 * a.Hkv + (a.q ? a.Hq : 0);
    const bool turn = tt < a.rot / 16;
    const int at = turn ? tt * 8 : a.rot + (tt - a.rot / 16) * 8, dist = turn ? a.rot / 2 : (D - a.rot) / 2;
    // a value head lies in chunks half a head apart; its lanes read it so
    uint4* const data = norm_data + warp * (T * 64) + lane;
#pragma unroll
    for (int u = 0; u < T; ++u) {
        const int h = (g0 + u) * Heads + sub;
        if (real && h < heads) {
            const bool value = h >= a.Hkv && h < 2 * a.Hkv;
            const uint16_t* src = h < a.Hkv       ? a.k + row * a.ldk + (int64_t)h * D
                                  : value         ? a.v + row * a.ldv + (int64_t)(h - a.Hkv) * D
                                                  : a.q + row * a.ldq + (int64_t)(h - 2 * a.Hkv) * D;
            cp_async16(data + u * 64, src + (value ? tt * 8 : at));
            cp_async16(data + u * 64 + 32, src + (value ? tt * 8 + D / 2 : at + dist));
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // the weights in the order in which lanes take them
    for (int i = tid; i < 8 * G; i += kNormWarps * 32) {
        const int which = i / (4 * G), c = i / G & 3, l = i % G;
        const bool tl = l < a.rot / 16;
        const int al = (tl ? l * 8 : a.rot + (l - a.rot / 16) * 8) + (c & 1) * 4 + (c < 2 ? 0 : tl ? a.rot / 2 : (D - a.rot) / 2);
        const float* w = a.norm[which];
        if (w) weight[which][c][l] = make_float4(w[al], w[al + 1], w[al + 2], w[al + 3]);
    }
    // the row's place and angles
    int64_t place = -1;
    int by = 0;
    if (real) {
        const int s = dg::warp_owner(a.cu_q, a.n_seq, (int)row);
        const int p = row_position(a, (int)row, s);
        by = a.positions ? a.positions[row] : p;
        if (p >= 0) {
            const int32_t page = a.kv.page_table[(int64_t)s * a.kv.max_pages + (p >> a.kv.page_shift)];
            if (page < 0 || page >= a.kv.n_pages) {
                if (lane == 0) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            } else {
                place = page * a.kv.page_stride + (p & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride;
            }
        }
        for (int j = lane; j < half; j += 32) {
            const int64_t u = (int64_t)(turns_of(a.inv_freq[j]) * (uint64_t)(int64_t)by);
            float sn, c;
            sincospif((float)u * 1.0842021724855044e-19f, &sn, &c);  // 2^-63: half turns in [-1, 1]
            // pair j is a lane's e-th: dimensions e of both its chunks, or neighbours, four pairs a chunk
            const int second = Interleaved && j >= half / 2, jj = second ? j - half / 2 : j;
            const int l = Interleaved ? jj / 4 : jj / 8, e = Interleaved ? jj % 4 + 4 * second : jj % 8;
            reinterpret_cast<float2*>(&turns[warp][e / 2][l])[e & 1] = make_float2(c, sn);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // the weights; and a warp's own turns
    if (place < 0) return;   // (the whole warp: it has one row)
#pragma unroll 1
    for (int u = 0; u < T; ++u) {
        if ((g0 + u) * Heads >= heads) break;
        const int h = (g0 + u) * Heads + sub;
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (h < heads) {
            x = data[u * 64];
            y = data[u * 64 + 32];
        }
        const bool key = h < a.Hkv, value = !key && h < 2 * a.Hkv;
        const bool normed = !value && a.norm[key ? 0 : 1], turned = !value && turn;
        if (__any_sync(0xffffffffu, normed || turned)) {
            float f[16];
            unpack16(x, y, f);
            if (__any_sync(0xffffffffu, normed)) {
                float n[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) n[e] = f[e];
                const float r = norm_of<D>(n, a.eps);
                if (normed) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 w = weight[key ? 0 : 1][c][tt];
                        f[4 * c] = n[4 * c] * r * w.x;
                        f[4 * c + 1] = n[4 * c + 1] * r * w.y;
                        f[4 * c + 2] = n[4 * c + 2] * r * w.z;
                        f[4 * c + 3] = n[4 * c + 3] * r * w.w;
                    }
                }
            }
            if (turned) {
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                    const float4 z = turns[warp][e2][tt];
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const int e = 2 * e2 + o, i = Interleaved ? 2 * e : e, j = Interleaved ? 2 * e + 1 : e + 8;
                        const float c = o ? z.z : z.x, sn = o ? z.w : z.y, p0 = f[i], p1 = f[j];
                        f[i] = p0 * c - p1 * sn;
                        f[j] = p0 * sn + p1 * c;
                    }
                }
            }
            if (normed || turned) pack16(f, x, y);
        }
        if (h >= heads) continue;
        uint16_t* dst = key     ? a.kv.k + place + h * a.kv.head_stride
                        : value ? a.kv.v + place + (h - a.Hkv) * a.kv.head_stride
                                : a.q_out + (row * a.Hq + (h - 2 * a.Hkv)) * D;
        *reinterpret_cast<uint4*>(dst + (value ? tt * 8 : at)) = x;
        *reinterpret_cast<uint4*>(dst + (value ? tt * 8 + D / 2 : at + dist)) = y;
    }
}

template <bool Interleaved, int D>
cudaError_t launch_norm(NormArgs& a, bool small, cudaStream_t stream) {
    constexpr int T = 8;
    a.groups = ((a.q ? a.Hq : 0) + 2 * a.Hkv + 512 / D - 1) / (512 / D);
    a.chunks = small ? a.groups : (a.groups + T - 1) / T;
    const int64_t tasks = a.total_q * a.chunks;
    a.narrow = tasks < (1LL << 31);
    const int64_t row_blocks = (tasks + kNormWarps - 1) / kNormWarps;
    const int64_t blocks = row_blocks + (std::max(a.n_seq, a.rot / 2) + kNormWarps * 32 - 1) / (kNormWarps * 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.row_blocks = (uint32_t)row_blocks;
    if (small)
        return dghost::launch_pdl(k_kv_append_norm<Interleaved, D, 1>, dim3((unsigned)blocks), dim3(kNormWarps * 32),
                                  kNormWarps * 1024, stream, a);
    constexpr int kBytes = kNormWarps * T * 1024;
    // the attribute once a device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        e = cudaFuncSetAttribute(k_kv_append_norm<Interleaved, D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return dghost::launch_pdl(k_kv_append_norm<Interleaved, D, T>, dim3((unsigned)blocks), dim3(kNormWarps * 32), kBytes, stream, a);
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

namespace {

// Checks and arguments shared by dg_kv_append and dg_kv_append_norm; false: `rc` is the answer.
bool append_args(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, const uint16_t* q, int64_t ldq,
                 uint16_t* q_out, const int32_t* cu_q, int32_t n_seq, int64_t total_q, int32_t Hq, int32_t Hkv, int32_t D,
                 const double* inv_freq, int32_t rot_dim, const dg_paged_kv* cache, AppendArgs& a, dg_status& rc) {
    auto answer = [&](dg_status s) {
        rc = s;
        return false;
    };
    if (n_seq < 0 || n_seq > 65535 || total_q < 0 || total_q >= (1LL << 31) || Hq < 1 || Hq > 65535 || Hkv < 1 ||
        Hkv > 65535)
        return answer(DG_ERR_INVALID_ARG);
    if (D != 64 && D != 128 && D != 256) return answer(DG_ERR_UNSUPPORTED);
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 || (rot_dim > 0 && !inv_freq)) return answer(DG_ERR_INVALID_ARG);
    if (n_seq == 0 || total_q == 0) return answer(DG_OK);
    if (!k || !v || !cu_q || (q != nullptr) != (q_out != nullptr)) return answer(DG_ERR_INVALID_ARG);
    if (ldk < (int64_t)Hkv * D || ldv < (int64_t)Hkv * D || (q && ldq < (int64_t)Hq * D)) return answer(DG_ERR_INVALID_ARG);
    if (ldk >= (1LL << 31) || ldv >= (1LL << 31) || (q && ldq >= (1LL << 31))) return answer(DG_ERR_INVALID_ARG);
    if (q && q_out == q && ldq != (int64_t)Hq * D) return answer(DG_ERR_INVALID_ARG);
    if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) || ldk % 8 || ldv % 8 ||
        (q && ldq % 8) || !dghost::on_multiple(cu_q, 4) || !dghost::on_multiple(inv_freq, 8))
        return answer(DG_ERR_ALIGNMENT);
    const dg_status ok = dghost::paged_kv(cache, D, &a.kv);
    if (ok != DG_OK) return answer(ok);
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
    return true;
}

}  // namespace

extern "C" dg_status dg_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, const uint16_t* q,
                                  int64_t ldq, uint16_t* q_out, const int32_t* cu_q, int32_t n_seq, int64_t total_q,
                                  int32_t Hq, int32_t Hkv, int32_t D, const double* inv_freq, int32_t rot_dim,
                                  int32_t interleaved, const dg_paged_kv* cache, dg_stream_t stream) {
    AppendArgs a;
    dg_status rc;
    if (!append_args(k, ldk, v, ldv, q, ldq, q_out, cu_q, n_seq, total_q, Hq, Hkv, D, inv_freq, rot_dim, cache, a, rc)) return rc;
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

extern "C" dg_status dg_kv_append_norm(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, const uint16_t* q,
                                       int64_t ldq, uint16_t* q_out, const int32_t* cu_q, int32_t n_seq, int64_t total_q,
                                       int32_t Hq, int32_t Hkv, int32_t D, const float* q_norm, const float* k_norm,
                                       float eps, const int32_t* positions, const double* inv_freq, int32_t rot_dim,
                                       int32_t interleaved, const dg_paged_kv* cache, dg_stream_t stream) {
    if ((q_norm || k_norm) && !(eps >= 0x1p-126f && eps < INFINITY)) return DG_ERR_INVALID_ARG;
    NormArgs a;
    dg_status rc;
    if (!append_args(k, ldk, v, ldv, q, ldq, q_out, cu_q, n_seq, total_q, Hq, Hkv, D, inv_freq, rot_dim, cache, a, rc)) return rc;
    if (q_norm && !q) return DG_ERR_INVALID_ARG;
    if (!dghost::on_multiple(q_norm, 4) || !dghost::on_multiple(k_norm, 4) || !dghost::on_multiple(positions, 4))
        return DG_ERR_ALIGNMENT;
    a.norm[0] = k_norm;
    a.norm[1] = q_norm;
    a.positions = positions;
    a.eps = eps;
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    // One group of heads a warp while they all run at once, then eight (us one / eight, rows of 16 / 8 heads of 128: 64 3.6 /
    // 5.9, 256 4.1 / 6.0, 512 5.3 / 6.2, 1024 8.5 / 7.0).
    const bool small = total_q * a.tasks <= (int64_t)sms * 1152;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (D == 64)
        e = interleaved ? launch_norm<true, 64>(a, small, st) : launch_norm<false, 64>(a, small, st);
    else if (D == 128)
        e = interleaved ? launch_norm<true, 128>(a, small, st) : launch_norm<false, 128>(a, small, st);
    else
        e = interleaved ? launch_norm<true, 256>(a, small, st) : launch_norm<false, 256>(a, small, st);
    if (e == cudaErrorInvalidConfiguration) return DG_ERR_INVALID_ARG;
    dghost::count_launch();
    return dghost::cuda_status(e);
}
