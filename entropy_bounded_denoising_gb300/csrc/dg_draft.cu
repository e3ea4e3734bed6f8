// dg_draft.cu -- what follows a pass over drafted tokens: the walk that accepts them against the target's
// distribution (dg_verify_drafts) and the accepted path kept in the cache (dg_kv_keep).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dg_paged.cuh"

namespace cg = cooperative_groups;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------------ verification
// A cluster of CTAs owns a sequence and walks its tree, so that only the rows on the walk are read: all of a
// cluster's threads take the statistics of one row, its first CTA decides which child goes on and tells the
// others.  The token after the path is drawn by inversion: the weights of the last row, as 64-bit fixed point, are
// summed by warps (each of which owns a contiguous part of the row), the first CTA finds the CTA in whose part the
// threshold falls, and there a warp walks its part again.
//
// Precision.  A token is drawn wrongly when an error of the cumulated probability moves a token's border past
// the random number: with errors e, about e times the number of tokens.  Weights in plain fp32 (2^-25 each) would
// miss one draw in a thousand on 262144 tokens; here a weight is 2^(j / 64) from a table of 62 bits times 2^g, |g| <= 1/128,
// by its Taylor polynomial, within 2^-31 of the exact one, and the sums are exact, whatever their order.
// Acceptance compares with fp32 sums, unless they come within their own bound of the border: then the row
// is summed like the last one (`kSum`) and compared again.
constexpr int kVThreads = 512, kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxNodes = 1024;

// 2^(j / 64) 2^62, rounded.
__constant__ uint64_t kPow[64] = {
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull, 0x42d561b3e6243d8aull,
    0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull, 0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull,
    0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull, 0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull,
    0x4b4a169b900c2d00ull, 0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full, 0x52ff6b54d8a89c75ull,
    0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull, 0x56ac1f752150a563ull, 0x579dbc56b48521baull,
    0x5891fac0e95612c8ull, 0x5988e20954889245ull, 0x5a827999fcef3242ull, 0x5b7ec8f19468bbc9ull, 0x5c7dd7a3b17dcf75ull,
    0x5d7fad59099f22feull, 0x5e8451cfac061b5full, 0x5f8bccdb3d398841ull, 0x6096266533384a2bull, 0x61a3666d124bb204ull,
    0x62b39508aa836d6full, 0x63c6ba6455dcd8aeull, 0x64dcdec3371793d1ull, 0x65f60a7f79393e2eull, 0x6712460a8fc24072ull,
    0x683199ed779592caull, 0x69540ec8f895722dull, 0x6a79ad55e7f6fd10ull, 0x6ba27e656b4eb57aull, 0x6cce8ae13c57ebdbull,
    0x6dfddbcbed791babull, 0x6f307a412f074892ull, 0x70666f76154a7089ull, 0x719fc4b95f452d29ull, 0x72dc8373be41a454ull,
    0x741cb5281e25ee34ull, 0x75606373ee921c97ull, 0x76a7980f6cca15c2ull, 0x77f25ccdee6d7ae6ull, 0x7940bb9e2cffd89dull,
    0x7a92be8a92436616ull, 0x7be86fb985689ddcull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull};

struct VerifyArgs {
    const void* logits;
    const int32_t* tokens;
    const int32_t* parents;
    const float* probs;
    const int32_t* cu_q;
    const float *temperature, *uniforms, *next_uniforms;
    int32_t *n_accept, *path, *out_tokens;
    int64_t ld, ldq, total, V;
    int32_t n_seq, frac;      // frac: bits of a weight below the point (a row's sum stays below 2^63)
    unsigned* status;
};

enum : int { kStats, kSum, kLeft, kFind, kExit };

// What the first CTA tells the others to do with a row.
struct Command {
    int op;
    int node;          // row of the sequence
    int minus;         // kSum, and kFind after it: 1: leave out the tokens of the node's children; -1: for a decision
    int draft;         // kLeft, and kFind after it: the rejected draft (else -1)
    int cta;           // kFind: the CTA that finds the token,
    float top;         // the row's maximum
    uint64_t total;    // kLeft: the row's sum
    uint64_t target;   // kFind: the sum to pass, counted from that CTA's part
    int64_t out;       // and the place of the token
};

struct Partial {       // of one CTA: kStats: maximum, sum, its place, 0 / 1: a NaN or +inf; kSum, kLeft: sum
    float top, sum;
    int arg, bad;
    uint64_t fixed;
};

struct __align__(16) VShared {
    Command cmd;
    Partial part[kMaxCluster];        // in the first CTA: everyone's
    uint64_t warp_sum[kVWarps];       // fixed-point sums of the warps' parts
    float w_top[kVWarps], w_sum[kVWarps];
    int w_arg[kVWarps], w_bad[kVWarps];
    float c_hi, c_lo;                 // log2(e) / temperature
    int n_gone;                       // rejected tokens of the last node that lie in this CTA's part
    int gone[kMaxNodes];
    int path[kMaxNodes];              // the first CTA's
    int rejected[kMaxNodes];
    uint64_t pow[64];
};

template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
};

// The logits of a vector: 16 bytes at vector v of a row; -inf from V on.
template <typename T>
DG_DEVINL void unpack(const uint4& r, int64_t v, int64_t V, float (&x)[Vec<T>::kN]) {
    constexpr int N = Vec<T>::kN;
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if constexpr (sizeof(T) == 2)
            x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else
            x[e] = __uint_as_float(w[e]);
    }
    if ((v + 1) * N > V) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (v * N + e >= V) x[e] = -INFINITY;
    }
}

DG_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^((x - top) c) as mantissa m in [2^62, 2^63) (a little above at most) and exponent n <= 0: m 2^(n - 62).  The exponent
// in two floats: the difference (its own rounding kept where both are fp32), its product with c; then 2^(j / 64)
// 2^g with the polynomial's terms up to g^4 (the next is below 2^-44).
template <typename T>
DG_DEVINL uint64_t weight(float x, float top, float c_hi, float c_lo, const uint64_t* pow, int& n) {
    const float d = x - top;
    float hi = d * c_hi;
    float lo = fmaf(d, c_hi, -hi);
    lo = fmaf(d, c_lo, lo);
    if constexpr (sizeof(T) == 4) {   // and what x - top lost
        const float z = d - x;
        lo = fmaf((x - (d - z)) - (top + z), c_hi, lo);
    }
    if (!(hi > -200.f)) {             // nothing at any place after the point (and no index out of the table)
        n = -200;
        return 1ull << 62;
    }
    const float t = fmaf(hi, 64.f, 12582912.f);   // 1.5 2^23: rounds to a whole number
    const int k = __float_as_int(t) - 0x4b400000;
    float g = fmaf(t - 12582912.f, -0.015625f, hi);
    g += lo;
    const float e = g * fmaf(g, fmaf(g, fmaf(g, 9.6181291e-3f, 5.5504109e-2f), 0.24022651f), 0.69314718f);
    const uint64_t h = pow[k & 63];
    const float hf = (float)(uint32_t)(h >> 32);  // in units of 2^-30
    const int s = __float2int_rn(hf * e * 128.f); // |e| < 2^-7: units of 2^-37, below 2^31
    n = k >> 6;
    return h + ((uint64_t)(int64_t)s << 25);
}

// The same with `frac` bits after the point, rounded.
template <typename T>
DG_DEVINL uint64_t fixed_weight(float x, float top, float c_hi, float c_lo, const uint64_t* pow, int frac) {
    int n;
    const uint64_t m = weight<T>(x, top, c_hi, c_lo, pow, n);
    const int s = 62 - frac - n;      // >= 18
    return s > 63 ? 0ull : (m + (1ull << (s - 1))) >> s;
}

DG_DEVINL float unit(float q) { return fminf(fmaxf(q, 0.f), 1.f); }   // (a NaN is 0)

// w - q total, or 0: q in [0, 1] a float, so the product is a 24-bit number times the total, shifted.
DG_DEVINL uint64_t left_of(uint64_t w, float q, uint64_t total) {
    q = unit(q);
    const uint32_t b = __float_as_uint(q), e = b >> 23;
    if (e >= 127) return 0;           // 1: more than any weight
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int s = 150 - (e ? (int)e : 1);   // 24 .. 149
    const uint64_t lo = m * total, hi = __umul64hi(m, total);
    uint64_t p;
    if (s < 64)
        p = (lo >> s) | (hi << (64 - s));
    else
        p = s < 128 ? hi >> (s - 64) : 0;
    return w > p ? w - p : 0;
}

DG_DEVINL uint64_t warp_add(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The part of a row that a warp of the cluster owns, in vectors.
struct Part {
    int64_t from, to;
};
template <typename T>
DG_DEVINL Part part_of(int64_t V, int cta, int n_cta, int warp) {
    const int64_t nv = (V + Vec<T>::kN - 1) / Vec<T>::kN;
    const int64_t each = (nv + (int64_t)n_cta * kVWarps * 32 - 1) / ((int64_t)n_cta * kVWarps * 32) * 32;
    const int64_t from = ((int64_t)cta * kVWarps + warp) * each;
    return Part{min(from, nv), min(from + each, nv)};
}
// and who owns a token.
template <typename T>
DG_DEVINL int part_with(int64_t V, int n_cta, int64_t token) {
    const int64_t nv = (V + Vec<T>::kN - 1) / Vec<T>::kN;
    const int64_t each = (nv + (int64_t)n_cta * kVWarps * 32 - 1) / ((int64_t)n_cta * kVWarps * 32) * 32;
    return (int)(token / Vec<T>::kN / each);
}

// A row's maximum, its smallest place, and (with Sum) sum of 2^((x - maximum) c), of this CTA's part.
template <typename T, bool Sum>
DG_DEVINL void row_stats(VShared& sh, const T* row, int64_t V, int cta, int n_cta, Partial* to) {
    constexpr int N = Vec<T>::kN, kDeep = 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Part p = part_of<T>(V, cta, n_cta, warp);
    const uint4* src = reinterpret_cast<const uint4*>(row);
    const float c = sh.c_hi;
    float top = -INFINITY, sum = 0.f;
    int arg = 0x7fffffff;
    bool bad = false;
    for (int64_t v0 = p.from + lane; v0 < p.to; v0 += 32 * kDeep) {
        uint4 r[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (v0 + k * 32 < p.to) r[k] = __ldg(src + v0 + k * 32);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int64_t v = v0 + k * 32;
            if (v >= p.to) break;
            float x[N];
            unpack<T>(r[k], v, V, x);
            float most = x[0];
#pragma unroll
            for (int e = 1; e < N; ++e) most = fmaxf(most, x[e]);
            if constexpr (Sum) {
                if (most > top) {
                    sum *= ex2((top - most) * c);   // (0 of -inf: 0 stays 0)
                    top = most;
                }
                const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int e = 0; e < N; ++e) sum += ex2((x[e] - at) * c);   // a NaN or +inf makes it a NaN
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) bad = bad || !(x[e] < INFINITY);
                if (most > top) {
                    top = most;
#pragma unroll
                    for (int e = N - 1; e >= 0; --e)
                        if (x[e] == most) arg = (int)(v * N + e);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, top, o);
        const float m = fmaxf(top, t);
        if constexpr (Sum) {
            const float s = __shfl_xor_sync(0xffffffffu, sum, o);
            const float at = m == -INFINITY ? 0.f : m;
            sum = sum * ex2((top - at) * c) + s * ex2((t - at) * c);
        } else {
            const int g = __shfl_xor_sync(0xffffffffu, arg, o);
            arg = t > top ? g : t == top ? min(arg, g) : arg;
            bad = bad | __shfl_xor_sync(0xffffffffu, (int)bad, o);
        }
        top = m;
    }
    if (lane == 0) {
        sh.w_top[warp] = top;
        sh.w_sum[warp] = sum;
        sh.w_arg[warp] = arg;
        sh.w_bad[warp] = bad;
    }
    __syncthreads();
    if (tid == 0) {
        Partial q{-INFINITY, 0.f, 0x7fffffff, 0, 0};
        for (int w = 0; w < kVWarps; ++w) q.top = fmaxf(q.top, sh.w_top[w]);
        const float at = q.top == -INFINITY ? 0.f : q.top;
        for (int w = 0; w < kVWarps; ++w) {
            q.sum += sh.w_sum[w] * ex2((sh.w_top[w] - at) * c);
            if (sh.w_top[w] == q.top) q.arg = min(q.arg, sh.w_arg[w]);
            q.bad |= sh.w_bad[w];
        }
        *to = q;
    }
}

// The fixed-point weights of a vector.
template <typename T>
DG_DEVINL void vector_weights(const VShared& sh, const uint4& r, int64_t v, int64_t V, float top, int frac,
                              const float* q_row, uint64_t total, uint64_t (&w)[Vec<T>::kN]) {
    constexpr int N = Vec<T>::kN;
    float x[N];
    unpack<T>(r, v, V, x);
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = fixed_weight<T>(x[e], top, sh.c_hi, sh.c_lo, sh.pow, frac);
    if (q_row) {   // (four probabilities that begin before V end within the row; weights from V on are 0)
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
            if (v * N + 4 * h >= V) continue;
            const float4 q = __ldg(reinterpret_cast<const float4*>(q_row + v * N) + h);
            w[4 * h] = left_of(w[4 * h], q.x, total);
            w[4 * h + 1] = left_of(w[4 * h + 1], q.y, total);
            w[4 * h + 2] = left_of(w[4 * h + 2], q.z, total);
            w[4 * h + 3] = left_of(w[4 * h + 3], q.w, total);
        }
    }
}

// Sums of the weights by warp (q_row: of what a draft's distribution leaves of them), and the CTA's.
template <typename T>
DG_DEVINL void row_sums(VShared& sh, const T* row, const VerifyArgs& a, const Command& c, const float* q_row, int cta,
                        int n_cta, int q0, int ql, Partial* to) {
    constexpr int N = Vec<T>::kN;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Part p = part_of<T>(a.V, cta, n_cta, warp);
    const uint4* src = reinterpret_cast<const uint4*>(row);
    uint64_t sum = 0;
    for (int64_t v = p.from + lane; v < p.to; v += 32) {
        uint64_t w[N];
        vector_weights<T>(sh, __ldg(src + v), v, a.V, c.top, a.frac, q_row, c.total, w);
#pragma unroll
        for (int e = 0; e < N; ++e) sum += w[e];
    }
    sum = warp_add(sum);
    if (lane == 0) sh.warp_sum[warp] = sum;
    if (tid == 0) sh.n_gone = 0;
    __syncthreads();
    if (c.minus > 0) {   // the rejected children's tokens in this CTA's part, each once
        for (int i = c.node + 1 + tid; i < ql; i += kVThreads) {
            const int32_t t = a.tokens[q0 + i];
            if ((a.parents ? a.parents[q0 + i] : i - 1) != c.node || t < 0 || t >= a.V) continue;
            const int owner = part_with<T>(a.V, n_cta, t);
            if (owner / kVWarps != cta) continue;
            bool again = false;
            for (int k = c.node + 1; k < i && !again; ++k)
                again = a.tokens[q0 + k] == t && (a.parents ? a.parents[q0 + k] : k - 1) == c.node;
            if (again) continue;
            float x;
            if constexpr (sizeof(T) == 2)
                x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[t] << 16);
            else
                x = reinterpret_cast<const float*>(row)[t];
            const uint64_t w = fixed_weight<T>(x, c.top, sh.c_hi, sh.c_lo, sh.pow, a.frac);
            atomicAdd((unsigned long long*)&sh.warp_sum[owner % kVWarps], (unsigned long long)(0 - w));
            const int at = atomicAdd(&sh.n_gone, 1);   // (in any order: the list is searched)
            if (at < kMaxNodes) sh.gone[at] = t;
        }
        __syncthreads();
    }
    if (tid == 0) {
        Partial q{};
        for (int w = 0; w < kVWarps; ++w) q.fixed += sh.warp_sum[w];
        *to = q;
    }
}

// The token whose cumulated weight passes the target, which lies in this CTA's part (warp_sum and gone are as row_sums left
// them for these weights).
template <typename T>
DG_DEVINL void find_token(VShared& sh, const T* row, const VerifyArgs& a, const Command& c, const float* q_row, int cta, int n_cta) {
    constexpr int N = Vec<T>::kN;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t target = c.target;
    int owner = 0;
    while (owner < kVWarps - 1 && target >= sh.warp_sum[owner]) target -= sh.warp_sum[owner++];
    if (warp != owner) return;
    const Part p = part_of<T>(a.V, cta, n_cta, warp);
    const uint4* src = reinterpret_cast<const uint4*>(row);
    for (int64_t v0 = p.from; v0 < p.to; v0 += 32) {
        const int64_t v = v0 + lane;
        uint64_t w[N], mine = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = 0;
        if (v < p.to) {
            vector_weights<T>(sh, __ldg(src + v), v, a.V, c.top, a.frac, q_row, c.total, w);
            if (c.minus > 0)
                for (int i = 0; i < min(sh.n_gone, kMaxNodes); ++i)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (v * N + e == sh.gone[i]) w[e] = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) mine += w[e];
        }
        uint64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, incl > target);
        if (past) {
            if (lane == __ffs(past) - 1) {
                uint64_t s = incl - mine;
                int at = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    s += w[e];
                    if (s <= target) at = e + 1;
                }
                a.out_tokens[c.out] = (int32_t)(v * N + at);
            }
            return;
        }
        target -= __shfl_sync(0xffffffffu, incl, 31);
    }
}

// The first CTA's first warp: tries the children of `node` in order.  The row's maximum and sum are given (fixed point when
// `exact`).  Returns the accepted child, -1: none, -2: too near to say with an fp32 sum.  `last`: the rejected draft.
template <typename T>
DG_DEVINL int decide(VShared& sh, const VerifyArgs& a, const T* row, int q0, int ql, int node, float T_, const Partial& st,
                     bool exact, int n_cta, int& last) {
    const int lane = threadIdx.x & 31;
    last = -1;
    // The sum's bound: its exponents' roundings (2^-23 of each, weighted by weights that fall faster than exponents
    // grow), the exponentials (2^-22), the joins, and 2^-24 an addition of a thread.
    const double sum = exact ? ldexp((double)st.fixed, -a.frac) : (double)st.sum;
    const double slack = exact ? 0.0 : sum * (0x1p-17 + (double)a.V / (n_cta * kVThreads) * 0x1p-24);
    double left = sum;
    int n_rejected = 0;
    const int end = a.parents ? ql : min(ql, node + 2);
    for (int base = node + 1; base < end; base += 32) {
        const int c = base + lane;
        const bool child = c < end && (a.parents ? a.parents[q0 + c] == node : true);
        int32_t token = -1;
        double w = 0.0, u = 0.0, q = 1.0;
        if (child) {
            token = a.tokens[q0 + c];
            if (T_ > 0.f) {
                u = a.uniforms[q0 + c];
                if (token >= 0 && token < a.V) {
                    float x;
                    if constexpr (sizeof(T) == 2)
                        x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[token] << 16);
                    else
                        x = reinterpret_cast<const float*>(row)[token];
                    int n;
                    const uint64_t m = weight<T>(x, st.top, sh.c_hi, sh.c_lo, sh.pow, n);
                    w = n <= -200 ? 0.0 : ldexp((double)m, n - 62);
                    if (a.probs) q = unit(a.probs[(int64_t)(q0 + c) * a.ldq + token]);
                }
            }
        }
        uint32_t todo = __ballot_sync(0xffffffffu, child);
        while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const int32_t t = __shfl_sync(0xffffffffu, token, from);
            if (T_ == 0.f) {
                if (t == st.arg) return base + from;
                last = base + from;
                continue;
            }
            const double wt = __shfl_sync(0xffffffffu, w, from), ut = __shfl_sync(0xffffffffu, u, from);
            const double qt = __shfl_sync(0xffffffffu, q, from);
            if (a.probs) {
                const double lhs = ut * qt * sum;
                if (fabs(lhs - wt) < ut * qt * slack) return -2;
                if (lhs < wt) return base + from;
            } else {
                bool again = false;
                for (int i = lane; i < n_rejected; i += 32) again = again || sh.rejected[i] == t;
                again = __any_sync(0xffffffffu, again);
                if (!again) {
                    const double lhs = ut * fmax(left, 0.0);
                    if (fabs(lhs - wt) < ut * slack) return -2;
                    if (lhs < wt) return base + from;
                    left -= wt;
                    if (lane == 0) sh.rejected[n_rejected] = t;
                    __syncwarp();
                    ++n_rejected;
                }
            }
            last = base + from;
        }
    }
    return -1;
}

template <typename T>
__global__ void __launch_bounds__(kVThreads, 2) k_verify(const VerifyArgs a) {
    __shared__ VShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    dg::pdl_wait();
    dg::pdl_release();
    const int n_cta = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    const int s = (int)(blockIdx.x / n_cta), tid = threadIdx.x, warp = tid >> 5;
    VShared* lead = cluster.map_shared_rank(&sh, 0);
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], ql = q1 - q0;
    const float T_ = a.temperature[s];
    if (tid < 64) sh.pow[tid] = kPow[tid];
    if (tid == 0) {
        const double c = T_ > 0.f ? 1.4426950408889634 / (double)T_ : 1.0;
        sh.c_hi = (float)c;
        sh.c_lo = (float)(c - (double)sh.c_hi);
    }
    // The first CTA alone looks at what decides how often the cluster meets.
    int node = 0, accepted = 0;
    bool walks = false;
    if (cta == 0) {
        const bool offsets = q0 >= 0 && q1 >= q0 && (int64_t)q1 <= a.total;
        bool good = offsets && ql <= kMaxNodes;
        if (good && ql > 0) {
            good = T_ == 0.f || (T_ >= 0x1p-64f && T_ < INFINITY);
            if (T_ != 0.f) good = good && a.next_uniforms[s] >= 0.f && a.next_uniforms[s] < 1.f;
            for (int i = 1 + tid; good && i < ql; i += kVThreads) {
                if (a.parents) good = good && a.parents[q0 + i] >= 0 && a.parents[q0 + i] < i;
                if (T_ != 0.f) good = good && a.uniforms[q0 + i] >= 0.f && a.uniforms[q0 + i] < 1.f;
            }
        }
        good = !__syncthreads_or(!good);
        walks = good && ql > 0;
        if (!walks) {
            if (offsets)
                for (int i = tid; i < ql; i += kVThreads) a.path[q0 + i] = a.out_tokens[q0 + i] = -1;
            if (tid == 0) {
                a.n_accept[s] = -1;
                if (!good) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            }
        }
    }
    cluster.sync();   // everyone runs before anyone writes to its shared memory

    auto tell = [&](const Command& c) {   // the first CTA's first threads: one command to every CTA
        if (tid < n_cta) *reinterpret_cast<Command*>(&cluster.map_shared_rank(&sh, tid)->cmd) = c;
    };
    // The first CTA's state between commands (the same in all its threads).
    Command next{kStats, 0, 0, -1, 0, 0.f, 0, 0, 0};
    if (cta == 0 && !walks) next.op = kExit;
    __shared__ int s_child, s_last;
    Partial stats{};            // of the row at `node`
    int rejected = -1;          // the draft rejected there
    uint64_t total = 0;
    while (true) {
        if (cta == 0) tell(next);
        cluster.sync();
        const Command c = sh.cmd;
        if (c.op == kExit) return;
        const T* row = reinterpret_cast<const T*>(a.logits) + (int64_t)(q0 + c.node) * a.ld;
        const float* q_row = c.draft >= 0 ? a.probs + (int64_t)(q0 + c.draft) * a.ldq : nullptr;
        if (c.op == kFind) {
            if (cta == c.cta) find_token<T>(sh, row, a, c, q_row, cta, n_cta);
            return;
        }
        if (c.op == kStats) {
            if (T_ > 0.f)
                row_stats<T, true>(sh, row, a.V, cta, n_cta, &lead->part[cta]);
            else
                row_stats<T, false>(sh, row, a.V, cta, n_cta, &lead->part[cta]);
        } else {
            row_sums<T>(sh, row, a, c, q_row, cta, n_cta, q0, ql, &lead->part[cta]);
        }
        cluster.sync();
        if (cta != 0) continue;

        // The first CTA decides what comes next.
        bool finish = false, no_token = false;
        auto draw_from = [&](uint64_t sum) {   // the token past next_uniforms * sum
            const float u = a.next_uniforms[s];
            const uint64_t U = (uint64_t)__float2ull_rz(u * 0x1p32f) << 32 |
                               __float2ull_rz((u * 0x1p32f - truncf(u * 0x1p32f)) * 0x1p32f);
            uint64_t target = __umul64hi(sum, U);
            int owner = 0;
            while (owner < n_cta - 1 && target >= sh.part[owner].fixed) target -= sh.part[owner++].fixed;
            next.op = kFind;
            next.cta = owner;
            next.target = target;
            next.out = q0 + accepted;
        };
        if (c.op == kStats) {
            Partial t{-INFINITY, 0.f, 0x7fffffff, 0, 0};
            for (int i = 0; i < n_cta; ++i) t.top = fmaxf(t.top, sh.part[i].top);
            const float at = t.top == -INFINITY ? 0.f : t.top;
            for (int i = 0; i < n_cta; ++i) {
                t.sum += sh.part[i].sum * ex2((sh.part[i].top - at) * sh.c_hi);
                if (sh.part[i].top == t.top) t.arg = min(t.arg, sh.part[i].arg);
                t.bad |= sh.part[i].bad;
            }
            stats = t;
            const bool nan = t.bad || !(t.top < INFINITY) || !(t.sum < INFINITY);
            if (nan || t.top == -INFINITY) {
                if (tid == 0) dg::raise_status(a.status, nan ? DG_DEV_NAN_INF_ROW : DG_DEV_EMPTY_ROW);
                finish = no_token = true;
            }
        } else {
            uint64_t f = 0;
            for (int i = 0; i < n_cta; ++i) f += sh.part[i].fixed;
            stats.fixed = f;
        }
        if (!finish && (c.op == kStats || (c.op == kSum && c.minus < 0))) {   // (minus -1: a sum asked for by a decision)
            __syncthreads();
            if (warp == 0) {
                int last;
                const int child = decide<T>(sh, a, row, q0, ql, c.node, T_, stats, c.op == kSum, n_cta, last);
                if (tid == 0) {
                    s_child = child;
                    s_last = last;
                }
            }
            __syncthreads();
            const int child = s_child;
            next = Command{kStats, c.node, 0, -1, 0, stats.top, 0, 0, 0};
            if (child == -2) {
                next.op = kSum;
                next.minus = -1;
            } else if (child >= 0) {
                if (tid == 0) {
                    sh.path[accepted] = child;
                }
                node = child;
                ++accepted;
                next.node = child;
            } else {
                rejected = s_last;
                if (T_ == 0.f) {
                    if (tid == 0) a.out_tokens[q0 + accepted] = stats.arg;
                    finish = true;
                } else {
                    next.op = kSum;
                    next.minus = rejected >= 0 && !a.probs ? 1 : 0;
                }
            }
        } else if (!finish && c.op == kSum) {
            total = stats.fixed;
            if (a.probs && rejected >= 0) {
                next.op = kLeft;
                next.draft = rejected;
                next.total = total;
            } else if (c.minus > 0 && total == 0) {
                next.minus = 0;          // nothing is left: all of the row again
            } else {
                draw_from(total);
            }
        } else if (!finish) {            // kLeft
            if (stats.fixed == 0) {      // nothing is left: the row itself, whose sums are made again
                rejected = -1;
                next = Command{kSum, c.node, 0, -1, 0, stats.top, 0, 0, 0};
            } else {
                draw_from(stats.fixed);
            }
        }
        if (finish || next.op == kFind) {   // the walk's outputs
            __syncthreads();
            for (int i = tid; i < ql; i += kVThreads) {
                a.path[q0 + i] = i == 0 ? 0 : i <= accepted ? sh.path[i - 1] : -1;
                if (i < accepted)
                    a.out_tokens[q0 + i] = a.tokens[q0 + sh.path[i]];
                else if (i > accepted || no_token)
                    a.out_tokens[q0 + i] = -1;
            }
            if (tid == 0) a.n_accept[s] = accepted;
            if (finish) next.op = kExit;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ kept paths
// A thread owns 16 bytes of a head in one layer's keys or values and takes the path's nodes in order.  Node path[i] goes to
// slot i <= path[i] behind the context, and every later node lies at path[k] >= k > i: nothing is overwritten
// before it is read.
constexpr int kKeepThreads = 256;
constexpr int kKeepChunk = 256;    // moves whose places are worked out at a time

struct KeepArgs {
    dg::PagedKV kv;
    const int32_t *cu_q, *path, *n_accept;
    int32_t* new_len;
    int64_t layer_stride, total_q, columns;   // columns: 16-byte columns of all layers, keys and values
    int32_t n_seq, n_layers, row_chunks, head_chunks;   // chunks of a token's row in one layer, of a head
    unsigned* status;
};

__global__ void __launch_bounds__(kKeepThreads) k_kv_keep(const KeepArgs a) {
    __shared__ int64_t src[kKeepChunk], dst[kKeepChunk];
    dg::pdl_wait();
    dg::pdl_release();
    const int s = blockIdx.y, tid = threadIdx.x;
    const int32_t kept = a.n_accept[s], q0 = a.cu_q[s], q1 = a.cu_q[s + 1], kl = a.kv.kv_len[s];
    const int ql = q1 - q0;
    bool good = q0 >= 0 && q1 >= q0 && (int64_t)q1 <= a.total_q && kl >= ql && (int64_t)kl <= a.kv.capacity() && kept < ql &&
                kept >= -1;
    if (kept == -1) good = true;
    const int ctx = kl - ql;
    const int32_t* table = a.kv.page_table + (int64_t)s * a.kv.max_pages;
    auto place = [&](int p, bool& ok) -> int64_t {
        const int32_t page = table[p >> a.kv.page_shift];
        ok = ok && page >= 0 && page < a.kv.n_pages;
        return page * a.kv.page_stride + (p & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride;
    };
    const int n = good ? kept + 1 : 0;
    int64_t from = 0, to = 0;      // of this thread's first node
    for (int i = tid; i < n; i += kKeepThreads) {
        const int32_t x = a.path[q0 + i], before = i ? a.path[q0 + i - 1] : -1;
        bool ok = x > before && x < ql && x >= 0;
        if (ok && x != i) {
            const int64_t f = place(ctx + x, ok), t = place(ctx + i, ok);
            if (i == tid) {
                from = f;
                to = t;
            }
        }
        good = good && ok;
    }
    good = !__syncthreads_or(!good);
    if (tid == 0 && blockIdx.x == 0) {
        if (!good) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        a.new_len[s] = good && kept >= 0 ? ctx + n : kl;
    }
    if (!good) return;
    const int64_t column = (int64_t)blockIdx.x * kKeepThreads + tid;
    const bool mine = column < a.columns;
    const int64_t plane = column / a.row_chunks;   // 2 layer + (0: keys, 1: values)
    const int chunk = (int)(column - plane * a.row_chunks), head = chunk / a.head_chunks;
    uint16_t* base = (plane & 1 ? a.kv.v : a.kv.k) + (plane >> 1) * a.layer_stride + head * a.kv.head_stride +
                     (chunk - head * a.head_chunks) * 8;
    for (int i0 = 0; i0 < n; i0 += kKeepChunk) {
        if (i0) __syncthreads();
        const int i = i0 + tid;
        if (i < n) {
            const int32_t x = a.path[q0 + i];
            bool ok = true;
            if (i0 && x != i) {
                from = place(ctx + x, ok);
                to = place(ctx + i, ok);
            }
            src[tid] = x != i && ok ? from : -1;
            dst[tid] = to;
        }
        __syncthreads();
        if (!mine) continue;
        const int m = min(kKeepChunk, n - i0);
        constexpr int kDeep = 4;
        for (int k = 0; k < m; k += kDeep) {
            uint4 r[kDeep];
#pragma unroll
            for (int e = 0; e < kDeep; ++e)
                if (k + e < m && src[k + e] >= 0) r[e] = *reinterpret_cast<const uint4*>(base + src[k + e]);
#pragma unroll
            for (int e = 0; e < kDeep; ++e)
                if (k + e < m && src[k + e] >= 0) *reinterpret_cast<uint4*>(base + dst[k + e]) = r[e];
        }
    }
}

}  // namespace

extern "C" dg_status dg_verify_drafts(const void* logits, dg_dtype dtype, int64_t ld, const int32_t* tokens,
                                      const int32_t* parents, const float* draft_probs, int64_t ldq, const int32_t* cu_q,
                                      int32_t n_seq, int64_t total, int64_t V, const float* temperature,
                                      const float* uniforms, const float* next_uniforms, int32_t* n_accept, int32_t* path,
                                      int32_t* out_tokens, dg_stream_t stream) {
    if (n_seq < 0 || n_seq > 65535 || total < 0 || total >= (1LL << 31) || V < 2 || V >= (1LL << 30) || ld < V ||
        (dtype != DG_BF16 && dtype != DG_FP32) || (parents && draft_probs) || (draft_probs && ldq < V))
        return DG_ERR_INVALID_ARG;
    const int64_t es = dtype == DG_BF16 ? 2 : 4;
    if (V * es >= (1LL << 31)) return DG_ERR_UNSUPPORTED;
    if (n_seq == 0) return DG_OK;
    if (!cu_q || !temperature || !next_uniforms || !n_accept) return DG_ERR_INVALID_ARG;
    if (total > 0 && (!logits || !tokens || !uniforms || !path || !out_tokens)) return DG_ERR_INVALID_ARG;
    if (ld >= (1LL << 40) || (draft_probs && ldq >= (1LL << 40))) return DG_ERR_INVALID_ARG;
    if (!aligned16(logits) || ld * es % 16 || !aligned16(draft_probs) || (draft_probs && ldq % 4)) return DG_ERR_ALIGNMENT;
    const void* words[] = {tokens, parents, cu_q, temperature, uniforms, next_uniforms, n_accept, path, out_tokens};
    for (const void* p : words)
        if (!dghost::on_multiple(p, 4)) return DG_ERR_ALIGNMENT;
    VerifyArgs a;
    a.logits = logits;
    a.tokens = tokens;
    a.parents = parents;
    a.probs = draft_probs;
    a.cu_q = cu_q;
    a.temperature = temperature;
    a.uniforms = uniforms;
    a.next_uniforms = next_uniforms;
    a.n_accept = n_accept;
    a.path = path;
    a.out_tokens = out_tokens;
    a.ld = ld;
    a.ldq = ldq;
    a.total = total;
    a.V = V;
    a.n_seq = n_seq;
    int bits = 1;
    while ((1LL << bits) < V) ++bits;
    a.frac = std::min(44, 62 - bits);
    a.status = dghost::status_word();
    const int cluster = 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_seq * cluster);
    cfg.blockDim = dim3(kVThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dghost::kPdl ? 2 : 1;
    const cudaError_t e = dtype == DG_BF16 ? cudaLaunchKernelEx(&cfg, k_verify<uint16_t>, a) : cudaLaunchKernelEx(&cfg, k_verify<float>, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}

extern "C" dg_status dg_kv_keep(const dg_paged_kv* cache, int32_t n_layers, int64_t layer_stride, const int32_t* cu_q,
                                int32_t n_seq, int64_t total_q, int32_t Hkv, int32_t D, const int32_t* path,
                                const int32_t* n_accept, int32_t* new_len, dg_stream_t stream) {
    if (n_seq < 0 || n_seq > 65535 || total_q < 0 || total_q >= (1LL << 31) || Hkv < 1 || Hkv > 65535 || n_layers < 1 ||
        n_layers > 65535)
        return DG_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return DG_ERR_UNSUPPORTED;
    if (n_layers > 1 && (layer_stride >= (1LL << 55) || layer_stride <= -(1LL << 55))) return DG_ERR_INVALID_ARG;
    if (n_seq == 0) return DG_OK;
    if (!cu_q || !n_accept || !new_len || (total_q > 0 && !path)) return DG_ERR_INVALID_ARG;
    KeepArgs a;
    const dg_status ok = dghost::paged_kv(cache, D, &a.kv);
    if (ok != DG_OK) return ok;
    for (const int32_t* p : {cache->kv_len, n_accept}) {   // what other blocks of the sequence still read
        const uintptr_t from = reinterpret_cast<uintptr_t>(new_len), at = reinterpret_cast<uintptr_t>(p);
        if (from < at + 4 * (uintptr_t)n_seq && at < from + 4 * (uintptr_t)n_seq) return DG_ERR_INVALID_ARG;
    }
    if (n_layers > 1 && layer_stride % 8) return DG_ERR_ALIGNMENT;
    if (!dghost::on_multiple(cu_q, 4) || !dghost::on_multiple(path, 4) || !dghost::on_multiple(n_accept, 4) ||
        !dghost::on_multiple(new_len, 4))
        return DG_ERR_ALIGNMENT;
    a.cu_q = cu_q;
    a.path = path;
    a.n_accept = n_accept;
    a.new_len = new_len;
    a.layer_stride = n_layers > 1 ? layer_stride : 0;
    a.total_q = total_q;
    a.n_seq = n_seq;
    a.n_layers = n_layers;
    a.head_chunks = D / 8;
    a.row_chunks = Hkv * (D / 8);
    a.columns = (int64_t)n_layers * 2 * a.row_chunks;
    a.status = dghost::status_word();
    const int64_t blocks = (a.columns + kKeepThreads - 1) / kKeepThreads;
    if (blocks > 0x7fffffffLL) return DG_ERR_INVALID_ARG;
    const cudaError_t e = dghost::launch_pdl(k_kv_keep, dim3((unsigned)blocks, (unsigned)n_seq), dim3(kKeepThreads), 0,
                                             (cudaStream_t)stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}
