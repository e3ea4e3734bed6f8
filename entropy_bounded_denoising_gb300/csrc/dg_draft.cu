// dg_draft.cu -- what follows a pass over drafted tokens: the walk that accepts them against the target's
// distribution (dg_verify_drafts) and the accepted path kept in the cache (dg_kv_keep).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "dg_paged.cuh"

namespace cg = cooperative_groups;

namespace {

// 16 bytes into the shared memory of a CTA of the cluster, counted by the barrier there once they lie in their place (one
// trip; a store, and an arrival that waits for it, take two).
DG_DEVINL void send16(uint32_t to, const uint4& v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
                 : "memory");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------------ verification
// A cluster of CTAs owns a sequence and walks its tree, so that only the rows on the walk are read: all of a
// cluster's threads take the statistics of one row, its first CTA (the lead) decides which child goes on and tells the
// others.  CTAs leave their parts in the lead's shared memory and arrive on its barrier, the lead leaves its command in
// theirs: bounded waits between two CTAs, not barriers of all threads.  The token after the path is drawn by inversion:
// the weights of the last row, as 64-bit fixed point, are summed by warps (each of which owns a contiguous part of the
// row), the lead finds the CTA in whose part the threshold falls, and there the warps halve the part of the owner
// between them until one vector is left.
//
// Precision.  A token is drawn wrongly when an error of the cumulated probability moves a token's border past
// the random number: with errors e, about e times the number of tokens.  Weights in plain fp32 (2^-25 each) would
// miss one draw in a thousand on 262144 tokens; here a weight is 2^(j / 32) from a table times 2^g, |g| <= 1/64, by its
// Taylor polynomial, in two floats within 2^-31 of the exact one (2^-32 as a rule).  The two are added up over a vector
// of 16 bytes so that nothing is lost (multiples of 2^-20 exactly, what is left within 2^-43), turned into fixed point, and
// added exactly from there on, whatever the order.
// Acceptance compares fp32 sums, unless they come within their own bound of the border: then the row is summed
// like the last one (kSum) and compared again.
//
// Measured: one chain of 5 drafts over 32768 tokens, bf16, 9 to 18 us by what is accepted: a node takes 3 to 4, the row's
// maximum, its sum and the two trips to and from the lead.  64 trees of 32 over 262144 tokens 61 to 64 us, where the bytes of
// the rows walked take 8: the sums of a row that decides, some 47 lane cycles a token, and sequences that walk further than
// others.  With weights in plain instead of packed pairs of fp32 7 us more, with CTAs of 256 threads, two an SM, too.
constexpr int kVThreads = 128, kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxNodes = 1024;
constexpr int kSegments = 64;      // that a part is searched in at a time
constexpr int kDeep = 5;           // vectors a lane has on their way

// 2^(j / 32), rounded, and what the rounding left out, relative.
__constant__ float kPow[32] = {
    0x1.0000000000000p+0f, 0x1.059b0e0000000p+0f, 0x1.0b55860000000p+0f, 0x1.11301e0000000p+0f,
    0x1.172b840000000p+0f, 0x1.1d48740000000p+0f, 0x1.2387a60000000p+0f, 0x1.29e9e00000000p+0f,
    0x1.306fe00000000p+0f, 0x1.371a740000000p+0f, 0x1.3dea640000000p+0f, 0x1.44e0860000000p+0f,
    0x1.4bfdae0000000p+0f, 0x1.5342b60000000p+0f, 0x1.5ab07e0000000p+0f, 0x1.6247ec0000000p+0f,
    0x1.6a09e60000000p+0f, 0x1.71f75e0000000p+0f, 0x1.7a11480000000p+0f, 0x1.82589a0000000p+0f,
    0x1.8ace540000000p+0f, 0x1.93737c0000000p+0f, 0x1.9c49180000000p+0f, 0x1.a5503c0000000p+0f,
    0x1.ae89fa0000000p+0f, 0x1.b7f7700000000p+0f, 0x1.c199be0000000p+0f, 0x1.cb720e0000000p+0f,
    0x1.d5818e0000000p+0f, 0x1.dfc9740000000p+0f, 0x1.ea4afa0000000p+0f, 0x1.f507660000000p+0f};
__constant__ float kPowRest[32] = {
    0x0.0p+0f, -0x1.9474140000000p-25f, 0x1.8d96d40000000p-25f, -0x1.dda2fc0000000p-25f,
    -0x1.9c0c220000000p-27f, -0x1.a2fbb20000000p-25f, 0x1.9649040000000p-25f, -0x1.2b0dbc0000000p-25f,
    0x1.1250020000000p-25f, -0x1.cde8ce0000000p-26f, 0x1.370be40000000p-25f, 0x1.336de20000000p-30f,
    -0x1.0a35500000000p-25f, -0x1.c541b40000000p-26f, -0x1.00d8ac0000000p-27f, -0x1.6cb2840000000p-25f,
    0x1.26055c0000000p-26f, 0x1.8b2bb80000000p-26f, -0x1.05cb440000000p-25f, -0x1.1c21420000000p-26f,
    0x1.67a1ca0000000p-28f, -0x1.348e560000000p-25f, 0x1.a3b5e40000000p-28f, -0x1.0b7ec80000000p-25f,
    -0x1.f9c3040000000p-27f, -0x1.e4c8860000000p-26f, -0x1.6961b40000000p-28f, -0x1.b5151e0000000p-28f,
    -0x1.a5217c0000000p-28f, -0x1.ab71320000000p-26f, 0x1.61428e0000000p-28f, -0x1.2ad5f80000000p-27f};

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

// What the lead tells the others to do with a row.
struct __align__(16) Command {
    int op;
    int node;          // row of the sequence
    int minus;         // kSum, and kFind after it: 1: leave out the tokens of the node's children; -1: for a decision
    int draft;         // kLeft, and kFind after it: the rejected draft (else -1)
    int cta;           // kFind: the CTA that finds the token,
    float top;         // the row's maximum
    float w_hi, w_lo;  // kLeft: the row's sum, in units of the largest weight
    uint64_t target;   // kFind: the sum to pass, counted from that CTA's part
    int64_t out;       // and the place of the token
};
static_assert(sizeof(Command) == 48, "sent 16 bytes at a time");

struct __align__(16) Partial {       // of one CTA: kStats: maximum, sum, its place, a NaN or +inf
    float top, sum;
    int arg, bad;
    DG_DEVINL uint64_t fixed() const { return (uint32_t)arg | (uint64_t)(uint32_t)bad << 32; }   // kSum, kLeft: the sum
    DG_DEVINL void set_fixed(uint64_t v) {
        arg = (int)(uint32_t)v;
        bad = (int)(uint32_t)(v >> 32);
    }
};

struct __align__(16) VShared {
    Command cmd;
    Partial part[kMaxCluster];        // in the lead: everyone's
    uint64_t told, parts;             // barriers: a command is here; (the lead's) every part is
    uint64_t warp_sum[kVWarps];       // fixed-point sums of the warps' parts
    uint64_t segment[kSegments];
    float w_top[kVWarps], w_sum[kVWarps];
    int w_arg[kVWarps], w_bad[kVWarps];
    float pow[32], rest[32];
    float c_hi, c_lo, d_min;          // log2(e) / temperature, and the difference whose weight is 2^-120
    int64_t V;
    int frac;
    int n_gone;                       // rejected tokens of the last node that lie in this CTA's part
    int child, last;                  // what the lead's first warp decided
    uint4 ring[kVWarps][kDeep][32];   // vectors on their way
    int gone[kMaxNodes];
    int path[kMaxNodes];              // the lead's, as the rest:
    int rejected[kMaxNodes];
    int token[kMaxNodes], parent[kMaxNodes];
    float uniform[kMaxNodes];
};

// A lane's vectors of a row, `hop` apart, on their way through its own places in shared memory: in registers they would be
// waited for when they are moved along, or the loop unrolled past the instruction cache.
struct Stream {
    const uint4 *src, *place;
    int64_t ask, hop, to;
    int at;

    DG_DEVINL Stream(VShared& sh, const uint4* row, int64_t v, int64_t hop_, int64_t to_)
        : src(row), place(&sh.ring[threadIdx.x >> 5][0][threadIdx.x & 31]), ask(v), hop(hop_), to(to_), at(0) {
        for (int k = 0; k < kDeep - 1; ++k) request(k);
    }
    DG_DEVINL void request(int slot) {
        if (ask < to)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dg::smem_u32(place + slot * 32)), "l"(src + ask) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
        ask += hop;
    }
    DG_DEVINL uint4 next() {   // the next vector (anything behind the last)
        request(at ? at - 1 : kDeep - 1);   // the place that was read last
        asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
        const uint4 r = place[at * 32];
        at = at == kDeep - 1 ? 0 : at + 1;
        return r;
    }
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
template <typename T>
DG_DEVINL float logit(const T* row, int64_t t) {
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[t] << 16);
    else
        return reinterpret_cast<const float*>(row)[t];
}

DG_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats at a time (one rounding each, as the scalar forms).
DG_DEVINL uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
DG_DEVINL void f2_split(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
DG_DEVINL uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
DG_DEVINL uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
DG_DEVINL uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
DG_DEVINL uint64_t f2_sub(uint64_t a, uint64_t b) { return f2_fma(b, f2(-1.f, -1.f), a); }

// 2^((x - top) c) of two logits as w (1 + e), w a table's 2^(j / 32) times a power of two, |e| < 2^-6.  The exponent in two
// floats: the difference (with what its rounding left out where logits are fp32; of bf16 logits it is exact unless one
// is 2^16 times the other), its product with c, cut into j, the power and g, |g| <= 1 / 64; e from the terms up to g^4 (the
// next is below 2^-39) and what the table's rounding left out.  Differences below d_min, -inf and NaN among them, weigh
// 2^-120: nothing at any place after the point.
template <typename T>
DG_DEVINL void weights2(const VShared& sh, float x0, float x1, float top, uint64_t& w, uint64_t& e) {
    const uint64_t x = f2(x0, x1), nt = f2(-top, -top);
    const uint64_t c = f2(sh.c_hi, sh.c_hi), nc = f2(-sh.c_hi, -sh.c_hi), cl = f2(sh.c_lo, sh.c_lo);
    const uint64_t magic = f2(12582912.f, 12582912.f);       // 1.5 2^23: rounds to a whole number
    uint64_t d = f2_add(x, nt);
    float d0, d1;
    f2_split(d, d0, d1);
    uint64_t left = 0;
    if constexpr (sizeof(T) == 4) {
        const uint64_t z = f2_sub(d, x);
        left = f2_add(f2_sub(x, f2_sub(d, z)), f2_sub(nt, z));
        float l0, l1;
        f2_split(left, l0, l1);
        left = f2(d0 > sh.d_min ? l0 : 0.f, d1 > sh.d_min ? l1 : 0.f);
    }
    d = f2(fmaxf(d0, sh.d_min), fmaxf(d1, sh.d_min));
    const uint64_t p = f2_mul(d, c), over = f2_fma(d, nc, p);   // over: what p's rounding has too much
    const uint64_t t = f2_fma(p, f2(32.f, 32.f), magic);
    uint64_t g = f2_fma(f2_sub(t, magic), f2(-0.03125f, -0.03125f), p);
    g = f2_fma(d, cl, f2_sub(g, over));
    if constexpr (sizeof(T) == 4) g = f2_fma(left, c, g);
    e = f2_fma(g, f2(9.6181291e-3f, 9.6181291e-3f), f2(5.5504109e-2f, 5.5504109e-2f));
    e = f2_fma(g, e, f2(0.24022651f, 0.24022651f));
    e = f2_fma(g, e, f2(0.69314718f, 0.69314718f));
    float t0, t1;
    f2_split(t, t0, t1);
    const int k0 = __float_as_int(t0), k1 = __float_as_int(t1);   // (whole number in the low bits, the rest of the magic above)
    e = f2_fma(g, e, f2(sh.rest[k0 & 31], sh.rest[k1 & 31]));
    w = f2(__int_as_float(__float_as_int(sh.pow[k0 & 31]) + (k0 & ~31) * (1 << 18)),
           __int_as_float(__float_as_int(sh.pow[k1 & 31]) + (k1 & ~31) * (1 << 18)));
}

DG_DEVINL float unit(float q) { return fminf(fmaxf(q, 0.f), 1.f); }   // (a NaN is 0)

// The sum of a vector's weights in fixed point; with Left of what q times the row's sum leaves of them.  Elements whose
// bit of `out` is set are left out.  What a weight has in multiples of 2^-20 adds up exactly; the rest, below 2^-6 of the
// weight, in fp32.
template <typename T, bool Left>
DG_DEVINL uint64_t vector_sum(const VShared& sh, const uint4& r, int64_t v, const float* q_row, uint32_t out) {
    constexpr int N = Vec<T>::kN;
    const int64_t V = sh.V;
    float x[N];
    unpack<T>(r, v, V, x);
    float q[N];
    if constexpr (Left) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {   // (four that begin before V end within the row)
            const float4 f = v * N + 4 * h < V ? __ldg(reinterpret_cast<const float4*>(q_row + v * N) + h) : make_float4(1.f, 1.f, 1.f, 1.f);
            q[4 * h] = unit(f.x);
            q[4 * h + 1] = unit(f.y);
            q[4 * h + 2] = unit(f.z);
            q[4 * h + 3] = unit(f.w);
        }
    }
    const uint64_t grid = f2(12.f, 12.f), minus_grid = f2(-12.f, -12.f);   // 1.5 2^3: rounds to multiples of 2^-20
    uint64_t coarse = 0, fine = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        uint64_t w, e;
        weights2<T>(sh, x[i], x[i + 1], sh.cmd.top, w, e);
        if constexpr (Left) {                   // w (1 + e) - q (w_hi + w_lo), or 0
            const uint64_t hi = f2_fma(w, e, w), lo = f2_fma(w, e, f2_sub(w, hi));
            const uint64_t qq = f2(q[i], q[i + 1]), wh = f2(sh.cmd.w_hi, sh.cmd.w_hi);
            const uint64_t p = f2_mul(qq, wh);
            const uint64_t pl = f2_fma(qq, f2(sh.cmd.w_lo, sh.cmd.w_lo), f2_fma(qq, wh, f2_mul(p, f2(-1.f, -1.f))));
            const uint64_t d = f2_sub(hi, p), z = f2_sub(d, hi);
            const uint64_t err = f2_sub(f2_sub(hi, f2_sub(d, z)), f2_add(p, z));
            const uint64_t l = f2_add(err, f2_sub(lo, pl));
            const uint64_t h = f2_add(d, l);
            const uint64_t rest = f2_add(f2_sub(d, h), l);
            float h0, h1, l0, l1;
            f2_split(h, h0, h1);
            f2_split(rest, l0, l1);
            w = f2(h0 > 0.f ? h0 : 0.f, h1 > 0.f ? h1 : 0.f);
            e = f2(h0 > 0.f ? l0 : 0.f, h1 > 0.f ? l1 : 0.f);   // here the rest itself
        }
        if (out >> i & 3u) {
            float h0, h1;
            f2_split(w, h0, h1);
            w = f2(out >> i & 1u ? 0.f : h0, out >> i & 2u ? 0.f : h1);
            if constexpr (Left) {
                f2_split(e, h0, h1);
                e = f2(out >> i & 1u ? 0.f : h0, out >> i & 2u ? 0.f : h1);
            }
        }
        const uint64_t m = f2_add(f2_add(w, grid), minus_grid);
        coarse = f2_add(coarse, m);
        fine = f2_add(fine, f2_sub(w, m));
        fine = Left ? f2_add(fine, e) : f2_fma(w, e, fine);
    }
    float c0, c1, g0, g1;
    f2_split(coarse, c0, c1);
    f2_split(fine, g0, g1);
    // (a vector's fine part stays below 2^-3: within 2^47 - 32-bit parts of it, in two steps)
    const int64_t whole = __float2int_rn((c0 + c1) * 1048576.f);
    const float f = g0 + g1, high = rintf(f * 1048576.f);
    const int64_t first = whole + (int64_t)(int)high;
    const float low = fmaf(high, -0x1p-20f, f);
    return (uint64_t)((first << (sh.frac - 20)) + __float2int_rn(low * __int_as_float((sh.frac + 127) << 23)));
}

DG_DEVINL uint64_t warp_add(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The part of a row that a warp of the cluster owns, in vectors, a multiple of 32 except at the row's end.
template <typename T>
DG_DEVINL int64_t part_size(int64_t V, int n_cta) {
    const int64_t nv = (V + Vec<T>::kN - 1) / Vec<T>::kN;
    return (nv + (int64_t)n_cta * kVThreads - 1) / ((int64_t)n_cta * kVThreads) * 32;
}
struct Part {
    int64_t from, to;
};
template <typename T>
DG_DEVINL Part part_of(int64_t V, int cta, int n_cta, int warp) {
    const int64_t nv = (V + Vec<T>::kN - 1) / Vec<T>::kN, each = part_size<T>(V, n_cta);
    const int64_t from = ((int64_t)cta * kVWarps + warp) * each;
    return Part{min(from, nv), min(from + each, nv)};
}

// Joins the statistics of the first n (a power of two) lanes, for all of them.
template <bool Sum, int n>
DG_DEVINL Partial join_stats(Partial q, float c) {
    float top = q.top;
#pragma unroll
    for (int o = n / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (Sum) {
        q.sum *= ex2((q.top - (top == -INFINITY ? 0.f : top)) * c);   // (-inf: 0; a NaN or +inf: a NaN)
#pragma unroll
        for (int o = n / 2; o; o >>= 1) q.sum += __shfl_xor_sync(0xffffffffu, q.sum, o);
    } else {
        if (q.top != top) q.arg = 0x7fffffff;
#pragma unroll
        for (int o = n / 2; o; o >>= 1) {
            q.arg = min(q.arg, __shfl_xor_sync(0xffffffffu, q.arg, o));
            q.bad |= __shfl_xor_sync(0xffffffffu, q.bad, o);
        }
    }
    q.top = top;
    return q;
}

// A row's maximum, its smallest place (without Sum), and with Sum the sum of 2^((x - maximum) c), of this CTA's part.
template <typename T, bool Sum>
DG_DEVINL Partial row_stats(VShared& sh, const T* row, int64_t V, int cta, int n_cta) {
    constexpr int N = Vec<T>::kN;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Part p = part_of<T>(V, cta, n_cta, warp);
    const uint4* src = reinterpret_cast<const uint4*>(row);
    const float c = sh.c_hi;
    float top = -INFINITY, sum = 0.f;
    int arg = 0x7fffffff;
    bool bad = false;
    int64_t v = p.from + lane;
    Stream in(sh, src, v, 32, p.to);
#pragma unroll 1
    for (; v < p.to; v += 32) {
        const uint4 now = in.next();
        float x[N];
        unpack<T>(now, v, V, x);
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
    const Partial w = join_stats<Sum, 32>(Partial{top, sum, arg, bad}, c);
    if (lane == 0) {
        sh.w_top[warp] = w.top;
        sh.w_sum[warp] = w.sum;
        sh.w_arg[warp] = w.arg;
        sh.w_bad[warp] = w.bad;
    }
    __syncthreads();
    Partial q{-INFINITY, 0.f, 0x7fffffff, 0};
    if (warp == 0) {
        if (lane < kVWarps) q = Partial{sh.w_top[lane], sh.w_sum[lane], sh.w_arg[lane], sh.w_bad[lane]};
        q = join_stats<Sum, kVWarps>(q, c);
    }
    return q;
}

// The elements of vector v that are left out.
template <typename T>
DG_DEVINL uint32_t left_out(const VShared& sh, int64_t v) {
    uint32_t out = 0;
    for (int i = 0; i < min(sh.n_gone, kMaxNodes); ++i)
        if (sh.gone[i] / Vec<T>::kN == v) out |= 1u << (sh.gone[i] % Vec<T>::kN);
    return out;
}

// A warp's sum of every `hop`-th 32 vectors of from .. to - 1; with `tiles`, each 32 vectors' sum there instead.  A function of
// its own: in line, twice, its constants and the walk's state do not fit the registers together.
template <typename T, bool Left>
__device__ __noinline__ uint64_t range_sum(VShared& sh, const uint4* src, const float* q_row, int64_t from, int64_t hop,
                                           int64_t to, uint64_t* tiles) {
    const int lane = threadIdx.x & 31;
    uint64_t sum = 0;
    int64_t v = from + lane;
    Stream in(sh, src, v, hop, to);
    const bool gone = sh.n_gone > 0;
#pragma unroll 1
    for (; v - lane < to; v += hop) {
        const uint4 now = in.next();
        const uint64_t s = v < to ? vector_sum<T, Left>(sh, now, v, q_row, gone ? left_out<T>(sh, v) : 0u) : 0ull;
        if (tiles) {
            const uint64_t all = warp_add(s);
            if (lane == 0) tiles[(v - lane - from) / 32] = all;
        } else {
            sum += s;
        }
    }
    return tiles ? 0 : warp_add(sum);
}

// Sums of the weights by warp (Left: of what a draft's distribution leaves of them), and the CTA's.
template <typename T, bool Left>
DG_DEVINL Partial row_sums(VShared& sh, const T* row, const VerifyArgs& a, const Command& c, const float* q_row, int cta,
                           int n_cta, int q0, int ql) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) sh.n_gone = 0;
    __syncthreads();
    if (c.minus > 0) {   // the rejected children's tokens in this CTA's part
        const int64_t part = part_size<T>(a.V, n_cta) * kVWarps;
        for (int i = c.node + 1 + tid; i < ql; i += kVThreads) {
            const int32_t t = a.tokens[q0 + i];
            if ((a.parents ? a.parents[q0 + i] : i - 1) != c.node || t < 0 || t >= a.V || t / Vec<T>::kN / part != cta) continue;
            const int at = atomicAdd(&sh.n_gone, 1);   // (in any order, and the same one twice: a list that is searched)
            if (at < kMaxNodes) sh.gone[at] = t;
        }
        __syncthreads();
    }
    const Part p = part_of<T>(a.V, cta, n_cta, warp);
    const uint64_t sum = range_sum<T, Left>(sh, reinterpret_cast<const uint4*>(row), q_row, p.from, 32, p.to, nullptr);
    if (lane == 0) sh.warp_sum[warp] = sum;
    __syncthreads();
    Partial q{};
    if (tid == 0)
    {
        uint64_t f = 0;
        for (int w = 0; w < kVWarps; ++w) f += sh.warp_sum[w];
        q.set_fixed(f);
    }
    return q;
}

// The token whose cumulated weight passes the target, which lies in this CTA's part (warp_sum and gone are as row_sums left
// them for these weights).  The CTA's warps sum up to 64 segments of what is left, until that is 32 vectors.
template <typename T, bool Left>
__device__ __noinline__ void find_token(VShared& sh, const T* row, const float* q_row, int cta, int n_cta, int32_t* out_tokens) {
    constexpr int N = Vec<T>::kN;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint4* src = reinterpret_cast<const uint4*>(row);
    uint64_t target = sh.cmd.target;
    int owner = 0;
    while (owner < kVWarps - 1 && target >= sh.warp_sum[owner]) target -= sh.warp_sum[owner++];
    Part p = part_of<T>(sh.V, cta, n_cta, owner);
    while (p.to - p.from > 32) {
        const int64_t tiles = (p.to - p.from + 31) / 32, each = (tiles + kSegments - 1) / kSegments * 32;
        const int n = (int)((p.to - p.from + each - 1) / each);
        if (each == 32) {
            range_sum<T, Left>(sh, src, q_row, p.from + warp * 32, 32 * kVWarps, p.to, sh.segment + warp);
        } else {
#pragma unroll 1
            for (int i = warp; i < n; i += kVWarps) {
                const int64_t from = p.from + i * each;
                const uint64_t s = range_sum<T, Left>(sh, src, q_row, from, 32, min(from + each, p.to), nullptr);
                if (lane == 0) sh.segment[i] = s;
            }
        }
        __syncthreads();
        int i = 0;
        while (i < n - 1 && target >= sh.segment[i]) target -= sh.segment[i++];
        p = Part{p.from + i * each, min(p.from + (i + 1) * each, p.to)};
        __syncthreads();   // (the next round writes the segments)
    }
    if (warp != 0) return;
    const int64_t v = p.from + lane;
    const bool in = v < p.to;
    uint4 r = make_uint4(0, 0, 0, 0);
    uint32_t out = 0;
    uint64_t mine = 0;
    if (in) {
        r = __ldg(src + v);
        out = sh.n_gone ? left_out<T>(sh, v) : 0u;
        mine = vector_sum<T, Left>(sh, r, v, q_row, out);
    }
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, in && incl > target);
    const int at = past ? __ffs(past) - 1 : 0;   // the vector's lane; then a lane sums its elements up to the lane's own
    r.x = __shfl_sync(0xffffffffu, r.x, at);
    r.y = __shfl_sync(0xffffffffu, r.y, at);
    r.z = __shfl_sync(0xffffffffu, r.z, at);
    r.w = __shfl_sync(0xffffffffu, r.w, at);
    out = __shfl_sync(0xffffffffu, out, at);
    const uint64_t before = __shfl_sync(0xffffffffu, incl - mine, at);
    const bool passes = before + vector_sum<T, Left>(sh, r, p.from + at, q_row, out | (0xfffffffeu << (lane & (N - 1)))) > target;
    const uint32_t which = __ballot_sync(0xffffffffu, passes) & ((1u << N) - 1);
    if (lane == 0)
        out_tokens[sh.cmd.out] = (int32_t)min((p.from + at) * N + (which ? __ffs(which) - 1 : N - 1), sh.V - 1);
}

// What the lead's first warp knows of a child before the row's statistics are there.
struct Child {
    bool is;
    int32_t token;
    float x, u, q;
};
template <typename T>
DG_DEVINL Child child_of(const VShared& sh, const VerifyArgs& a, const T* row, int q0, int ql, int node, int c, float T_) {
    Child k{false, -1, -INFINITY, 0.f, 1.f};
    if (c >= ql || (a.parents ? sh.parent[c] != node : c != node + 1)) return k;
    k.is = true;
    k.token = sh.token[c];
    if (T_ > 0.f) {
        k.u = sh.uniform[c];
        if (k.token >= 0 && k.token < a.V) {
            k.x = logit<T>(row, k.token);
            if (a.probs) k.q = unit(a.probs[(int64_t)(q0 + c) * a.ldq + k.token]);
        }
    }
    return k;
}

// The lead's first warp: tries the children of `node` in order (`k`: the first 32 nodes' behind it).  The row's maximum and
// sum are given (fixed point when Exact).  Returns the accepted child, -1: none, -2: too near to say with an fp32 sum.
// `last`: the rejected draft.
template <typename T, bool Exact>
DG_DEVINL int decide(VShared& sh, const VerifyArgs& a, const T* row, int q0, int ql, int node, float T_, const Partial& st,
                     int n_cta, Child k, int& last) {
    using F = std::conditional_t<Exact, double, float>;
    const int lane = threadIdx.x & 31;
    last = -1;
    // The sum's bound: its exponents' roundings (2^-23 of each, weighted by weights that fall faster than exponents
    // grow), the exponentials (2^-22), the joins, this comparison, and 2^-24 an addition of a thread.  Every rejected sibling
    // taken off it rounds once more, 2^-24 of it at most.
    const F sum = Exact ? (F)ldexp((double)st.fixed(), -a.frac) : (F)st.sum;
    const F slack = Exact ? (F)0 : sum * ((F)0x1p-15f + (F)a.V / (F)(n_cta * kVThreads) * (F)0x1p-23f);
    F left = sum;
    int n_rejected = 0;
    const int end = a.parents ? ql : min(ql, node + 2);
    for (int base = node + 1; base < end; base += 32) {
        if (base > node + 1) k = child_of<T>(sh, a, row, q0, ql, node, base + lane, T_);
        F w = 0;
        if (T_ > 0.f && k.is && k.token >= 0 && k.token < a.V) {
            if constexpr (Exact) {
                uint64_t ww, ee;
                weights2<T>(sh, k.x, k.x, st.top, ww, ee);
                float h, l, unused;
                f2_split(ww, h, unused);
                f2_split(ee, l, unused);
                w = h > 0x1p-119f ? (F)h + (F)h * (F)l : (F)0;
            } else {
                w = ex2((k.x - st.top) * sh.c_hi);
            }
        }
        // Against 0 any probability wins, also one that is too small for its weight to be told from 0.
        const uint32_t possible = __ballot_sync(0xffffffffu, k.is && k.x > -INFINITY);
        uint32_t todo = __ballot_sync(0xffffffffu, k.is);
        while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const int32_t t = __shfl_sync(0xffffffffu, k.token, from);
            if (T_ == 0.f) {
                if (t == st.arg) return base + from;
                last = base + from;
                continue;
            }
            const F wt = __shfl_sync(0xffffffffu, w, from), ut = __shfl_sync(0xffffffffu, k.u, from);
            if (a.probs) {
                const F q = (F)__shfl_sync(0xffffffffu, k.q, from), m = ut * q, lhs = m * sum;
                if ((ut == 0 || q == 0) && (possible >> from & 1u)) return base + from;
                if (!Exact && fabsf((float)(lhs - wt)) <= (float)(m * slack) && (lhs > 0 || wt > 0)) return -2;
                if (lhs < wt) return base + from;
            } else {
                bool again = false;
                for (int i = lane; i < n_rejected; i += 32) again = again || sh.rejected[i] == t;
                again = __any_sync(0xffffffffu, again);
                if (!again) {
                    if (ut == 0 && (possible >> from & 1u)) return base + from;
                    const F lhs = ut * (left > 0 ? left : (F)0);
                    const F bound = slack + sum * ((F)n_rejected * (F)0x1p-24f);
                    if (!Exact && fabsf((float)(lhs - wt)) <= (float)(ut * bound) && (ut > 0 || wt > 0)) return -2;
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
__global__ void __launch_bounds__(kVThreads, 4) k_verify(const __grid_constant__ VerifyArgs a) {
    __shared__ VShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int n_cta = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    const int s = (int)(blockIdx.x / n_cta), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        dg::mbar_init(&sh.told, 1);
        dg::mbar_init(&sh.parts, 1);
        dg::fence_mbar_init();
    }
    if (tid < 32) {
        sh.pow[tid] = kPow[tid];
        sh.rest[tid] = kPowRest[tid];
    }
    __syncthreads();
    auto arrived = cluster.barrier_arrive();   // everyone runs, with its barriers, before anyone reaches into another CTA
    dg::pdl_wait();
    dg::pdl_release();
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1];
    const float T_ = a.temperature[s];
    const bool offsets = q0 >= 0 && q1 >= q0 && (int64_t)q1 <= a.total;
    const int ql = offsets ? q1 - q0 : 0;
    if (tid == 0) {
        const double c = T_ > 0.f ? 1.4426950408889634 / (double)T_ : 1.0;
        sh.c_hi = (float)c;
        sh.c_lo = (float)(c - (double)sh.c_hi);
        sh.d_min = -120.f / sh.c_hi;
        sh.n_gone = 0;
        sh.V = a.V;
        sh.frac = a.frac;
    }
    // The lead alone looks at what decides how often the cluster meets.
    int accepted = 0;
    bool walks = false;
    if (cta == 0) {
        bool good = offsets && ql <= kMaxNodes;
        if (good && ql > 0) {
            good = T_ == 0.f || (T_ >= 0x1p-64f && T_ <= 0x1p64f);
            if (T_ != 0.f) good = good && a.next_uniforms[s] >= 0.f && a.next_uniforms[s] < 1.f;
            for (int i = tid; i < ql; i += kVThreads) {
                const int32_t up = a.parents ? a.parents[q0 + i] : i - 1, t = a.tokens[q0 + i];
                const float u = T_ != 0.f ? a.uniforms[q0 + i] : 0.f;
                sh.parent[i] = up;
                sh.token[i] = t;
                sh.uniform[i] = u;
                if (i > 0) good = good && up >= 0 && up < i && u >= 0.f && u < 1.f;
            }
        }
        good = !__syncthreads_or(!good);
        walks = good && ql > 0;
        if (!walks) {
            for (int i = tid; i < ql; i += kVThreads) a.path[q0 + i] = a.out_tokens[q0 + i] = -1;
            if (tid == 0) {
                a.n_accept[s] = -1;
                if (!good) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            }
        }
    } else {
        __syncthreads();
    }

    // The first command is known to all: the root's statistics.  (A sequence that is refused gives its CTAs nothing to
    // read; the lead's command to leave is on its way.)
    Command c{kStats, 0, 0, -1, 0, 0.f, 0.f, 0.f, 0, 0};
    Partial stats{};            // of the row at `node` (the lead's)
    int rejected = -1;          // the draft rejected there
    uint32_t meeting = 0;
    bool met = true;            // false: a wait of this CTA ran out, for all its threads alike
    for (;; ++meeting) {
        const T* row = reinterpret_cast<const T*>(a.logits) + (int64_t)(q0 + c.node) * a.ld;
        const float* q_row = c.draft >= 0 ? a.probs + (int64_t)(q0 + c.draft) * a.ldq : nullptr;
        Child k{false, -1, 0.f, 0.f, 0.f};
        if (cta == 0 && warp == 0 && walks) k = child_of<T>(sh, a, row, q0, ql, c.node, c.node + 1 + lane, T_);
        Partial mine{-INFINITY, 0.f, 0x7fffffff, 0};
        if (tid == 0) dg::mbar_arrive_expect_tx(cta == 0 ? &sh.parts : &sh.told, cta == 0 ? 16u * n_cta : (uint32_t)sizeof(Command));
        if (c.op == kStats) {
            if (ql > 0) mine = T_ > 0.f ? row_stats<T, true>(sh, row, a.V, cta, n_cta) : row_stats<T, false>(sh, row, a.V, cta, n_cta);
        } else {
            mine = c.op == kLeft ? row_sums<T, true>(sh, row, a, c, q_row, cta, n_cta, q0, ql)
                                 : row_sums<T, false>(sh, row, a, c, nullptr, cta, n_cta, q0, ql);
        }
        if (meeting == 0) cluster.barrier_wait(std::move(arrived));
        if (tid == 0) {   // this CTA's part to the lead
            send16(dg::mapa_shared(&sh.part[cta], 0),
                   make_uint4(__float_as_uint(mine.top), __float_as_uint(mine.sum), (uint32_t)mine.arg, (uint32_t)mine.bad),
                   dg::mapa_shared(&sh.parts, 0));
        }
        if (cta != 0) {
            met = __syncthreads_and(dg::mbar_wait_cluster(&sh.told, meeting & 1u));
            if (!met) break;
            c = sh.cmd;
            if (c.op == kExit || c.op == kFind) break;
            continue;
        }

        // The lead decides what comes next.
        Command next{kExit, c.node, 0, -1, 0, stats.top, 0.f, 0.f, 0, 0};
        bool finish = !walks, no_token = false;
        met = __syncthreads_and(dg::mbar_wait_cluster(&sh.parts, meeting & 1u));
        if (!met) {
            finish = true;
            walks = false;
        }
        auto draw_from = [&](uint64_t sum) {   // the token past next_uniforms * sum
            const float u = a.next_uniforms[s];
            const uint64_t U = (uint64_t)__float2ull_rz(u * 0x1p32f) << 32 |
                               __float2ull_rz((u * 0x1p32f - truncf(u * 0x1p32f)) * 0x1p32f);
            uint64_t target = __umul64hi(sum, U);
            int owner = 0;
            while (owner < n_cta - 1 && target >= sh.part[owner].fixed()) target -= sh.part[owner++].fixed();
            next = c;
            next.op = kFind;
            next.cta = owner;
            next.target = target;
            next.out = q0 + accepted;
        };
        if (walks && c.op == kStats) {
            Partial t{-INFINITY, 0.f, 0x7fffffff, 0};
            if (lane < n_cta) t = sh.part[lane];
            t = T_ > 0.f ? join_stats<true, kMaxCluster>(t, sh.c_hi) : join_stats<false, kMaxCluster>(t, 0.f);
            t.top = __shfl_sync(0xffffffffu, t.top, 0);   // (all lanes': the first half has joined)
            t.sum = __shfl_sync(0xffffffffu, t.sum, 0);
            t.arg = __shfl_sync(0xffffffffu, t.arg, 0);
            t.bad = __shfl_sync(0xffffffffu, t.bad, 0);
            if (T_ > 0.f) t.bad = 0;
            stats = t;
            const bool nan = t.bad || !(t.top < INFINITY) || !(t.sum < INFINITY);
            if (nan || t.top == -INFINITY) {
                if (tid == 0) dg::raise_status(a.status, nan ? DG_DEV_NAN_INF_ROW : DG_DEV_EMPTY_ROW);
                finish = no_token = true;
            }
        } else if (walks) {
            uint64_t f = 0;
            for (int i = 0; i < n_cta; ++i) f += sh.part[i].fixed();
            stats.set_fixed(f);
        }
        if (!finish && (c.op == kStats || (c.op == kSum && c.minus < 0))) {   // (minus -1: a sum asked for by a decision)
            if (warp == 0) {
                int last;
                const int child = c.op == kSum ? decide<T, true>(sh, a, row, q0, ql, c.node, T_, stats, n_cta, k, last)
                                               : decide<T, false>(sh, a, row, q0, ql, c.node, T_, stats, n_cta, k, last);
                if (lane == 0) {
                    sh.child = child;
                    sh.last = last;
                }
            }
            __syncthreads();
            const int child = sh.child;
            next.op = kStats;
            next.top = stats.top;
            if (child == -2) {
                next.op = kSum;
                next.minus = -1;
            } else if (child >= 0) {
                if (tid == 0) sh.path[accepted] = child;
                ++accepted;
                next.node = child;
            } else {
                rejected = sh.last;
                if (T_ == 0.f) {
                    if (tid == 0) a.out_tokens[q0 + accepted] = stats.arg;
                    finish = true;
                } else {
                    next.op = kSum;
                    next.minus = rejected >= 0 && !a.probs ? 1 : 0;
                }
            }
        } else if (!finish && c.op == kSum) {
            if (a.probs && rejected >= 0) {
                const double w = ldexp((double)stats.fixed(), -a.frac);
                next.op = kLeft;
                next.draft = rejected;
                next.w_hi = (float)w;
                next.w_lo = (float)(w - (double)next.w_hi);
            } else if (c.minus > 0 && stats.fixed() == 0) {
                next.op = kSum;          // nothing is left: all of the row again
            } else {
                draw_from(stats.fixed());
            }
        } else if (!finish) {            // kLeft
            if (stats.fixed() == 0) {      // nothing is left: the row itself, whose sums are made again
                rejected = -1;
                next.op = kSum;
            } else {
                draw_from(stats.fixed());
            }
        }
        if (finish) next.op = kExit;
        __syncthreads();   // the parts are read: the next ones may come
        if (tid > 0 && tid < n_cta) {
            const uint4* words = reinterpret_cast<const uint4*>(&next);
            const uint32_t to = dg::mapa_shared(&sh.cmd, (uint32_t)tid), bar = dg::mapa_shared(&sh.told, (uint32_t)tid);
#pragma unroll
            for (int i = 0; i < (int)(sizeof(Command) / 16); ++i) send16(to + 16 * i, words[i], bar);
        }
        if (walks && (next.op == kExit || next.op == kFind)) {   // the walk's outputs
            for (int i = tid; i < ql; i += kVThreads) {
                a.path[q0 + i] = i == 0 ? 0 : i <= accepted ? sh.path[i - 1] : -1;
                if (i < accepted)
                    a.out_tokens[q0 + i] = sh.token[sh.path[i]];
                else if (i > accepted || no_token)
                    a.out_tokens[q0 + i] = -1;
            }
            if (tid == 0) a.n_accept[s] = accepted;
        }
        if (next.op == kExit) break;
        if (next.op == kFind) {
            c = next;
            if (tid == 0) sh.cmd = next;
            __syncthreads();
            break;
        }
        c = next;
        if (tid == 0) sh.cmd = next;
    }
    // This CTA sends nothing more.  None leaves before all have come so far, so that nobody sends into the memory of a CTA
    // that is gone: also after a wait that ran out (all are bounded, so all come here), whose CTA then waits, as
    // long again at most, for what may be on its way to it.
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // (no data to be seen behind it)
    if (met && c.op == kFind && c.cta == cta) {
        const T* row = reinterpret_cast<const T*>(a.logits) + (int64_t)(q0 + c.node) * a.ld;
        if (c.draft >= 0)
            find_token<T, true>(sh, row, a.probs + (int64_t)(q0 + c.draft) * a.ldq, cta, n_cta, a.out_tokens);
        else
            find_token<T, false>(sh, row, nullptr, cta, n_cta, a.out_tokens);
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (!met) {
        if (tid == 0) dg::raise_status(a.status, DG_DEV_TIMEOUT);
        (void)dg::mbar_wait_cluster(cta == 0 ? &sh.parts : &sh.told, meeting & 1u);
    }
}

// ------------------------------------------------------------------ kept paths
// A thread owns 16 bytes of a head in one layer's keys or values and takes the path's nodes in order.  Node path[i] goes to
// slot i <= path[i] behind the context, and every later node lies at path[k] >= k > i: nothing is overwritten
// before it is read.  250 paths in 8 layers, 33 MB to and fro, take 7.9 us, one path in 12 layers 3.1: a launch, and four reads
// that wait for one another (offsets, path, pages, data).
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
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    // CTAs of a sequence: as many as have a vector a thread of the row, two at least, and run at once: four an SM, three in
    // clusters of sixteen, which do not fill the GPU.  Where a CTA's part of a row is long, several waves of larger clusters are as
    // good.
    // Measured (us with 16 / 8 / 4 / 2 / 1 CTAs), chains of 5 with draft rows: over 2k tokens 8 18.1 / 17.3 / 17.4 / 17.6 / 19.7, 600
    // - / 113 / 63 / 40 / 28; 4k 300 - / 61 / 36 / 24 / 26; 32k 1 13.9 / 15.0 / 18.0 / 23.1, 28 23.0 / 24.9, 37 30 / 24.6 / 30.1, 96 - /
    // 40 / 37 / 48, 200 - / 66 / 57 / 62 / 84; 262k 24 60 / 84, 48 94 / 102, 64 109 / 110 / 157, 200 - / 245 / 273 / 377, 600 - / 651 / 644 /
    // 710 / 820.  Over 443 shapes (1 to 600 chains, trees of 32 and single rows of 1k to 262k tokens, bf16 and fp32) the rule
    // loses 0.7 % to the best on average, at most 26 %.
    const int64_t row_bytes = V * es;
    int cluster = kMaxCluster;
    while (cluster > 2 && cluster * (int64_t)kVThreads * 16 > row_bytes) cluster /= 2;
    while (cluster > 1 &&
           n_seq * (int64_t)cluster > (cluster > 8 ? 3 : 4) * (int64_t)sms * std::max<int64_t>(1, row_bytes / cluster / 16384))
        cluster /= 2;
    // clusters past 8 are asked for once a device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DG_ERR_CUDA;
    if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        if (cudaFuncSetAttribute(k_verify<uint16_t>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(k_verify<float>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return DG_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
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
    // what other blocks, of this sequence and of others, still read
    const std::pair<const int32_t*, int64_t> read[] = {{cache->kv_len, n_seq}, {n_accept, n_seq}, {cu_q, (int64_t)n_seq + 1},
                                                       {path, total_q}, {cache->page_table, (int64_t)n_seq * cache->max_pages}};
    for (const auto& [p, words] : read) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(new_len), at = reinterpret_cast<uintptr_t>(p);
        if (from < at + 4 * (uintptr_t)words && at < from + 4 * (uintptr_t)n_seq) return DG_ERR_INVALID_ARG;
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
