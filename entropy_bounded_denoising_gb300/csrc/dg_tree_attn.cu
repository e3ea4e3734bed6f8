// dg_tree_attn.cu -- attention of drafted trees, and through a sliding window with first tokens that stay
// visible, over the paged key / value cache, on the tensor cores (tcgen05 + TMEM + TMA, sm_103a).
//
// An item is (sequence, key head, up to 128 rows), a row one (query, query head of that key head): the rows that share
// keys share a tile, so keys and values are read once for 128 / (Hq / Hkv) queries.  It visits tiles of 64 keys: those of
// the first tokens that stay visible, then those from the window's (or the context's) first to its last key.  All
// tiles of all items, in order, form one line that is cut into equal runs, one for each of the resident CTAs; a
// run's first and last items may be pieces, which go to the workspace as (maximum, sums, unnormalised output)
// and are joined by a second kernel in the order of the line.
//
// The weights are rounded to bf16 for the product with V, so the product is divided by the sum of the rounded ones: a row
// is then an exact mean of the values it sees, with weights off by half a bf16 step.  Divided by the unrounded sum the
// mean itself is off by as much again (values that are all alike came out a step away).  lse takes the unrounded sum.
//
// A CTA (two an SM; one for heads of 256):
//   warp 0      walks the run, publishes its pieces in a ring and copies their queries, and their keys and
//               values through one ring of five tiles (ten for heads of 64), page by page, a box a lane;
//   warp 1      issues the products: S = Q K^T (128 x 64) into TMEM, O += P V with P from TMEM;
//   warps 2..5  the softmax, a row a thread.
// A tile that not all rows see whole gets each row's 64-bit mask: the window's and the context's ranges, and the row's
// words of the tree mask, shifted to the tile.  Keys of it that no row sees have their values zeroed in shared
// memory before the product (what they hold is nobody's, and 0 * NaN is not 0).
//
// Measured: 32 trees of 64 nodes over up to 4k keys, 16 / 8 heads of 128: 82 us, where their bytes take 53 and the same
// call with all keys in L2 takes 62: start and join take 12, the rest is the copies' (4.9 TB/s; a ring of four tiles
// for five 2 us more, copies asked into L2 three to eight tiles ahead 7 to 26).  Two prompts of 4000 through windows of 1500, 8 / 4
// heads of 64: 51 us, 406 TFLOP/s, bound by a tile's chain of steps, in the softmax 1300 to 1400 cycles.  9 trees of 199 nodes
// through windows of 2500, 20 / 4 heads of 256: 97.6 us, 641 TFLOP/s; a tile takes some 2600 cycles, of which the softmax works
// 1450 and waits 1000 for S.  The copies are not why (93.8 with all pages one sequence's); S, whose 16 products take 720 cycles,
// follows on the tensor pipe the last P V, of nearly 600, and the hand-overs between warps come on top.
// Waits by one lane and a shuffle, for all lanes' own, made the chain 10 % longer.  At heads of 256 the queries in tensor
// memory took 1 us off, and two softmax warps a quarter of the rows, each for half of a tile's keys, added 3.
#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <atomic>
#include <limits>
#include <utility>

#include "dg_tree.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 128;      // rows of an item
constexpr int kKeys = 64;       // keys of a tile
constexpr int kSub = 64;        // columns of a 128-byte swizzle atom
constexpr uint32_t kQSub = kTile * kSub * 2;
constexpr uint32_t kAtom = 8 * kSub * 2;   // of keys and values: 8 slots x 64 columns
constexpr float kRescaleAbove = 8.f;   // log2 units a row's maximum may grow before it moves: P <= 2^8
constexpr int kThreads = 192;
constexpr int kRing = 4;        // pieces published ahead
constexpr int kReaders = 5;     // of a piece: the products, four softmax warps

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct TreeArgs {
    uint16_t* o;
    float* lse;
    const int32_t* cu_q;
    const uint32_t* mask;       // null: causal
    const int32_t* positions;
    int64_t total_q;
    int32_t n_seq, max_q_len, Hq, Hkv, group, mask_words, window, sinks;
    int32_t hpt, qpt, head_tiles;   // heads and queries of an item; items a query's heads take
    int32_t rows;               // of a piece in the workspace (multiple of 32)
    int32_t negate;             // the products' sign: scale_log2 is the scale's magnitude, so the largest score stays the largest
    float scale_log2;
    int32_t box_shift;          // slots of a copy of keys or values: 8 .. 64
    int32_t by_slot, mul2, mul3, mul8;   // its coordinates: (0, by_slot * slot, mul2 * head, mul3 * head + mul8 * (slot / 8), page)
    dg::PagedKV kv;
    float4* part_o;             // [grid][2][D / 4][rows]
    float4* part_ml;            // [grid][2][rows]: maximum, sum of the weights, of the rounded weights
    int4* desc;                 // [grid][2]: CTAs that follow (0: nothing to join), first query's row, first head, queries; heads
    unsigned* status;
};

template <int D>
struct TreeCfg {
    static constexpr uint32_t kQBytes = (D / kSub) * kQSub, kKVBytes = kKeys * D * 2;
    static constexpr uint32_t kBufs = D == 64 ? 10 : 5;     // tiles of keys or values on their way or in use
    // The rounded weights' sum: for heads of 64 by the product, whose values have 16 more columns, all ones; for heads of 128
    // tensor memory has no room for them, for heads of 256 an instruction, and the softmax adds (for heads of 64 4 us
    // more of 50).
    static constexpr bool kSumsByProduct = D == 64;
    static constexpr int kValueCols = D + (kSumsByProduct ? 16 : 0);
    static constexpr uint32_t kOffQ = 0, kOffKV = kQBytes, kOffOnes = kOffKV + kBufs * kKVBytes,
                              kOffBar = kOffOnes + (kSumsByProduct ? 2 * kAtom : 0);
    static constexpr uint32_t kColS = 0, kColO = 64, kColL = kColO + D, kColP = kColO + kValueCols;
    static constexpr uint32_t kTmemCols = D == 256 ? 512 : 256;
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    static constexpr int kMaxCtas = D == 256 ? 256 : 512;   // grid bound the workspace is sized for
};

DG_DEVINL uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}
DG_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Packed fp32 pairs (one rounding per element, as the scalar forms).
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
// a and b plus the two halves of a pair, in fp32.
DG_DEVINL void add_bf16x2(uint32_t pair, float& a, float& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(pair));
}

// A run's part of one item.
struct Piece {
    int32_t s, hk, h0, nh;       // sequence, key head, first query head and heads
    int32_t qrow, qi0, nq;       // first query: row of q and index in the sequence; queries
    int32_t ql, kl;
    int32_t sink_end, ns;        // keys below sink_end stay visible; tiles of them before the body's
    int32_t jlo, jhi;            // the body's keys that some row may see
    int32_t t0, nt;              // tiles of the piece, of the item's
    int32_t last;                // the CTA that has the item's last tile
    uint32_t flags;              // kStarts, kEnds
    // the tile that comes i-th
    DG_DEVINL int tile(int i) const { return t0 + i < ns ? t0 + i : jlo / kKeys + t0 + i - ns; }
};
constexpr uint32_t kStarts = 1, kEnds = 2;

// Keys and values share one ring of buffers, in the order K0, K1, V0, K2, V1, ..., that of the products.
DG_DEVINL uint32_t keys_at(uint32_t n) { return n == 0 ? 0u : 2u * n - 1u; }
DG_DEVINL uint32_t values_at(uint32_t n) { return 2u * n + 2u; }
template <uint32_t N>
struct RingAt {   // a place in the ring and the parity of its use
    uint32_t slot, parity;
    DG_DEVINL explicit RingAt(uint32_t n) : slot(n % N), parity(n / N & 1u) {}
};

struct __align__(8) TreeShared {
    uint64_t qfull, qempty, oempty;
    uint64_t full[10], empty[10];
    uint64_t sfull, sempty;
    uint64_t pfull[2], pvdone[2];
    uint64_t mmadone;
    uint64_t wfull[kRing], wempty[kRing];
    uint64_t met;                 // the four softmax warps' own barrier (bounded, unlike bar.sync)
    uint64_t seen[2][4];          // of a masked tile, by warp: the keys some row sees
    int64_t sums[kThreads / 32];
    int64_t found_start;
    Piece piece[kRing];           // nt 0: no more
    int32_t top_position[2][8];   // by warp: the last and the first position of its rows
    int32_t found_seq, zeros;     // zeros: some sequence has queries and no keys
    uint32_t tmem_base;
    int abort_flag;
};
// (Two CTAs an SM of 115712 bytes each, two CTAs' own kilobytes beside them, are all of its shared memory.)
template <int D>
constexpr size_t tree_smem() {
    static_assert((TreeCfg<D>::kOffBar + sizeof(TreeShared)) <= (TreeCfg<D>::kCtasPerSm == 2 ? 115712 : 232448), "shared memory");
    return TreeCfg<D>::kOffBar + sizeof(TreeShared);
}

DG_DEVINL bool try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(dg::smem_u32(bar)), "r"(parity), "r"(200u)
        : "memory");
    return ok != 0;
}
DG_DEVINL bool wait(uint64_t* bar, uint32_t parity) {   // bounded, as every wait of the library
    for (uint32_t i = 0; i < 4u * dg::kWaitPolls; ++i)
        if (try_wait(bar, parity)) return true;
    return false;
}
DG_DEVINL bool wait_warp(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < 4u * dg::kWaitPolls; ++i)
        if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    return false;
}
DG_DEVINL bool aborted(const TreeShared& sh) { return *(volatile const int*)&sh.abort_flag != 0; }
DG_DEVINL void do_abort(TreeShared& sh, unsigned* status) {
    *(volatile int*)&sh.abort_flag = 1;
    dg::raise_status(status, DG_DEV_TIMEOUT);
}

// ------------------------------------------------------------------ the line
// A sequence on it: its items (query tiles x heads' tiles x key heads) and the line's length an item has, at least its
// tiles.  Of a tree every item visits the same tiles, and of a single query tile the length is exact; the query tiles of
// a longer causal sequence get the most that one of them may have.
struct SeqLine {
    dg::PagedSeq seq;
    int q_tiles;
    int64_t len;
    DG_DEVINL int64_t cost(const TreeArgs& a) const { return (int64_t)q_tiles * a.head_tiles * a.Hkv * len; }
};

struct Range {
    int sink_end, ns, jlo, jhi, nt;
};
// The tiles of query tile qt.
DG_DEVINL Range range_of(const TreeArgs& a, const dg::PagedSeq& q, int qt) {
    Range r;
    const int ctx = q.kl - q.ql;
    const int64_t first = a.mask ? ctx : (int64_t)ctx + (int64_t)qt * a.qpt;
    r.jhi = a.mask ? q.kl - 1 : ctx + (int)min((int64_t)q.ql, ((int64_t)qt + 1) * a.qpt) - 1;
    r.jlo = a.window < 0 ? 0 : (int)max((int64_t)0, first - a.window);
    r.sink_end = min(a.sinks, r.jlo);
    r.ns = min((r.sink_end + kKeys - 1) / kKeys, r.jlo / kKeys);
    r.nt = r.ns + r.jhi / kKeys - r.jlo / kKeys + 1;
    return r;
}

// What a sequence's line is worked out from, asked for ahead of its use.
struct RawSeq {
    int32_t q0, q1, kl;
};
DG_DEVINL RawSeq raw_seq(const TreeArgs& a, int s) {
    return s < a.n_seq ? RawSeq{a.cu_q[s], a.cu_q[s + 1], a.kv.kv_len[s]} : RawSeq{0, 0, 0};
}

DG_DEVINL SeqLine seq_line(const TreeArgs& a, const RawSeq& x) {
    SeqLine p;
    p.seq = dg::paged_seq_of(a.kv, a.total_q, x.q0, x.q1, x.kl, dg::kMaxKeys);
    if (p.seq.ql > a.max_q_len) p.seq.ok = false;
    p.q_tiles = p.seq.ok && p.seq.kl > 0 ? (p.seq.ql <= a.qpt ? (p.seq.ql > 0 ? 1 : 0) : (int)(((int64_t)p.seq.ql + a.qpt - 1) / a.qpt)) : 0;
    p.len = 0;
    if (p.q_tiles == 1 || (p.q_tiles > 0 && a.mask)) {
        p.len = range_of(a, p.seq, 0).nt;
    } else if (p.q_tiles > 0) {
        p.len = min((int64_t)((p.seq.kl - 1) / kKeys + 1),
                    ((int64_t)a.window + a.qpt + kKeys - 2) / kKeys + 1 + ((int64_t)a.sinks + kKeys - 1) / kKeys);
    }
    return p;
}

struct Run {
    int64_t per_cta, start, end, seq_start;
    int seq;
    bool zeros;      // some sequence has queries and no keys
};

DG_DEVINL int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
DG_DEVINL int64_t warp_scan(int64_t v) {   // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Tiles of a run, at least (us for 2 / 4 / 8 tiles, trees of 64 nodes, 8 key heads of 128: one over 300 keys 20.8 / 22.0 / 28.1,
// over 4096 26.7 / 23.2 / 24.5, two over 1000 21.7 / 23.9 / 26.9, eight over 300 18.4 / 20.1 / 27.6).
constexpr int kMinRun = 2;

DG_DEVINL void cut(Run& r, int64_t total) {
    r.per_cta = max((int64_t)kMinRun, total < (1LL << 31) ? (int64_t)(((uint32_t)total + gridDim.x - 1) / gridDim.x)
                                                          : (total + gridDim.x - 1) / gridDim.x);
    r.start = min(total, (int64_t)blockIdx.x * r.per_cta);
    r.end = min(total, r.start + r.per_cta);
    r.seq = 0;
    r.seq_start = 0;
}

// The whole CTA: two passes over the sequences' costs, the second up to the one that the run begins in.  (By one warp
// alone, while the others wait for its pieces, within 1 % for 1 to 100 sequences.)
DG_DEVINL Run find_run(const TreeArgs& a, TreeShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0, first = 0;
    bool zeros = false;
#pragma unroll 4
    for (int s = tid; s < a.n_seq; s += kThreads) {
        const SeqLine p = seq_line(a, raw_seq(a, s));
        if (blockIdx.x == 0 && !p.seq.ok) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        const int64_t c = p.cost(a);
        zeros = zeros || (p.seq.ok && p.seq.kl == 0 && p.seq.ql > 0);
        if (s == tid) first = c;
        mine += c;
    }
    mine = warp_sum(mine);
    if (lane == 0) sh.sums[warp] = mine;
    Run r;
    r.zeros = __syncthreads_or(zeros);
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) total += sh.sums[w];
    __syncthreads();
    cut(r, total);
    if (r.start >= r.end) return r;   // the same for the whole CTA
    int64_t base = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += kThreads) {
        const int s = s0 + tid;
        const int64_t c = s0 == 0 ? first : seq_line(a, raw_seq(a, s)).cost(a);
        int64_t incl = warp_scan(c);
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        int64_t before = base, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sh.sums[w];
            all += sh.sums[w];
        }
        incl += before;
        if (c > 0 && incl - c <= r.start && r.start < incl) {
            sh.found_seq = s;
            sh.found_start = incl - c;
        }
        base += all;
        __syncthreads();
        if (base > r.start) break;   // the same for the whole CTA
    }
    r.seq = sh.found_seq;
    r.seq_start = sh.found_start;
    return r;
}

// Walks a run piece by piece (a warp, uniformly).  From item to item by counting: a division or a read that is waited for
// costs the copies behind it a tile.
struct Walk {
    int64_t begin, at, end, per_cta;   // of the item on the line; where the run is in it
    int s, hk, qt, ht;
    SeqLine p;
    RawSeq next_raw;                   // of the sequence behind it

    DG_DEVINL void start(const TreeArgs& a, const Run& r) {
        end = r.end;
        at = r.start;
        per_cta = r.per_cta;
        s = r.seq;
        hk = qt = ht = 0;
        begin = r.seq_start;
        const RawSeq raw = raw_seq(a, s);
        next_raw = raw_seq(a, s + 1);
        p = seq_line(a, raw);
        if (at >= end) return;
        const int64_t off = at - begin, per_head = (int64_t)p.q_tiles * a.head_tiles;
        const int64_t item = off < (1LL << 31) ? (uint32_t)off / (uint32_t)p.len : off / p.len;
        begin += item * p.len;
        if (item < (1LL << 31) && per_head < (1LL << 31)) {
            hk = (int)((uint32_t)item / (uint32_t)per_head);
            const uint32_t x = (uint32_t)item - (uint32_t)hk * (uint32_t)per_head;
            qt = a.head_tiles == 1 ? (int)x : (int)(x / (uint32_t)a.head_tiles);
            ht = (int)(x - (uint32_t)qt * (uint32_t)a.head_tiles);
        } else {
            hk = (int)(item / per_head);
            const int64_t x = item - hk * per_head;
            qt = (int)(x / a.head_tiles);
            ht = (int)(x - (int64_t)qt * a.head_tiles);
        }
    }

    DG_DEVINL bool next(const TreeArgs& a, Piece& z) {
        while (at < end) {
            const int64_t to = min(end, begin + p.len);
            const int t0 = (int)(at - begin);
            const Range r = range_of(a, p.seq, qt);
            const bool skip = t0 >= r.nt;   // past the item's last tile: the line has room for the longest
            if (!skip) {
                z.s = s;
                z.hk = hk;
                z.h0 = hk * a.group + ht * a.hpt;
                z.nh = min(a.hpt, a.group - ht * a.hpt);
                z.qi0 = qt * a.qpt;
                z.qrow = p.seq.q0 + z.qi0;
                z.nq = min(a.qpt, p.seq.ql - z.qi0);
                z.ql = p.seq.ql;
                z.kl = p.seq.kl;
                z.sink_end = r.sink_end;
                z.ns = r.ns;
                z.jlo = r.jlo;
                z.jhi = r.jhi;
                z.t0 = t0;
                z.nt = (int)min((int64_t)r.nt, to - begin) - t0;
                z.flags = (t0 == 0 ? kStarts : 0u) | (t0 + z.nt == r.nt ? kEnds : 0u);
                z.last = z.flags == kStarts ? (int)((begin + r.nt - 1) / per_cta) : 0;
            }
            begin += p.len;
            at = to;
            if (++ht == a.head_tiles) {
                ht = 0;
                if (++qt == p.q_tiles) {
                    qt = 0;
                    if (++hk == a.Hkv) {
                        hk = 0;
                        do {   // the next sequence that has work
                            if (++s >= a.n_seq) {
                                at = end;
                                break;
                            }
                            p = seq_line(a, next_raw);
                            next_raw = raw_seq(a, s + 1);
                        } while (p.q_tiles == 0);
                    }
                }
            }
            if (!skip) return true;
        }
        return false;
    }
};

// The k-th piece of the run, for a thread or a whole warp; nt = 0 at the end.
DG_DEVINL Piece take(TreeShared& sh, uint32_t k, bool& ok) {
    const int slot = (int)(k % kRing);
    if (!wait(&sh.wfull[slot], (k / kRing) & 1u)) {
        ok = false;
        Piece z;
        z.nt = 0;
        return z;
    }
    const Piece z = sh.piece[slot];
    dg::mbar_arrive(&sh.wempty[slot]);
    return z;
}
// For a whole warp: the piece stays where it is until the warp leaves it.
DG_DEVINL bool await_piece(TreeShared& sh, uint32_t k) { return wait_warp(&sh.wfull[k % kRing], (k / kRing) & 1u); }
DG_DEVINL void leave_piece(TreeShared& sh, uint32_t k) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) dg::mbar_arrive(&sh.wempty[k % kRing]);
}

// Bits below n.
DG_DEVINL uint64_t below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// The keys j0 .. j0 + 63 from lo to hi, and those below `sinks` up to hi.
DG_DEVINL uint64_t keys_between(int j0, int lo, int hi, int sinks) {
    return below(hi - j0 + 1) & (~below(lo - j0) | below(sinks - j0));
}

// The nodes among them that a query sees, `row` being its row.
DG_DEVINL uint64_t seen_nodes(const TreeArgs& a, const Piece& z, int j0, int64_t row) {
    const uint32_t* w = a.mask + row * a.mask_words;
    const int n0 = j0 - (z.kl - z.ql);       // node of bit 0, from -63 on
    auto word = [&](int i) -> uint64_t { return i >= 0 && i < a.mask_words ? w[i] : 0u; };
    const int i = n0 >> 5, sh = n0 & 31;     // (floors)
    uint64_t bits = (word(i) >> sh) | (word(i + 1) << (32 - sh));
    if (sh) bits |= word(i + 2) << (64 - sh);
    return bits & below(z.kl - j0) & ~below(-n0);
}

// ------------------------------------------------------------------ the kernel
template <int D>
__global__ void __launch_bounds__(kThreads, TreeCfg<D>::kCtasPerSm)
    k_tree(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const TreeArgs a) {
    using C = TreeCfg<D>;
    constexpr uint32_t kKVBytes = C::kKVBytes;
    constexpr uint32_t kColS = C::kColS, kColO = C::kColO, kColP = C::kColP, kTmemCols = C::kTmemCols;
    constexpr uint32_t kBufs = C::kBufs;
    using At = RingAt<kBufs>;
    extern __shared__ __align__(1024) unsigned char smem[];
    TreeShared& sh = *reinterpret_cast<TreeShared*>(smem + C::kOffBar);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        dg::mbar_init(&sh.qfull, 1);
        dg::mbar_init(&sh.qempty, 1);
        dg::mbar_init(&sh.oempty, 4);
        for (uint32_t i = 0; i < kBufs; ++i) {
            dg::mbar_init(&sh.full[i], 1);
            dg::mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            dg::mbar_init(&sh.pfull[i], 4);
            dg::mbar_init(&sh.pvdone[i], 1);
        }
        dg::mbar_init(&sh.sfull, 1);
        dg::mbar_init(&sh.sempty, 4);
        dg::mbar_init(&sh.mmadone, 1);
        dg::mbar_init(&sh.met, 4);
        for (int i = 0; i < kRing; ++i) {
            dg::mbar_init(&sh.wfull[i], 1);
            dg::mbar_init(&sh.wempty[i], kReaders);
        }
        sh.abort_flag = 0;
        dg::fence_mbar_init();
    }
    if constexpr (C::kSumsByProduct) {
        if (threadIdx.x < 2 * kAtom / 16)
            reinterpret_cast<uint4*>(smem + C::kOffOnes)[threadIdx.x] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        dg::fence_proxy_async_smem();
    }
    if (warp == 1) {
        dg::tmem_alloc(&sh.tmem_base, kTmemCols);
        dg::tmem_relinquish();
    }
    dg::tc_fence_before();
    __syncthreads();
    dg::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
    dg::pdl_wait();
    dg::pdl_release();
    const Run run = find_run(a, sh);
    const uint32_t sQ = dg::smem_u32(smem + C::kOffQ);

    if (warp == 0) {
        // ------------------------------------------------ the walk and the copies, a whole warp
        // Tile n's keys, then tile n - 1's values, in the ring's order; behind a piece's
        // first keys its queries, whose place the same product frees as that of the second tile's keys.  A lane copies a
        // box of a page's slots; the lanes hold the page numbers of the tiles to come, and ask for
        // the next ones (the next piece's first ones too) before they are needed.
        if (lane == 0) {
            dg::prefetch_tmap(&tmQ);
            dg::prefetch_tmap(&tmK);
            dg::prefetch_tmap(&tmV);
        }
        constexpr int kCols = D / kSub;
        const int box_shift = a.box_shift, size = 1 << box_shift, boxes = kKeys >> box_shift;
        const int ahead = 32 / boxes;                       // tiles whose pages the warp holds
        const int my_tile = lane / boxes, my_box = lane - my_tile * boxes;   // as a holder
        const int box = min(lane, boxes - 1);                                // as a copier
        const uint32_t q_bytes = (uint32_t)(a.hpt * a.qpt) * kSub * 2 * kCols;
        if (lane == 0) sh.zeros = run.zeros;
        Walk walk;
        walk.start(a, run);
        Piece z, zn;
        auto entries = [&](const Piece& x, int i) -> int32_t {   // of tiles i .. i + ahead - 1; n_pages reads zeros
            const int ti = i + my_tile;
            if (ti >= x.nt) return (int32_t)a.kv.n_pages;
            const int j = x.tile(ti) * kKeys + (my_box << box_shift);
            if (j > x.jhi || (j + (size - 1) < x.jlo && j >= x.sink_end)) return (int32_t)a.kv.n_pages;
            const int32_t page = a.kv.page_table[(int64_t)x.s * a.kv.max_pages + (j >> a.kv.page_shift)];
            if (page >= 0 && page < a.kv.n_pages) return page;
            dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            return (int32_t)a.kv.n_pages;
        };
        bool ok = true, more = walk.next(a, zn);
        int32_t en = more ? entries(zn, 0) : 0;
        uint32_t n_keys = 0, n_values = 0, n_queries = 0;   // copies asked for
        int v_page = 0, v_slot = 0, v_hk = 0;               // of the last tile's values
        auto copy = [&](const CUtensorMap* tm, const At& to, int slot, int hk, int page) {
            if (!wait_warp(&sh.empty[to.slot], to.parity ^ 1u)) return false;
            if (lane == 0) dg::mbar_arrive_expect_tx(&sh.full[to.slot], kKVBytes);
            __syncwarp();
            if (lane < boxes)
                dg::tma_load_5d(smem + C::kOffKV + to.slot * kKVBytes + (box << box_shift) * D * 2, tm, 0, a.by_slot * slot,
                                a.mul2 * hk, a.mul3 * hk + a.mul8 * (slot >> 3), page, &sh.full[to.slot]);
            return true;
        };
        auto values = [&]() {                               // of the tile before
            if (!copy(&tmV, At(values_at(n_values)), v_slot, v_hk, v_page)) return false;
            ++n_values;
            return true;
        };
        for (uint32_t k = 0; ok; ++k) {
            const int slot = (int)(k % kRing);
            if (!wait_warp(&sh.wempty[slot], ((k / kRing) & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            z = zn;
            if (!more || aborted(sh)) z.nt = 0;
            z.nt = __shfl_sync(0xffffffffu, z.nt, 0);
            if (lane == 0) {
                sh.piece[slot] = z;
                dg::mbar_arrive(&sh.wfull[slot]);           // releases the piece to its readers
            }
            if (z.nt == 0) break;
            int32_t e = en, e_next = entries(z, ahead);
            int held = 0;                                   // the tile that e's first entries are of
            for (int i = 0; i < z.nt; ++i) {
                if (i == held + ahead) {
                    held = i;
                    e = e_next;
                    e_next = entries(z, i + ahead);
                }
                const int j0 = z.tile(i) * kKeys;
                const int page = __shfl_sync(0xffffffffu, e, ((i - held) * boxes + box) & 31);
                const int at = (j0 + (box << box_shift)) & ((1 << a.kv.page_shift) - 1);
                if (!copy(&tmK, At(keys_at(n_keys)), at, z.hk, page)) {
                    ok = false;
                    break;
                }
                ++n_keys;
                if (n_keys > 1 && !values()) {
                    ok = false;
                    break;
                }
                v_page = page;
                v_slot = at;
                v_hk = z.hk;
                if (i == 0) {
                    if (!wait_warp(&sh.qempty, (k & 1u) ^ 1u)) {   // the last piece's last S has read its queries
                        ok = false;
                        break;
                    }
                    if (lane == 0) dg::mbar_arrive_expect_tx(&sh.qfull, q_bytes);
                    __syncwarp();
                    if (lane < kCols)
                        dg::tma_load_3d(smem + C::kOffQ + lane * kQSub, &tmQ, lane * kSub, z.h0, z.qrow, &sh.qfull);
                    ++n_queries;
                }
                if (i == min(1, z.nt - 1)) {   // the next piece, and its first pages, behind copies on their way
                    more = walk.next(a, zn);
                    en = more ? entries(zn, 0) : 0;
                }
            }
        }
        if (ok && n_keys > 0) ok = values();
        if (!ok && lane == 0) do_abort(sh, a.status);
        if (__any_sync(0xffffffffu, !ok || aborted(sh))) {   // never leave with a copy still landing in shared memory
            const uint32_t top = max(n_keys > 0 ? keys_at(n_keys - 1) + 1 : 0u, n_values > 0 ? values_at(n_values - 1) + 1 : 0u);
            for (uint32_t n = top > kBufs ? top - kBufs : 0u; n < top; ++n) {   // the last use of each buffer
                const bool is_keys = n == 0 || (n & 1u);
                if (is_keys ? (n + 1) / 2 < n_keys : n / 2 - 1 < n_values) (void)wait_warp(&sh.full[At(n).slot], At(n).parity);
            }
            if (n_queries > 0) (void)wait_warp(&sh.qfull, (n_queries - 1u) & 1u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ the products
        if (dg::elect_leader()) {
            // S = Q K^T: both K-major, bit 13 negates Q; O += P V: the values' rows are N-major
            const uint32_t idS = dg::instr_desc(kTile, kKeys, false) | (a.negate ? 1u << 13 : 0u);
            constexpr uint32_t idO = dg::instr_desc(kTile, C::kValueCols, true);
            const uint32_t sOnes = dg::smem_u32(smem + C::kOffOnes);
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t k = 0; ok && !aborted(sh); ++k) {
                const int nt = take(sh, k, ok).nt;
                if (nt == 0) break;
                if (!wait(&sh.qfull, k & 1u)) {
                    ok = false;
                    break;
                }
                for (int i = 0; i <= nt; ++i) {
                    if (i < nt) {   // S of tile g + i, once the softmax has read the last S
                        const uint32_t gs = g + (uint32_t)i;
                        const At at(keys_at(gs));
                        if (!wait(&sh.full[at.slot], at.parity) || !wait(&sh.sempty, (gs & 1u) ^ 1u)) {
                            ok = false;
                            break;
                        }
                        dg::tc_fence_after();
                        const uint32_t sK = dg::smem_u32(smem + C::kOffKV + at.slot * kKVBytes);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t offq = (uint32_t)(kk >> 2) * kQSub + (uint32_t)(kk & 3) * 32u;
                            const uint32_t offk = (uint32_t)(kk >> 2) * kAtom + (uint32_t)(kk & 3) * 32u;
                            dg::tc_mma_f16(tmem + kColS, dg::smem_desc(sQ + offq, 16, 1024, 128),
                                           dg::smem_desc(sK + offk, 16, (D / kSub) * kAtom, 128), idS, kk > 0 ? 1u : 0u);
                        }
                        dg::tc_commit(&sh.sfull);
                        dg::tc_commit(&sh.empty[at.slot]);
                        if (i == nt - 1) dg::tc_commit(&sh.qempty);   // the queries, after the piece's last S
                    }
                    if (i >= 1) {   // O += P V of tile g + i - 1 once the softmax has written P
                        const uint32_t gp = g + (uint32_t)i - 1u;
                        const int st = (int)(gp & 1u);
                        const At at(values_at(gp));
                        if (!wait(&sh.pfull[st], (gp >> 1) & 1u) || !wait(&sh.full[at.slot], at.parity) ||
                            (i == 1 && !wait(&sh.oempty, (k & 1u) ^ 1u))) {   // the last piece's O read out
                            ok = false;
                            break;
                        }
                        dg::tc_fence_after();
                        const uint32_t sV = dg::smem_u32(smem + C::kOffKV + at.slot * kKVBytes);
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk) {
                            const uint32_t v = sV + (uint32_t)kk * 16u * D * 2u;   // 16 keys; the next 64 columns: kAtom on, or the ones
                            dg::tc_mma_f16_ts(tmem + kColO, tmem + kColP + (uint32_t)(st * 32 + kk * 8),
                                              dg::smem_desc(v, C::kSumsByProduct ? sOnes - v : kAtom, (D / kSub) * kAtom, 128), idO,
                                              (i > 1 || kk > 0) ? 1u : 0u);
                        }
                        dg::tc_commit(&sh.pvdone[st]);
                        dg::tc_commit(&sh.empty[at.slot]);
                    }
                }
                g += (uint32_t)nt;
            }
            if (!ok) do_abort(sh, a.status);
            dg::tc_commit(&sh.mmadone);   // every product has completed before the tensor memory is released
            (void)wait(&sh.mmadone, 0);
        }
    } else {
        // ------------------------------------------------ softmax, a row a thread
        const int q = warp & 3;   // the quarter of TMEM's lanes this warp may access
        const int row = q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        uint32_t g = 0, masked = 0, meetings = 0;
        bool ok = true, to_join = false;
        // Each warp has left something for the others.  (What it leaves next but one is behind another meeting: two places
        // of each kind are enough.)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) dg::mbar_arrive(&sh.met);
            return wait_warp(&sh.met, meetings++ & 1u);
        };
        for (uint32_t k = 0; ok; ++k) {
            if (!await_piece(sh, k)) {
                ok = false;
                break;
            }
            const Piece& z = sh.piece[k % kRing];   // (read again where it is needed: kept in registers it spills them)
            const int nt = z.nt;
            if (nt == 0) break;
            const int ctx = z.kl - z.ql;
            const int qi = row / a.hpt, hi = row - qi * a.hpt;
            const bool valid = qi < z.nq && hi < z.nh;
            const bool idle = !__any_sync(0xffffffffu, valid);   // no row of this warp's: only its arrivals
            const int64_t qrow = (int64_t)z.qrow + (valid ? qi : 0);
            int pos = ctx + z.qi0 + (valid ? qi : 0), low = ctx + z.qi0, top = low + z.nq - 1;
            if (a.mask && a.window >= 0) {   // the nodes' own positions, and the last of the item's
                pos = max(a.positions[qrow], ctx);
                const int w = __reduce_max_sync(0xffffffffu, valid ? pos : ctx), w0 = __reduce_min_sync(0xffffffffu, valid ? pos : 0x7fffffff);
                int32_t* tops = sh.top_position[k & 1u];
                if (lane == 0) {
                    tops[q] = w;
                    tops[4 + q] = w0;
                }
                if (!meet()) {
                    ok = false;
                    break;
                }
                top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
                low = min(min(tops[4], tops[5]), min(tops[6], tops[7]));
            }
            const int all_hi = a.mask ? ctx - 1 : ctx + z.qi0;   // every row sees keys up to it,
            const int all_lo = a.window < 0 ? 0 : max(0, top - a.window);   // from here on;
            const int any_lo = a.window < 0 ? 0 : max(0, low - a.window);   // some row from here on;
            const int row_lo = a.window < 0 ? 0 : max(0, pos - a.window), row_hi = a.mask ? ctx - 1 : pos;   // and this one
            float m_ref = -INFINITY, l = 0.f, lr = 0.f;   // lr: of the rounded weights
            for (int i = 0; i < nt; ++i) {
                const uint32_t gi = g + (uint32_t)i;
                if (!wait_warp(&sh.sfull, gi & 1u)) {
                    ok = false;
                    break;
                }
                dg::tc_fence_after();
                float x[2][32];
                if (!idle) {
                    uint32_t raw[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) dg::tmem_ld32_nowait(tmem + lane_base + kColS + (uint32_t)(c * 32), raw[c]);
                    dg::tmem_ld_wait_dep(raw[0]);
                    dg::tmem_ld_wait_dep(raw[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[c][e] = __uint_as_float(raw[c][e]);
                }
                dg::tc_fence_before();
                __syncwarp();
                if (lane == 0) dg::mbar_arrive(&sh.sempty);
                const int j0 = z.tile(i) * kKeys, j1 = j0 + kKeys - 1;
                if (j1 > all_hi || (j0 < all_lo && j1 >= a.sinks)) {   // not all of it is seen by all
                    uint64_t m = valid ? keys_between(j0, row_lo, row_hi, a.sinks) : 0ull;
                    // rows' ranges follow each other without gaps: some row sees each key of the first to the last
                    uint64_t any_row = keys_between(j0, any_lo, a.mask ? ctx - 1 : top, a.sinks);
                    if (a.mask && j1 >= ctx) {   // nodes: the warps join what their rows see
                        const uint64_t nodes = valid ? seen_nodes(a, z, j0, qrow) : 0ull;
                        m |= nodes;
                        const uint32_t w0 = __reduce_or_sync(0xffffffffu, (uint32_t)nodes);
                        const uint32_t w1 = __reduce_or_sync(0xffffffffu, (uint32_t)(nodes >> 32));
                        uint64_t* seen = sh.seen[masked & 1u];
                        ++masked;
                        if (lane == 0) seen[q] = (uint64_t)w1 << 32 | w0;
                        if (!meet()) {
                            ok = false;
                            break;
                        }
                        any_row |= seen[0] | seen[1] | seen[2] | seen[3];
                    }
                    if (~any_row) {   // the values nobody sees
                        const At at(values_at(gi));
                        if (!wait_warp(&sh.full[at.slot], at.parity)) {
                            ok = false;
                            break;
                        }
                        unsigned char* vt = smem + C::kOffKV + at.slot * kKVBytes;
                        for (int c = row; c < kKeys * (D / kSub) * 8; c += 128) {   // 16-byte chunks
                            if (!(any_row >> ((c >> 6) / (D / kSub) * 8 + ((c >> 3) & 7)) & 1u))
                                reinterpret_cast<uint4*>(vt)[c] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        dg::fence_proxy_async_smem();   // before the product reads them (pfull below)
                    }
                    if (!idle) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t w = c ? (uint32_t)(m >> 32) : (uint32_t)m;
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[c][e] = w >> e & 1u ? x[c][e] : -INFINITY;
                        }
                    }
                }
                if (!idle) {
                    float mx[16];   // the tile's maximum of the raw scores
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        mx[e] = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
#pragma unroll
                    for (int wd = 8; wd >= 1; wd >>= 1)
#pragma unroll
                        for (int e = 0; e < wd; ++e) mx[e] = fmaxf(mx[e], mx[e + wd]);
                    const float tmax = mx[0] * a.scale_log2;   // (-inf stays: the scale is above 0)
                    const bool rescale = __any_sync(0xffffffffu, valid && tmax > m_ref + kRescaleAbove);
                    // O is rescaled after this piece's last P V only; else P's buffer must have been read by the
                    // product two tiles back, which may be the last piece's
                    if ((rescale && i > 0) || gi > 1) {
                        const uint32_t gj = (rescale && i > 0) ? gi - 1 : gi - 2;
                        if (!wait_warp(&sh.pvdone[gj & 1u], (gj >> 1) & 1u)) {
                            ok = false;
                            break;
                        }
                        dg::tc_fence_after();
                    }
                    if (rescale) {
                        const float m_new = fmaxf(m_ref, tmax);
                        const float alpha = m_new == -INFINITY ? 1.f : ex2(m_ref - m_new);
                        l *= alpha;
                        lr *= alpha;
                        if (i > 0) {
                            if constexpr (C::kSumsByProduct) {
                                const uint32_t ta = tmem + lane_base + C::kColL;
                                dg::tmem_st1(ta, dg::tmem_ld1(ta) * alpha);
                            }
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                const uint32_t ta = tmem + lane_base + kColO + (uint32_t)(c * 32);
                                dg::tmem_ld32(ta, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                                dg::tmem_st32(ta, o);
                                dg::tmem_st_wait();   // before the next chunk's load may reuse the registers
                            }
                        }
                        m_ref = m_new;
                    }
                    const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t cc = f2(a.scale_log2, a.scale_log2), mm = f2(neg_m, neg_m);
                    uint64_t acc = f2(0.f, 0.f);
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float z0, z1;
                            f2_split(f2_fma(f2(x[c][e], x[c][e + 1]), cc, mm), z0, z1);
                            const float p0 = ex2(z0), p1 = ex2(z1);
                            acc = f2_add(acc, f2(p0, p1));
                            pk[c * 16 + e / 2] = pack_bf16x2(p0, p1);
                        }
                    }
                    dg::tmem_st32u(tmem + lane_base + kColP + (gi & 1u) * 32u, pk);
                    if constexpr (!C::kSumsByProduct) {   // the rounded weights' sum, while they are on their way
                        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 32; ++e) add_bf16x2(pk[e], rs[2 * (e & 1)], rs[2 * (e & 1) + 1]);
                        lr += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                    }
                    float sa, sb;
                    f2_split(acc, sa, sb);
                    l += sa + sb;
                    dg::tmem_st_wait();
                }
                dg::tc_fence_before();
                __syncwarp();
                if (lane == 0) dg::mbar_arrive(&sh.pfull[gi & 1u]);
            }
            if (!ok) break;
            const uint32_t gl = g + (uint32_t)nt - 1u;   // the piece's last P V
            if (!wait_warp(&sh.pvdone[gl & 1u], (gl >> 1) & 1u)) {
                ok = false;
                break;
            }
            dg::tc_fence_after();
            if (!idle) {
                const bool whole = z.flags == (kStarts | kEnds);
                if constexpr (C::kSumsByProduct) lr = dg::tmem_ld1(tmem + lane_base + C::kColL);
                const float inv = lr > 0.f ? 1.f / lr : 0.f;
                const int64_t out = qrow * a.Hq + z.h0 + (valid ? hi : 0);
                const int64_t slot = (int64_t)blockIdx.x * 2 + (z.flags & kStarts ? 1 : 0);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    dg::tmem_ld32(tmem + lane_base + kColO + (uint32_t)(c * 32), o);
                    if (!valid) continue;
                    if (whole) {
                        if (!(l > 0.f)) {   // a row that sees nothing
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e];
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(a.o + out * D + c * 32 + e) = make_uint4(
                                pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv), pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            a.part_o[(slot * (D / 4) + c * 8 + e / 4) * a.rows + row] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (valid && whole && a.lse) a.lse[out] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
                if (valid && !whole) a.part_ml[slot * a.rows + row] = make_float4(m_ref, l, lr, 0.f);
            }
            if (row == 0 && (z.flags & kStarts) && !(z.flags & kEnds)) {
                a.desc[2 * blockIdx.x] = make_int4(z.last - (int)blockIdx.x, z.qrow, z.h0, z.nq);
                a.desc[2 * blockIdx.x + 1] = make_int4(z.nh, 0, 0, 0);
                to_join = true;
            }
            dg::tc_fence_before();
            __syncwarp();
            if (lane == 0) dg::mbar_arrive(&sh.oempty);   // O read out: the next piece may overwrite it
            leave_piece(sh, k);
            g += (uint32_t)nt;
        }
        if (!ok) do_abort(sh, a.status);
        if (row == 0 && !to_join) a.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }

    dg::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        dg::tc_fence_after();
        dg::tmem_dealloc(tmem, kTmemCols);
    }
    if (!sh.zeros) return;
    // the sequences without keys: their rows of zeros
    for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
        const dg::PagedSeq p = dg::paged_seq(a.kv, a.cu_q, a.total_q, s, dg::kMaxKeys);
        if (!p.ok || p.kl != 0 || p.ql > a.max_q_len) continue;
        const int64_t first = (int64_t)p.q0 * a.Hq, rows = (int64_t)p.ql * a.Hq;
        for (int64_t i = threadIdx.x; i < rows * (D / 8); i += kThreads)
            reinterpret_cast<uint4*>(a.o + first * D)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse)
            for (int64_t i = threadIdx.x; i < rows; i += kThreads) a.lse[first + i] = -INFINITY;
    }
}

// Joins an item's pieces: the last one of CTA c (slot 1) and the first ones (slot 0) of the CTAs that follow
// it.  blockIdx.x = c, blockIdx.y = 16 of the dimensions; most blocks find nothing to join.  A thread owns a row's
// 16 dimensions of every (kJoinThreads / rows)-th piece, kAtOnce pieces on their way at a time; the groups join in shared
// memory in a fixed order.  A few items of up to dozens of pieces each take large blocks (us large / small: one request over
// 16k keys 32 / 48, over 1k 21 / 19.5); more items, of which most blocks find none, small ones (8 requests over 2.3k keys
// 33 / 27, 64 over 400 51 / 36.6).
constexpr int kJoinDims = 16;
template <int D, int kJoinThreads, int kAtOnce>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const TreeArgs a) {
    constexpr int Q = kJoinDims / 4;
    __shared__ float4 s_o[kJoinThreads][Q];
    __shared__ float4 s_ml[kJoinThreads];
    dg::pdl_wait();
    dg::pdl_release();
    const int c = blockIdx.x;
    const int4 d0 = a.desc[2 * c];
    if (d0.x == 0) return;
    const int n = d0.x + 1, nh = a.desc[2 * c + 1].x;
    const int groups = kJoinThreads / a.rows, group = (int)threadIdx.x / a.rows, row = (int)threadIdx.x - group * a.rows;
    const int qi = row / a.hpt, hi = row - qi * a.hpt;
    const bool mine = group < groups && qi < d0.w && hi < nh;
    auto slot = [&](int i) -> int64_t { return i == 0 ? (int64_t)c * 2 + 1 : (int64_t)(c + i) * 2; };
    float M = -INFINITY, L = 0.f, Lr = 0.f;
    float4 o[Q];
#pragma unroll
    for (int e = 0; e < Q; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    // adds a piece (maximum, sums, output) to the thread's
    auto add = [&](const float4& ml, const float4 (&v)[Q]) {
        if (ml.x == -INFINITY && ml.y == 0.f) return;   // the row saw nothing of it, whatever its values
        // (a maximum of -inf beside a sum that is a NaN: all it saw there were NaNs, which it keeps)
        const float m = fmaxf(M, ml.x), f0 = M == -INFINITY ? 1.f : ex2(M - m), f1 = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);
        M = m;
        L = L * f0 + ml.y * f1;
        Lr = Lr * f0 + ml.z * f1;
#pragma unroll
        for (int e = 0; e < Q; ++e) {
            o[e].x = o[e].x * f0 + v[e].x * f1;
            o[e].y = o[e].y * f0 + v[e].y * f1;
            o[e].z = o[e].z * f0 + v[e].z * f1;
            o[e].w = o[e].w * f0 + v[e].w * f1;
        }
    };
    if (mine) {
        for (int i0 = group; i0 < n; i0 += kAtOnce * groups) {
            float4 ml[kAtOnce];
            float4 v[kAtOnce][Q];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + k * groups;
                ml[k] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
                if (i >= n) continue;
                ml[k] = a.part_ml[slot(i) * a.rows + row];
#pragma unroll
                for (int e = 0; e < Q; ++e) v[k][e] = a.part_o[(slot(i) * (D / 4) + blockIdx.y * Q + e) * a.rows + row];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) add(ml[k], v[k]);
        }
    }
    if (group > 0) {
        s_ml[threadIdx.x] = make_float4(M, L, Lr, 0.f);
#pragma unroll
        for (int e = 0; e < Q; ++e) s_o[threadIdx.x][e] = o[e];
    }
    __syncthreads();
    if (group > 0 || !mine) return;
    for (int k = 1; k < min(groups, n); ++k) {
        float4 v[Q];
#pragma unroll
        for (int e = 0; e < Q; ++e) v[e] = s_o[k * a.rows + row][e];
        add(s_ml[k * a.rows + row], v);
    }
    const float inv = Lr > 0.f ? 1.f / Lr : 0.f;
    const int64_t out = ((int64_t)d0.y + qi) * a.Hq + d0.z + hi;
    uint4* dst = reinterpret_cast<uint4*>(a.o + out * D + blockIdx.y * kJoinDims);
#pragma unroll
    for (int e = 0; e < Q; e += 2)
        dst[e / 2] = make_uint4(pack_bf16x2(o[e].x * inv, o[e].y * inv), pack_bf16x2(o[e].z * inv, o[e].w * inv),
                                pack_bf16x2(o[e + 1].x * inv, o[e + 1].y * inv), pack_bf16x2(o[e + 1].z * inv, o[e + 1].w * inv));
    if (blockIdx.y == 0 && a.lse) a.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------ host side
// Rows of a piece in the workspace.
int piece_rows(int32_t max_q_len, int32_t group) {
    return (int)std::min<int64_t>(kTile, ((int64_t)max_q_len * group + 31) / 32 * 32);
}
size_t piece_bytes(int32_t D, int rows) {
    const size_t ctas = D == 256 ? TreeCfg<256>::kMaxCtas : TreeCfg<128>::kMaxCtas;
    return ctas * 32 + ctas * 2 * rows * ((size_t)D * 4 + 16);
}

// Whether a call takes the kernels for few rows (dg_tree_split.cu), whose items of up to 16 rows pass over the keys each; a
// tile here takes all of a key head's up to 128, and a call 10 us more to start and to join.  The lengths are not known to the
// host.  Measured (us there / here), trees of one query head a key head, contexts of up to 400, 2300 and 8000 tokens:
//   heads of 64: 32 sequences, 8 key heads, 17 rows 17.6 / 20.6, 35 / 34, 84 / 97, 20 rows 17.9 / 20.9, 43 / 34, 91 / 91; 4 sequences, 32 rows
//     10.7 / 14.6, 16.2 / 16.1, 24.5 / 21.1;
//   heads of 128: 32 sequences, 8 key heads, 16 rows 19.9 / 21.3, 49 / 47, 116 / 114, 20 rows 25.4 / 24.6, 62 / 48, 145 / 120; 4
//     sequences, 20 rows 11.1 / 15.9, 18.4 / 19.2, 39 / 31; 2, 32 rows 11.1 / 21.0, 18.2 / 24.8, 33.2 / 33.5;
//   heads of 256: 32 sequences, 4 key heads, 9 rows 22.2 / 24.0, 54 / 47, 131 / 124, 16 rows 23.9 / 21.2, 55 / 48, 124 / 115; 2
//     sequences, 16 rows 12.5 / 22.2, 20.6 / 26.0, 27.7 / 30.3.
// Over 2414 shapes (heads of 64, 128, 256, 1 to 8 key heads, 1 to 128 sequences, 9 to 64 rows) the rule loses 1.6 % to the
// better path on average.  The most, 71 %, is 64 rows of short contexts (8 sequences, one key head of 256, 400 tokens 13.1 / 22.4),
// which over 8000 tokens lose up to 40 % there.
bool few_rows(int32_t n_seq, int32_t max_q_len, int32_t Hkv, int32_t group, int32_t D) {
    const int64_t rows = (int64_t)max_q_len * group;
    return rows <= (D == 64 ? 18 : D == 128 ? 16 : 8) || (rows <= 64 && n_seq * (int64_t)Hkv * rows * D <= 98304);
}

template <int D>
dg_status launch_tree(const dghost::TreeCall& c, void* workspace, cudaStream_t stream) {
    using C = TreeCfg<D>;
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    TreeArgs a;
    a.o = c.o;
    a.lse = c.lse;
    a.cu_q = c.cu_q;
    a.mask = c.mask;
    a.positions = c.positions;
    a.total_q = c.total_q;
    a.n_seq = c.n_seq;
    a.max_q_len = c.max_q_len;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.group = c.Hq / c.Hkv;
    a.mask_words = c.mask_words;
    a.window = c.window;
    a.sinks = c.sinks;
    a.hpt = std::min(a.group, kTile);
    a.qpt = kTile / a.hpt;
    a.head_tiles = (a.group + kTile - 1) / kTile;
    a.rows = piece_rows(c.max_q_len, a.group);
    // a scale of 0 weighs every key alike: the smallest float keeps masked scores (-inf) what they are and moves
    // no finite score by more than 5e-7
    a.scale_log2 = std::max(fabsf(c.scale) * kLog2e, std::numeric_limits<float>::denorm_min());
    a.negate = c.scale < 0.f;
    a.kv = c.kv;
    a.status = dghost::status_word();
    CUtensorMap tq, tk, tv;
    {   // queries: 64 columns x the item's heads x its queries
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.total_q};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.Hq * D * 2};
        const uint32_t box[3] = {(uint32_t)kSub, (uint32_t)a.hpt, (uint32_t)a.qpt};
        if (!dghost::encode_tmap(&tq, 0, 3, const_cast<uint16_t*>(c.q), dims, strides, box, 128)) return DG_ERR_CUDA;
    }
    // Keys and values lie in shared memory as [8 slots][64 columns of D][slot], so that one copy brings a head's slots of
    // a page, up to 64.  Its dimensions are 64 columns, 8 slots, D / 64, slots / 8, page: the head has to go with
    // one of them.  Slot by slot its columns follow the last head's; head by head its slots do.  For a cache with gaps
    // between the two a copy is of 8 slots.  (32 trees of 64 nodes over pages of 16, all keys in L2: 61 us, with a copy for
    // every 64 columns 65; from memory 82 both.)
    const uint64_t cols = D / kSub, ps = 1ull << a.kv.page_shift;
    uint64_t dims[5] = {(uint64_t)kSub, 8, cols, ps / 8, (uint64_t)a.kv.n_pages};
    uint64_t strides[4] = {(uint64_t)a.kv.slot_stride * 2, (uint64_t)kSub * 2, (uint64_t)a.kv.slot_stride * 16,
                           (uint64_t)a.kv.page_stride * 2};
    a.box_shift = std::min(a.kv.page_shift, 6);
    uint32_t box[5] = {(uint32_t)kSub, 8, (uint32_t)cols, 1u << (a.box_shift - 3), 1};
    a.by_slot = a.mul2 = a.mul3 = 0;
    a.mul8 = 1;
    if (a.kv.slot_stride < (1LL << 36) && (a.kv.head_stride == D || a.Hkv == 1)) {
        dims[2] *= (uint64_t)a.Hkv;
        a.mul2 = (int32_t)cols;
    } else if (a.kv.slot_stride < (1LL << 36) && a.kv.head_stride == a.kv.slot_stride << a.kv.page_shift) {
        dims[3] *= (uint64_t)a.Hkv;
        a.mul3 = (int32_t)(ps / 8);
    } else {
        dims[1] = ps;
        dims[3] = (uint64_t)a.Hkv;
        strides[2] = (uint64_t)a.kv.head_stride * 2;
        a.box_shift = 3;
        box[3] = 1;
        a.by_slot = a.mul3 = 1;
        a.mul8 = 0;
    }
    for (auto [tm, base] : {std::pair<CUtensorMap*, uint16_t*>{&tk, a.kv.k}, {&tv, a.kv.v}})
        if (!dghost::encode_tmap(tm, 0, 5, base, dims, strides, box, 128)) return DG_ERR_CUDA;
    // the attribute once a device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DG_ERR_CUDA;
    if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        if (cudaFuncSetAttribute(k_tree<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tree_smem<D>()) != cudaSuccess)
            return DG_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)std::min(sms * C::kCtasPerSm, C::kMaxCtas);
    a.desc = static_cast<int4*>(workspace);
    a.part_o = reinterpret_cast<float4*>(a.desc + 2 * C::kMaxCtas);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + (size_t)C::kMaxCtas * 2 * (D / 4) * a.rows);
    cudaError_t e = dghost::launch_pdl(k_tree<D>, dim3(grid), dim3(kThreads), tree_smem<D>(), stream, tq, tk, tv, a);
    dghost::count_launch();
    if (e != cudaSuccess) return DG_ERR_CUDA;
    const int64_t items = (int64_t)a.n_seq * a.Hkv * a.head_tiles * (((int64_t)a.max_q_len + a.qpt - 1) / a.qpt);
    e = items * 16 < grid ? dghost::launch_pdl(k_tree_join<D, 512, 4>, dim3(grid, D / kJoinDims), dim3(512), 0, stream, a)
                         : dghost::launch_pdl(k_tree_join<D, 128, 2>, dim3(grid, D / kJoinDims), dim3(128), 0, stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
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
    dghost::TreeCall c;
    const dg_status ok = dghost::paged_kv(cache, D, &c.kv);
    if (ok != DG_OK) return ok;
    if (!workspace || workspace_bytes < dg_tree_attention_workspace_bytes(n_seq, max_q_len, Hq, Hkv, D))
        return DG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DG_ERR_ALIGNMENT;
    c.q = q;
    c.o = o;
    c.lse = lse;
    c.cu_q = cu_q;
    c.mask = mask;
    c.positions = positions;
    c.total_q = total_q;
    c.n_seq = n_seq;
    c.max_q_len = max_q_len;
    c.Hq = Hq;
    c.Hkv = Hkv;
    c.mask_words = mask_words;
    c.window = window;
    c.sinks = window < 0 ? 0 : sinks;
    c.scale = scale;
    const cudaStream_t st = (cudaStream_t)stream;
    if (few_rows(n_seq, max_q_len, Hkv, Hq / Hkv, D)) return dghost::tree_split(c, D, workspace, st);
    if (D == 64) return launch_tree<64>(c, workspace, st);
    return D == 128 ? launch_tree<128>(c, workspace, st) : launch_tree<256>(c, workspace, st);
}

}  // namespace

extern "C" size_t dg_tree_attention_workspace_bytes(int32_t n_seq, int32_t max_q_len, int32_t Hq, int32_t Hkv, int32_t D) {
    if (n_seq < 1 || max_q_len < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
    // what either path needs, so that a workspace for a program's largest call serves its smaller ones
    return std::max(piece_bytes(D, piece_rows(max_q_len, Hq / Hkv)), dghost::tree_split_bytes(max_q_len, Hq / Hkv, D));
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
