// dg_paged_split.cuh -- the kernels of attention of a few query rows a sequence over the paged key / value cache
// (dg_paged_attention in dg_paged_attn.cu, which tells how they work; with Tree, dg_tree_attention and
// dg_sink_attention in dg_tree_split.cu).
#pragma once

#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dg_paged.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCtas = 512;              // grid bound the workspace is sized for
constexpr float kRescaleAbove = 8.f;       // log2 units the maximum may grow before it moves: P <= 2^8

struct SplitArgs {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    const int32_t* cu_q;
    const uint8_t* causal;
    int64_t total_q;
    int32_t n_seq, max_q_len, Hq, Hkv, group, window;
    float scale_log2;
    dg::PagedKV kv;
    float* part_o;    // [grid][2][rows][D]
    float4* part_ml;  // [grid][2][rows]: maximum, sum, sum of the rounded weights, -
    int4* desc;       // [grid][2]: CTAs that follow (0: nothing to join), rows, first row of q, key head; first row
    unsigned* status;
};

// Of a drafted tree, or of a window with first tokens that stay visible (no mask: causal).
struct TreeSplitArgs : SplitArgs {
    const uint32_t* mask;
    const int32_t* positions;
    int32_t mask_words, sinks;
};
template <typename A>
constexpr bool kIsTree = std::is_same_v<A, TreeSplitArgs>;
template <bool Tree>
using SplitArgsOf = std::conditional_t<Tree, TreeSplitArgs, SplitArgs>;

template <int D, int NB>
struct SplitCfg {
    // Warps, keys of a warp's step, stages of its ring and CTAs an SM, measured on contexts from 1k to 128k
    // keys, one to 256 requests: for heads of 64 (8, 16, 3, 2), (4, 16, 3, 4) and (8, 16, 2, 3) come within 3 % of
    // (4, 32, 3, 2) either way; for 128 and eight rows (4, 16, 3, 2) takes 228 us where (6, 16, 2, 2) takes 218
    // and (8, 16, 3, 1) 233 (64 requests over 8k keys), but 16 rows need the registers of eight warps: 64 us
    // against 70 (32 requests of 5 drafts over 4k); for 256 (4, 16, 3, 1) takes 85 us where (7, 16, 2, 1) takes
    // 76.5 (128 requests over 1.2k keys), and the same on one long context.
    // 16 rows of 256 with their queries in registers, (7, 16, 2, 1), spill: 41.7 and 243 us (16 requests of 5 drafts
    // over 3k keys, 64 of 4 over 8k) against 38.1 and 234 with six warps and the queries in shared memory.
    static constexpr bool kSharedQ = D == 256 && NB == 2;
    static constexpr int kWarps = D == 64 ? 4 : D == 256 ? (NB == 1 ? 7 : 6) : NB == 1 ? 6 : 4, kThreads = kWarps * 32;
    static constexpr int kStep = D == 64 ? 32 : 16;        // keys of a warp's step
    static constexpr int kTileKeys = kWarps * kStep;       // keys of a tile
    static constexpr int kStages = D == 256 || (D == 128 && NB == 1) ? 2 : 3;
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    static constexpr uint32_t kHalf = kStep * D * 2;       // the keys of a step (or its values)
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr uint32_t kRing = kStages * kStage;    // a warp's ring
    static constexpr size_t kOffQ = (size_t)kWarps * kRing;  // two pieces' queries, when they lie in shared memory
    static constexpr size_t kSmem = kOffQ + (kSharedQ ? 2 * 8 * NB * D * 2 : 0);
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
// 16 bytes, or zeros when !ok (nothing is read then).
DG_DEVINL void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
DG_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DG_DEVINL void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
DG_DEVINL void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DG_DEVINL void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DG_DEVINL uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
DG_DEVINL void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The keys a query at position pos may see: [lo, hi], empty when hi < lo.
DG_DEVINL void key_range(int pos, int kl, int window, bool causal, int& lo, int& hi) {
    const int64_t W = window;
    lo = W >= 0 ? (int)max((int64_t)0, (int64_t)pos - W) : 0;
    hi = causal ? min(pos, kl - 1) : W >= 0 ? (int)min((int64_t)kl - 1, (int64_t)pos + W) : kl - 1;
}

// A sequence on the line: its row tiles, and the key tiles each of its items visits (one when it
// has queries and no keys, so that its rows get their zeros).
struct SeqPlan {
    dg::PagedSeq seq;
    int row_tiles, tile0, tiles;
    bool causal;
    int klo, sink_end, ns;   // of a tree: the first key behind the first tokens, their end and tiles of their own
    DG_DEVINL int64_t cost(int Hkv) const { return (int64_t)row_tiles * tiles * Hkv; }
};

template <int Rows, int Tile, typename A>
DG_DEVINL SeqPlan seq_plan(const A& a, int s) {
    SeqPlan p;
    p.seq = dg::paged_seq(a.kv, a.cu_q, a.total_q, s, dg::kMaxKeys);
    if constexpr (kIsTree<A>) {
        if (p.seq.ql > a.max_q_len) p.seq.ok = false;
        p.causal = !a.mask;
        p.row_tiles = p.seq.ok ? (int)(((int64_t)p.seq.ql * a.group + Rows - 1) / Rows) : 0;
        p.tile0 = p.klo = p.sink_end = p.ns = 0;
        p.tiles = 1;
        if (p.row_tiles > 0 && p.seq.kl > 0) {
            // positions begin at the context's length: nobody's window reaches farther back than the first one's
            p.klo = a.window < 0 ? 0 : max(0, p.seq.kl - p.seq.ql - a.window);
            p.sink_end = min(a.sinks, p.klo);
            p.ns = min((p.sink_end + Tile - 1) / Tile, p.klo / Tile);
            p.tiles = p.ns + (p.seq.kl - 1) / Tile - p.klo / Tile + 1;
        }
        return p;
    }
    p.causal = a.causal[s] != 0;
    p.row_tiles = p.seq.ok ? (int)(((int64_t)p.seq.ql * a.group + Rows - 1) / Rows) : 0;
    p.tile0 = 0;
    p.tiles = 1;
    if (p.row_tiles > 0 && p.seq.kl > 0) {
        int lo, hi, first, last;
        key_range(p.seq.kl - p.seq.ql, p.seq.kl, a.window, p.causal, first, hi);
        key_range(p.seq.kl - 1, p.seq.kl, a.window, p.causal, lo, last);
        p.tile0 = first / Tile;
        p.tiles = last / Tile - p.tile0 + 1;
    }
    return p;
}

DG_DEVINL int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The line's length and where a CTA's run starts on it.
struct Run {
    int64_t total, per_cta, start, end;
    int seq;            // the sequence at `start`
    int64_t seq_start;  // and where it begins
};

template <int Rows, int Tile, int kWarps, typename A>
DG_DEVINL Run find_run(const A& a) {
    constexpr int kThreads = kWarps * 32;
    __shared__ int64_t sums[4 * kWarps];
    __shared__ int64_t found_start;
    __shared__ int found_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Run r;
    auto cut = [&](int64_t total) {
        r.total = total;
        r.per_cta = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
        r.start = min(total, (int64_t)blockIdx.x * r.per_cta);
        r.end = min(total, r.start + r.per_cta);
        r.seq = 0;
        r.seq_start = 0;
    };
    auto cost_of = [&](int s) -> int64_t {
        const SeqPlan p = seq_plan<Rows, Tile>(a, s);
        if (blockIdx.x == 0 && (!p.seq.ok || p.seq.ql > a.max_q_len)) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        return p.cost(a.Hkv);
    };
    auto scan = [&](int64_t c) {
        int64_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        return incl;
    };
    if (a.n_seq <= 32) {   // every warp by itself: nothing to wait for
        const int64_t c = lane < a.n_seq ? cost_of(lane) : 0, incl = scan(c);
        cut(__shfl_sync(0xffffffffu, incl, 31));
        const uint32_t hit = __ballot_sync(0xffffffffu, incl - c <= r.start && r.start < incl);
        if (hit) {
            r.seq = __ffs(hit) - 1;
            r.seq_start = __shfl_sync(0xffffffffu, incl - c, r.seq);
        }
        return r;
    }
    constexpr int kFew = 4;
    if (a.n_seq <= kFew * kThreads) {   // up to four sequences a thread, read at once
        int64_t c[kFew], incl[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k) c[k] = k * kThreads + tid < a.n_seq ? cost_of(k * kThreads + tid) : 0;
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            incl[k] = scan(c[k]);
            if (lane == 31) sums[k * kWarps + warp] = incl[k];
        }
        __syncthreads();
        int64_t total = 0, before[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) before[k] = total;
                total += sums[k * kWarps + w];
            }
        cut(total);
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            const int64_t to = before[k] + incl[k];
            if (to - c[k] <= r.start && r.start < to) {
                found_seq = k * kThreads + tid;
                found_start = to - c[k];
            }
        }
        __syncthreads();
        r.seq = found_seq;
        r.seq_start = found_start;
        return r;
    }
    int64_t mine = 0, first_cost = 0;
    for (int s = tid; s < a.n_seq; s += kThreads) {
        const int64_t c = cost_of(s);
        if (s == tid) first_cost = c;
        mine += c;
    }
    mine = warp_sum(mine);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    cut(total);
    if (r.start >= r.end) return r;   // the same for the whole CTA
    int64_t base = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += kThreads) {
        const int s = s0 + tid;
        const int64_t c = s0 == 0 ? first_cost : s < a.n_seq ? seq_plan<Rows, Tile>(a, s).cost(a.Hkv) : 0;
        int64_t incl = scan(c);
        __syncthreads();   // the last round's readers of sums are done
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int64_t before = base, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        incl += before;
        if (c > 0 && incl - c <= r.start && r.start < incl) {
            found_seq = s;
            found_start = incl - c;
        }
        base += all;
        if (base > r.start) break;   // the same for the whole CTA
    }
    __syncthreads();
    r.seq = found_seq;
    r.seq_start = found_start;
    return r;
}

// A run's part of one item.
struct Piece {
    int32_t s, hk;            // sequence, key head
    int32_t row0, n_rows;     // rows of the item
    int32_t q0, kl, pos0;     // the sequence's first row of q, keys, position of its first query
    int32_t klo, khi;         // the keys that some row of the item may see
    int32_t tile0, steps;     // first tile and tiles of the piece
    int32_t tiles;            // of the item
    bool causal, starts, ends;
    int64_t at;               // where the piece begins on the line
};
struct TreePiece : Piece {
    int32_t sink_end, ns;     // keys below sink_end are seen too; tiles of them before the others'
};

// Walks a run piece by piece.
template <int Rows, int Tile, typename A>
struct Walk {
    using PieceOf = std::conditional_t<kIsTree<A>, TreePiece, Piece>;
    int64_t at, seq_start, end;
    int s;
    SeqPlan p;

    DG_DEVINL bool next(const A& a, PieceOf& z) {
        if (at >= end) return false;
        while (at >= seq_start + p.cost(a.Hkv)) {   // the next sequence that has work
            seq_start += p.cost(a.Hkv);
            p = seq_plan<Rows, Tile>(a, ++s);
        }
        const int64_t off = at - seq_start;
        const int item = off < (1LL << 31) ? (int)((uint32_t)off / (uint32_t)p.tiles) : (int)(off / p.tiles);
        const int t0 = (int)(off - (int64_t)item * p.tiles);
        z.s = s;
        z.hk = item / p.row_tiles;
        z.row0 = (item - z.hk * p.row_tiles) * Rows;
        z.n_rows = min(Rows, p.seq.ql * a.group - z.row0);
        z.q0 = p.seq.q0;
        z.kl = p.seq.kl;
        z.pos0 = p.seq.kl - p.seq.ql;
        z.causal = p.causal;
        if constexpr (kIsTree<A>) {
            z.klo = p.klo;
            z.khi = z.causal ? z.pos0 + (z.row0 + z.n_rows - 1) / a.group : z.kl - 1;
            z.sink_end = p.sink_end;
            z.ns = p.ns;
        } else {
            int unused;
            key_range(z.pos0 + z.row0 / a.group, z.kl, a.window, z.causal, z.klo, unused);
            key_range(z.pos0 + (z.row0 + z.n_rows - 1) / a.group, z.kl, a.window, z.causal, unused, z.khi);
        }
        z.tile0 = p.tile0 + t0;
        z.steps = (int)min((int64_t)(p.tiles - t0), end - at);
        z.tiles = p.tiles;
        z.starts = t0 == 0;
        z.ends = t0 + z.steps == p.tiles;
        z.at = at;
        at += z.steps;
        return true;
    }
};

// Pair: two neighbouring key heads of D / 2 as one of D.  Every query row is multiplied with the keys of
// both and takes the scores of its own; its output is its own half.  Half of the products go to waste, of which
// there are plenty; there are half as many items, and where tokens lie side by side the reads are twice as wide.
//
// Tree: an item visits the first tokens' tiles, then those from the window's first key on; steps that not every row sees
// whole are masked by the rows' ranges and, from the context's end on, by their words of the tree mask, and values
// that no row of the item sees are zeroed where they lie (what they hold is nobody's, and 0 * NaN is not 0).
template <int D, int NB, bool Pair, bool Tree>
__global__ void __launch_bounds__(SplitCfg<D, NB>::kThreads, SplitCfg<D, NB>::kCtasPerSm) k_paged_split(const SplitArgsOf<Tree> a) {
    using C = SplitCfg<D, NB>;
    using A = SplitArgsOf<Tree>;
    using PieceOf = std::conditional_t<Tree, TreePiece, Piece>;
    constexpr int Rows = 8 * NB, HD = Pair ? D / 2 : D;   // HD: of a query head
    constexpr int S = C::kStages, Tile = C::kTileKeys, kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int KB = C::kStep / 16;       // 16-key blocks of a step
    constexpr int KK = D / 16;              // 16-dimension blocks of a head
    constexpr int Chunks = D / 8;           // 16-byte chunks of a head
    constexpr int PerLoad = 32 / Chunks;    // key rows a warp's load instruction covers
    static_assert(Rows * D * 4 <= (int)C::kStage, "a warp's output fits a stage of its ring");
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kWarps][Rows];
    __shared__ float2 s_l[kWarps][Rows];
    __shared__ PieceOf s_piece[4];   // the run's current piece and the two behind it (piece k in place k % 4)
    dg::pdl_wait();
    dg::pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Run run = find_run<Rows, Tile, kWarps, A>(a);
    if (run.start >= run.end) {
        if (tid == 0) a.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    unsigned char* ring = smem + (size_t)warp * C::kRing;
    const uint32_t ring_s = dg::smem_u32(ring);
    const int page_mask = (1 << a.kv.page_shift) - 1;
    const int ch = lane % Chunks, rsub = lane / Chunks;
    int4 desc0 = make_int4(0, 0, 0, 0), desc1 = desc0;

    // Loads run ahead of the products by up to S steps, past the end of a piece into the next one.
    // Steps are counted over the run: step g lies in stage g % S, and is one cp.async group.
    uint32_t issued = 0, consumed = 0;
    struct {                       // the piece the loads are in
        const int32_t* table;
        int64_t head_at;
        int klo, khi, key0, steps, step;
        int sink_end, ns, t0;      // of a tree
        int32_t e[2 * KB];         // the pages of the next step's keys, eight at a time
    } in = {};
    // The first key of a step; of a tree `key0` is this warp's place in a tile, the tiles are counted from t0.
    auto key_of = [&](int key0, int step, int t0, int ns, int klo) -> int {
        if constexpr (Tree) {
            const int i = t0 + step;
            return (i < ns ? i : klo / Tile + i - ns) * Tile + key0;
        }
        return key0 + step * Tile;
    };
    // Whether some row may see a key from j to j + n - 1.
    auto in_sight = [&](int j, int n) -> bool { return j <= in.khi && (j + n - 1 >= in.klo || (Tree && j < in.sink_end)); };
    auto entry = [&](int half) -> int32_t {
        if (in.step >= in.steps) return -1;
        const int j = key_of(in.key0, in.step, in.t0, in.ns, in.klo) + half * 8;
        return in_sight(j, 8) ? in.table[j >> a.kv.page_shift] : -1;
    };
    auto open = [&](const PieceOf& z) {
        in.table = a.kv.page_table + (int64_t)z.s * a.kv.max_pages;
        in.head_at = Pair ? (z.hk * 2 + ch / (Chunks / 2)) * a.kv.head_stride + ch % (Chunks / 2) * 8
                          : z.hk * a.kv.head_stride + ch * 8;
        in.klo = z.klo;
        in.khi = z.khi;
        if constexpr (Tree) {
            in.key0 = warp * C::kStep;
            in.t0 = z.tile0;
            in.sink_end = z.sink_end;
            in.ns = z.ns;
        } else {
            in.key0 = z.tile0 * Tile + warp * C::kStep;
        }
        in.steps = z.steps;
        in.step = 0;
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) in.e[b] = entry(b);
    };
    auto issue = [&]() {   // one step's keys and values into its stage; then the next step's pages
        const int j0 = key_of(in.key0, in.step, in.t0, in.ns, in.klo);
        const uint32_t dst = ring_s + (issued % S) * C::kStage;
#pragma unroll
        for (int half = 0; half < 2 * KB; ++half) {
            const int32_t page = in.e[half];
            const bool good = page >= 0 && page < a.kv.n_pages;
            const int jh = j0 + half * 8;
            if (!good && in_sight(jh, 8) && lane == 0) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
            const int64_t off = good ? page * a.kv.page_stride + (int64_t)((jh & page_mask) + rsub) * a.kv.slot_stride + in.head_at : 0;
            const uint16_t* ks = a.kv.k + off;
            const uint16_t* vs = a.kv.v + off;
            const int64_t hop = good ? PerLoad * a.kv.slot_stride : 0;
#pragma unroll
            for (int i = 0; i < 8 / PerLoad; ++i) {
                const int row = half * 8 + i * PerLoad + rsub;
                const bool ok = good && in_sight(j0 + row, 1);
                const uint32_t d = dst + (uint32_t)row * (D * 2) + (uint32_t)((ch ^ (row & 7)) * 16);
                cp_async16(d, ks, ok);
                cp_async16(d + C::kHalf, vs, ok);
                ks += hop;
                vs += hop;
            }
        }
        cp_async_commit();
        ++issued;
        ++in.step;
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) in.e[b] = entry(b);
    };

    Walk<Rows, Tile, A> walk{run.start, run.seq_start, run.end, run.seq, seq_plan<Rows, Tile>(a, run.seq)};
    int place = 0;                 // of the current piece in s_piece
    bool more = false, more2 = false;   // there is a next one, and one behind it
    bool ahead = false;                 // the loads are in the next one
    // Fills the ring up to `limit` steps ahead of the products.
    auto fill = [&](uint32_t limit) {
        while (issued - consumed < limit) {
            if (in.step < in.steps) {
                issue();
            } else if (more && !ahead) {
                open(s_piece[(place + 1) & 3]);
                ahead = true;
            } else {
                break;
            }
        }
    };
    {
        PieceOf z;
        walk.next(a, z);
        open(z);
        fill(S - 1);   // on their way before the next piece is worked out
        if (tid == 0) s_piece[0] = z;
        more = walk.next(a, z);
        if (more && tid == 0) s_piece[1] = z;
    }
    __syncthreads();
    // Q^T as the second operand: lane holds column lane / 4, dimensions 2 (lane % 4) + {0, 1} (+ 8); in shared
    // memory two pieces' worth, [piece % 2][KK][NB][lane] (a piece's is seen after the meeting before it)
    uint32_t qf[C::kSharedQ ? 1 : NB][C::kSharedQ ? 1 : HD / 16][2];
    uint2* const q_shared = reinterpret_cast<uint2*>(smem + C::kOffQ);
    auto load_q = [&](const PieceOf& z, int p) {
        if constexpr (C::kSharedQ) {
            for (int i = tid; i < KK * NB * 32; i += kThreads) {
                const int l = i & 31, nb = (i >> 5) % NB, kk = (i >> 5) / NB;
                const bool ok = nb * 8 + l / 4 < z.n_rows;
                const int r = z.row0 + nb * 8 + (ok ? l / 4 : 0);
                const int qi = r / a.group;
                const uint16_t* src = a.q + ((int64_t)(z.q0 + qi) * a.Hq + z.hk * a.group + (r - qi * a.group)) * HD + (l & 3) * 2 + kk * 16;
                q_shared[(p & 1) * (KK * NB * 32) + i] =
                    ok ? make_uint2(*reinterpret_cast<const uint32_t*>(src), *reinterpret_cast<const uint32_t*>(src + 8))
                       : make_uint2(0u, 0u);
            }
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const bool ok = nb * 8 + lane / 4 < z.n_rows;
                const int r = z.row0 + nb * 8 + (ok ? lane / 4 : 0);
                const int qi = r / a.group;
                const uint16_t* src = a.q + ((int64_t)(z.q0 + qi) * a.Hq + z.hk * a.group + (r - qi * a.group)) * HD + (lane & 3) * 2;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    qf[nb][kk][0] = ok ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
                    qf[nb][kk][1] = ok ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
                }
            }
        }
    };
    load_q(s_piece[0], 0);
    fill(S - 1);
    if constexpr (C::kSharedQ) __syncthreads();

    const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8, k_col = (lane >> 4) & 1;
    const int v_row = (lane & 7) + ((lane >> 4) & 1) * 8, v_col = (lane >> 3) & 1;
    while (true) {
        // the ranges of this lane's rows of S^T (columns 2 (lane % 4) + {0, 1}), and the narrowest: it
        // decides whether a step needs its mask
        const int klo = s_piece[place].klo, khi = s_piece[place].khi, steps = s_piece[place].steps;
        const int key0 = Tree ? warp * C::kStep : s_piece[place].tile0 * Tile + warp * C::kStep;
        int rlo[NB][2], rhi[NB][2], all_lo, all_hi;
        int rq[Tree ? NB : 1][2];    // of a tree: the rows' queries,
        int sink_end = 0, ns = 0, t0 = 0, ctx = 0;
        bool upper[NB][2];   // of the pair's second head
        {
            const PieceOf& z = s_piece[place];
            int unused;
            if constexpr (Tree) {
                sink_end = z.sink_end;
                ns = z.ns;
                t0 = z.tile0;
                ctx = z.pos0;
                all_lo = 0;
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = min(nb * 8 + (lane & 3) * 2 + e, z.n_rows - 1), qi = (z.row0 + r) / a.group;
                    if constexpr (Tree) {
                        rq[nb][e] = qi;
                        int pos = z.pos0 + qi;
                        if (!z.causal && a.window >= 0) pos = max(a.positions[(int64_t)z.q0 + qi], z.pos0);
                        rlo[nb][e] = a.window < 0 ? 0 : (int)max((int64_t)0, (int64_t)pos - a.window);
                        rhi[nb][e] = z.causal ? pos : z.pos0 - 1;   // (beyond it by the mask)
                        all_lo = max(all_lo, rlo[nb][e]);
                    } else {
                        key_range(z.pos0 + qi, z.kl, a.window, z.causal, rlo[nb][e], rhi[nb][e]);
                    }
                    if constexpr (Pair) upper[nb][e] = z.row0 + r - qi * a.group >= a.group / 2;
                }
            if constexpr (Tree) {
                all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, 1));
                all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, 2));
                all_hi = z.causal ? z.pos0 + z.row0 / a.group : z.pos0 - 1;
            } else {
                key_range(z.pos0 + (z.row0 + z.n_rows - 1) / a.group, z.kl, a.window, z.causal, all_lo, unused);
                key_range(z.pos0 + z.row0 / a.group, z.kl, a.window, z.causal, unused, all_hi);
            }
        }
        float acc[KK][NB][4];
#pragma unroll
        for (int mt = 0; mt < KK; ++mt)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nb][e] = 0.f;
        // running maximum; sum of the weights (for lse) and of the weights as the product with V has them,
        // rounded to bf16, which the output is divided by: a row that one key decides is then exact
        float m[NB][2], l[NB][2], lr[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = lr[nb][0] = lr[nb][1] = 0.f;

        {   // the piece behind the next one, while loads are on their way (others see it after the meeting)
            PieceOf z;
            more2 = more && walk.next(a, z);
            if (more2 && tid == 0) s_piece[(place + 2) & 3] = z;
        }
        for (int step = 0; step < steps; ++step) {
            if (issued - consumed == (uint32_t)(S - 1))
                cp_async_wait<S - 2>();
            else
                cp_async_wait<0>();
            __syncwarp();   // every lane's part has landed, and the stage refilled now has been read
            fill(S);
            const uint32_t st = ring_s + (consumed % S) * C::kStage;
            ++consumed;
            const int j0 = key_of(key0, step, t0, ns, klo);
            if (j0 > khi || (j0 + C::kStep - 1 < klo && (!Tree || j0 >= sink_end))) continue;   // no key of the item
            float x[KB][NB][4];   // S^T: [key lane / 4 (+ 8 for 2, 3)][row 2 (lane % 4) + (0, 1)]
            {
                float c[KB][NB][2][4];   // even and odd 16-dimension blocks (a pair: its heads) apart: two chains a block of keys
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[kb][nb][0][e] = c[kb][nb][1][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        uint32_t kf[4];
                        ldmatrix4(kf, st + (uint32_t)(kb * 16 + k_row) * (D * 2) + (uint32_t)(((kk * 2 + k_col) ^ (lane & 7)) * 16));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            if constexpr (C::kSharedQ) {
                                const uint2 q = q_shared[((place & 1) * KK + kk) * (NB * 32) + nb * 32 + lane];
                                mma(c[kb][nb][kk & 1], kf, q.x, q.y);
                            } else {
                                constexpr int QK = HD / 16;
                                mma(c[kb][nb][Pair ? kk / QK : kk & 1], kf, qf[nb][kk % QK][0], qf[nb][kk % QK][1]);
                            }
                        }
                    }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[kb][nb][e] = (Pair ? (upper[nb][e & 1] ? c[kb][nb][1][e] : c[kb][nb][0][e])
                                                 : c[kb][nb][0][e] + c[kb][nb][1][e]) * a.scale_log2;
            }
            if constexpr (Tree) {
                const int j1 = j0 + C::kStep - 1;
                if (j1 > all_hi || (j0 < all_lo && j1 >= a.sinks)) {
                    const PieceOf& z = s_piece[place];
                    const uint32_t* const rows_mask = a.mask + (int64_t)z.q0 * a.mask_words;
                    bool dead = false;   // a key that no row sees
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int j = j0 + kb * 16 + lane / 4 + half * 8;
                            const bool node = !z.causal && j >= ctx && j < z.kl;
                            bool mine = false;
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    bool seen = j <= rhi[nb][e] && (j >= rlo[nb][e] || j < a.sinks);
                                    if (node)
                                        seen = rows_mask[(int64_t)rq[nb][e] * a.mask_words + ((j - ctx) >> 5)] >> ((j - ctx) & 31) & 1u;
                                    if (!seen) x[kb][nb][half * 2 + e] = -INFINITY;
                                    mine = mine || seen;
                                }
                            if (!(__ballot_sync(0xffffffffu, mine) >> (lane & 28) & 15u)) {
                                dead = true;
                                unsigned char* v = ring + (st - ring_s) + C::kHalf + (kb * 16 + lane / 4 + half * 8) * (D * 2);
                                for (int c = lane & 3; c < Chunks; c += 4) reinterpret_cast<uint4*>(v)[c] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    if (__any_sync(0xffffffffu, dead)) __syncwarp();
                }
            } else if (j0 < all_lo || j0 + C::kStep - 1 > all_hi) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = j0 + kb * 16 + lane / 4 + (e & 2) * 4;
                            if (j < rlo[nb][e & 1] || j > rhi[nb][e & 1]) x[kb][nb][e] = -INFINITY;
                        }
            }
            float top[NB][2];   // this lane's largest score of each of its rows
            bool grown = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nb][e] = fmaxf(x[0][nb][e], x[0][nb][e + 2]);
#pragma unroll
                    for (int kb = 1; kb < KB; ++kb) top[nb][e] = fmaxf(top[nb][e], fmaxf(x[kb][nb][e], x[kb][nb][e + 2]));
                    grown = grown || top[nb][e] > m[nb][e] + kRescaleAbove;
                }
            if (__any_sync(0xffffffffu, grown)) {   // some row's maximum moves: new references, old sums rescaled
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = top[nb][e];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        mx = fmaxf(mx, m[nb][e]);
                        const float f = mx == -INFINITY ? 1.f : ex2(m[nb][e] - mx);
                        l[nb][e] *= f;
                        lr[nb][e] *= f;
#pragma unroll
                        for (int mt = 0; mt < KK; ++mt) {
                            acc[mt][nb][e] *= f;
                            acc[mt][nb][e + 2] *= f;
                        }
                        m[nb][e] = mx;
                    }
            }
            uint32_t pf[KB][NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float r0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0], r1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const float p0 = ex2(x[kb][nb][0] - r0), p1 = ex2(x[kb][nb][1] - r1);
                    const float p2 = ex2(x[kb][nb][2] - r0), p3 = ex2(x[kb][nb][3] - r1);
                    l[nb][0] += p0 + p2;
                    l[nb][1] += p1 + p3;
                    const uint32_t w0 = pack_bf16x2(p0, p1), w1 = pack_bf16x2(p2, p3);
                    lr[nb][0] += __uint_as_float(w0 << 16) + __uint_as_float(w1 << 16);
                    lr[nb][1] += __uint_as_float(w0 & 0xffff0000u) + __uint_as_float(w1 & 0xffff0000u);
                    pf[kb][nb][0] = transpose8x8(w0);
                    pf[kb][nb][1] = transpose8x8(w1);
                }
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int mt = 0; mt < KK; ++mt) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, st + C::kHalf + (uint32_t)(kb * 16 + v_row) * (D * 2) + (uint32_t)(((mt * 2 + v_col) ^ (lane & 7)) * 16));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma(acc[mt][nb], vf, pf[kb][nb][0], pf[kb][nb][1]);
                }
        }

        // The warps meet: each leaves its unnormalised output in the stage it read last (the others are
        // already being filled for the next piece), its rows' dimensions turned so that the lanes' banks
        // differ, and its statistics.
        const uint32_t met = ((consumed - 1u) % S) * C::kStage;
        __syncwarp();
        float* mo = reinterpret_cast<float*>(ring + met);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nb][e], sum_r = lr[nb][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    sum_r += __shfl_xor_sync(0xffffffffu, sum_r, o);
                }
                if (lane < 4) {
                    s_m[warp][nb * 8 + lane * 2 + e] = m[nb][e];
                    s_l[warp][nb * 8 + lane * 2 + e] = make_float2(sum, sum_r);
                }
                const int r = nb * 8 + (lane & 3) * 2 + e, turn = (lane & 3) << 3;
#pragma unroll
                for (int mt = 0; mt < KK; ++mt) {
                    mo[r * D + ((mt * 16 + lane / 4) ^ turn)] = acc[mt][nb][e];
                    mo[r * D + ((mt * 16 + 8 + lane / 4) ^ turn)] = acc[mt][nb][e + 2];
                }
            }
        }
        if (more) load_q(s_piece[(place + 1) & 3], place + 1);   // on its way while the warps meet
        __syncthreads();
        const PieceOf z = s_piece[place];
        const int64_t slot = (int64_t)blockIdx.x * 2 + (z.starts ? 1 : 0);
        for (int i = tid; i < z.n_rows * (HD / 4); i += kThreads) {
            const int r = i / (HD / 4), d = (i - r * (HD / 4)) * 4;
            const int rr = z.row0 + r, qi = rr / a.group, head = rr - qi * a.group;
            const int col = Pair && head >= a.group / 2 ? HD + d : d;   // of the rows in shared memory
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
            float L = 0.f, Lr = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - M);
                L += s_l[w][r].x * f;
                Lr += s_l[w][r].y * f;
                const float4 v = *reinterpret_cast<const float4*>(smem + (size_t)w * C::kRing + met +
                                                                  ((size_t)r * D + (col ^ (((r >> 1) & 3) << 3))) * 4);
                o.x += v.x * f;
                o.y += v.y * f;
                o.z += v.z * f;
                o.w += v.w * f;
            }
            if (z.starts && z.ends) {
                const int64_t out = (int64_t)(z.q0 + qi) * a.Hq + z.hk * a.group + head;
                const float inv = Lr > 0.f ? 1.f / Lr : 0.f;
                *reinterpret_cast<uint2*>(a.o + out * HD + d) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (d == 0 && a.lse) a.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;  // (a NaN stays one)
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot * Rows + r) * HD + d) = o;
                if (d == 0) a.part_ml[slot * Rows + r] = make_float4(M, L, Lr, 0.f);
            }
        }
        if (z.starts && !z.ends) {
            const int64_t last = (z.at + z.tiles - 1) / run.per_cta;   // the CTA that has the item's last tile
            desc0 = make_int4((int)(last - blockIdx.x), z.n_rows, z.q0, z.hk);
            desc1 = make_int4(z.row0, 0, 0, 0);
        }
        if (!more) break;
        __syncthreads();   // the meeting buffers are free
        // on to the next piece; the loads are in it already, or begin with it
        place = (place + 1) & 3;
        if (!ahead) open(s_piece[place]);
        ahead = false;
        more = more2;
        fill(S - 1);
    }
    if (tid == 0) {
        a.desc[2 * blockIdx.x] = desc0;
        a.desc[2 * blockIdx.x + 1] = desc1;
    }
}

// Joins an item's pieces: the last one of CTA c (slot 1) and the first ones (slot 0) of the CTAs
// that follow it.  blockIdx.x = c, blockIdx.y = 64 of the dimensions; most blocks find nothing to join.
// A thread owns four dimensions of a row for every kGroups-th piece (a long context of one head is joined
// from dozens: reading them one after another took most of the kernel); the groups add up in
// shared memory in a fixed order.  The first pieces are on their way while the weights are worked out.
template <int D, int NB, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const SplitArgs a) {
    constexpr int Rows = 8 * NB;
    constexpr int kPlaces = Rows * 16;               // float4s of 64 dimensions of the rows
    constexpr int kGroups = kJoinThreads / kPlaces;  // 4, 2 or 1
    constexpr int kEarly = 4;                        // pieces a thread asks for before it knows their weights
    __shared__ float w[kMaxCtas][Rows];              // the pieces' maxima, then their weights
    __shared__ float s_l[Rows], s_lr[Rows], s_m[Rows];
    __shared__ float4 part[kGroups > 1 ? kGroups - 1 : 1][kPlaces];
    dg::pdl_wait();
    dg::pdl_release();
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int4 desc0 = a.desc[2 * c], desc1 = a.desc[2 * c + 1];
    if (desc0.x == 0) return;
    const int n = desc0.x + 1, n_rows = desc0.y, q0 = desc0.z, hk = desc0.w, row0 = desc1.x;
    auto slot = [&](int i) -> int64_t { return i == 0 ? (int64_t)c * 2 + 1 : (int64_t)(c + i) * 2; };
    const int group = tid / kPlaces, place = tid - group * kPlaces;
    const int r = place / 16, d = (int)blockIdx.y * 64 + (place & 15) * 4;
    const bool mine = r < n_rows;
    auto piece = [&](int k) { return *reinterpret_cast<const float4*>(a.part_o + (slot(k) * Rows + r) * D + d); };
    float4 early[kEarly];
#pragma unroll
    for (int e = 0; e < kEarly; ++e)
        if (mine && group + e * kGroups < n) early[e] = piece(group + e * kGroups);
    // weights: a row a warp
    for (int q = warp; q < n_rows; q += kJoinThreads / 32) {
        float M = -INFINITY;
        for (int i = lane; i < n; i += 32) {
            const float v = a.part_ml[slot(i) * Rows + q].x;
            w[i][q] = v;
            M = fmaxf(M, v);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f, Lr = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float m = w[i][q], f = m == -INFINITY ? 0.f : ex2(m - M);
            const float4 ml = a.part_ml[slot(i) * Rows + q];
            w[i][q] = f;
            L += ml.y * f;
            Lr += ml.z * f;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, o);
            Lr += __shfl_xor_sync(0xffffffffu, Lr, o);
        }
        if (lane == 0) {
            s_l[q] = L;
            s_lr[q] = Lr;
            s_m[q] = M;
        }
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v, float f) {
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
    };
    if (mine) {
#pragma unroll
        for (int e = 0; e < kEarly; ++e)
            if (group + e * kGroups < n) add(early[e], w[group + e * kGroups][r]);
#pragma unroll 8
        for (int k = group + kEarly * kGroups; k < n; k += kGroups) add(piece(k), w[k][r]);
    }
    if (group > 0) part[group - 1][place] = o;
    __syncthreads();
    if (group > 0 || !mine) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) add(part[g - 1][place], 1.f);
    const float L = s_l[r], inv = s_lr[r] > 0.f ? 1.f / s_lr[r] : 0.f;
    const int rr = row0 + r, qi = rr / a.group;
    const int64_t out = (int64_t)(q0 + qi) * a.Hq + hk * a.group + (rr - qi * a.group);
    *reinterpret_cast<uint2*>(a.o + out * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (d == 0 && a.lse) a.lse[out] = L == 0.f ? -INFINITY : (s_m[r] + log2f(L)) * kLn2;
}

// Rows of an item: 8 when the call's queries and a group fit them, else 16.
int item_rows(int32_t max_q_len, int32_t group) { return (int64_t)max_q_len * group <= 8 ? 8 : 16; }

// Whether two key heads of 64 go as one of 128: when the rows of both fit eight.  250 windows of 1000 keys, 8 / 8
// heads, 97.5 us head by head and 84.9 in pairs; 64 requests over 8k keys 130 / 113 (tokens side by side), 117 / 111
// (heads side by side); 200 over 300 keys, 16 / 8 heads, 39.7 / 28.0; 256 over 60 keys 25.2 / 16.8; one over 1k keys
// 7.9 / 7.3.  Not with 16 rows (32 requests of 8 queries over 3k keys 29.3 / 30.2, 26 of 8 over 54 keys 6.8 / 7.4,
// though 24.5 / 21.0 for 200 with 8 query heads a key head over 300), nor heads of 128 as 256 (64 over 8k keys 223 /
// 221, but 256 over 60 keys 27.6 / 28.4, one over 1k 7.9 / 8.6).
bool in_pairs(int32_t max_q_len, int32_t group, int32_t Hkv, int32_t D) {
    return D == 64 && Hkv % 2 == 0 && (int64_t)max_q_len * group * 2 <= 8;
}

size_t split_bytes(int rows, int32_t D) {
    return (size_t)kMaxCtas * 32 + (size_t)kMaxCtas * 2 * rows * ((size_t)D + 4) * 4;
}

template <int D, int NB, bool Pair = false, typename A = SplitArgs>
dg_status launch_split(const A& a, cudaStream_t stream) {
    constexpr int HD = Pair ? D / 2 : D;
    using C = SplitCfg<D, NB>;
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    // the attribute once a device: 0.4 us of a call that takes the host 4
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DG_ERR_CUDA;
    if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        if (cudaFuncSetAttribute(k_paged_split<D, NB, Pair, kIsTree<A>>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) !=
            cudaSuccess)
            return DG_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)std::min(sms * C::kCtasPerSm, kMaxCtas);
    cudaError_t e = dghost::launch_pdl(k_paged_split<D, NB, Pair, kIsTree<A>>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, a);
    dghost::count_launch();
    if (e != cudaSuccess) return DG_ERR_CUDA;
    // Many items are joined from a few pieces each, if at all, and half the threads a block come and go sooner;
    // few have many pieces.  42 items of 2 keys: 6.6 us with 512, 6.1 with 256; 256 of 5 drafts over 4k keys 65.1 /
    // 64.0; 4 of 128k keys 86.9 / 87.5, 8 of 1k 7.1 / 7.4.
    if (8 * (int64_t)a.n_seq * a.Hkv >= grid)
        e = dghost::launch_pdl(k_paged_join<HD, NB, 256>, dim3(grid, HD / 64), dim3(256), 0, stream, static_cast<const SplitArgs&>(a));
    else
        e = dghost::launch_pdl(k_paged_join<HD, NB, 512>, dim3(grid, HD / 64), dim3(512), 0, stream, static_cast<const SplitArgs&>(a));
    dghost::count_launch();
    return dghost::cuda_status(e);
}

}  // namespace
