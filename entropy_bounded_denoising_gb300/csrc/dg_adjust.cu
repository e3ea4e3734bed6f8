// dg_adjust.cu -- a request's edits of its logits before the step reads them: penalties for the
// tokens of its history, a bias per token, a grammar's mask.
//
// Every edit is a function of (canvas, token) but the mask, which is one of (position, token).  So a
// block owns one canvas's slice of the vocabulary for a group of positions, a thread 16 bytes of it:
// the block counts the slice's tokens in the canvas's lists once (shared memory), each thread turns
// its tokens' counts and biases into one fp32 addend a token that stays in registers, and the rows
// stream by with one mask byte a vector.  Nothing is sorted, gathered or kept between launches, and
// the lists are read from L2 once a block.
// Bound by memory: in place only vectors with an edited or excluded token are touched, and a vector that is
// excluded whole is written without being read.  8 canvases of 256 positions, fp32, 152k tokens, half of them
// excluded: 282 us; nearly every vector has an allowed token, so 0.95 GB are read and 0.88 written, 270 us
// at a copy's rate.  A grammar that leaves 1 % of 262k bf16 tokens, in place: 222 us for 1.01 GB written and
// 0.33 read (a vector with an allowed token is read, and 64 bytes come with it; writing only the excluded
// tokens of such vectors without reading them took 420).  One canvas over 32k tokens: 9.6 us, of
// which a copy of the logits takes 6.6 and the mask alone 7.5; the rest is the wait for the lists.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dg_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;
// Rows in flight a thread: the registers of the lists' addends hold four rows more when a call gives no lists.
// Masks alone, in place, 8 canvases of 256, four / six / eight rows: bf16, 1 % of 250k tokens left, 278 / 261 / 239 us,
// of 262k 231 / 220 / 222; fp32, half of 131k left, 322 / 320 / 326.
constexpr int unroll_of(bool lists) { return lists ? 4 : 8; }
constexpr int kMaxRows = 64; // rows of a block, at most
constexpr int kEarly = 2;    // entries of each list that a thread reads before anything else
constexpr int kAgain = 8;    // entries of a bias list with repeated tokens that a lane reads at a time

struct AdjustArgs {
    const unsigned char* x;
    unsigned char* out;
    int64_t ld_bytes, ld_out_bytes;
    int32_t L, V, rows;   // rows: positions of a block
    const dg_canvas_params* params;
    const int32_t *history, *cu_history;
    const dg_penalties* penalties;
    const int32_t* bias_tokens;
    const float* bias_values;
    const int32_t* cu_bias;
    const uint32_t* masks;
    const int32_t* mask_index;
    int64_t total_history, total_bias, mask_stride;
    int32_t n_masks;
    unsigned* status;
};

DG_DEVINL uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}

// 16 bytes, fetching no more than the 64 around them: a mask that leaves few tokens has few vectors read, and 128
// around each were half of the row (1 % of 262k bf16 tokens left, in place: 249 us without the hint, 222 with it;
// where most are read it makes no difference).  Not volatile: a row is read before its own store and after no
// other's.
DG_DEVINL uint4 load16(const unsigned char* p) {
    uint4 v;
    asm("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The penalties and biases of a vector's edited tokens: one fma each, by 1 / repetition or repetition
// (1 for a token without a count) and the token's addend.  `any`: the places of a vector that some lane of
// the warp has edited; lists are short beside the vocabulary, so most places are skipped by all.
template <int Bytes>
DG_DEVINL void edit(uint4& y, uint32_t any, uint32_t edited, uint32_t penalised, float down, float up, const float (&add)[16 / Bytes]) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int e = 0; e < 16 / Bytes; ++e) {
        if (!(any >> e & 1)) continue;
        const int i = Bytes == 2 ? e / 2 : e;
        const bool high = Bytes == 2 && (e & 1);
        const float v = __uint_as_float(Bytes == 4 ? w[i] : high ? w[i] & 0xffff0000u : w[i] << 16);
        const float f = !(penalised >> e & 1) ? 1.f : v > 0.f ? down : up;
        const float z = fmaf(v, f, add[e]);
        const uint32_t p = Bytes == 4 ? __float_as_uint(z) : pack_bf16x2(z, z);
        const uint32_t bits = Bytes == 4 ? p : high ? (w[i] & 0xffffu) | (p & 0xffff0000u) : (w[i] & 0xffff0000u) | (p & 0xffffu);
        if (edited >> e & 1) w[i] = bits;
    }
}

// -inf for the tokens whose bit of `keep` is clear.
template <int Bytes>
DG_DEVINL void exclude(uint4& y, uint32_t keep, const uint2* expand) {
    if (Bytes == 2) {
        const uint2 a = expand[keep & 15u], b = expand[keep >> 4];
        y.x = (y.x & a.x) | (0xff80ff80u & ~a.x);
        y.y = (y.y & a.y) | (0xff80ff80u & ~a.y);
        y.z = (y.z & b.x) | (0xff80ff80u & ~b.x);
        y.w = (y.w & b.y) | (0xff80ff80u & ~b.y);
    } else {
        y.x = keep & 1u ? y.x : 0xff800000u;
        y.y = keep & 2u ? y.y : 0xff800000u;
        y.z = keep & 4u ? y.z : 0xff800000u;
        y.w = keep & 8u ? y.w : 0xff800000u;
    }
}

// A vector's first n tokens (all but in a row's last vector: nothing past column V is written).
template <int Bytes, bool Lists>
DG_DEVINL void store(unsigned char* at, const uint4& y, int n) {
    constexpr int PerVec = 16 / Bytes;
    if (n == PerVec) {
        // (a plain store of fp32 without lists was compiled into four of 4 bytes: 422 us for 204; with lists it is
        // the quicker one, 9.2 us for 9.7 on one canvas)
        if constexpr (Lists)
            *reinterpret_cast<uint4*>(at) = y;
        else
            __stcg(reinterpret_cast<uint4*>(at), y);
        return;
    }
#pragma unroll
    for (int e = 0; e < PerVec; ++e) {
        if (e >= n) break;
        const uint32_t w = reinterpret_cast<const uint32_t*>(&y)[Bytes == 2 ? e / 2 : e];
        if (Bytes == 2)
            reinterpret_cast<uint16_t*>(at)[e] = (uint16_t)(e & 1 ? w >> 16 : w);
        else
            reinterpret_cast<uint32_t*>(at)[e] = w;
    }
}

// Adds up the biases of the warp's own tokens that have more than one, in list order: the warp reads the list,
// 256 entries at a time, and takes the entries of such tokens one after another.  (A thread that looked for its
// tokens' entries by itself took as many dependent reads as lay between them: 4000 tokens given twice 1170 us, this
// way 41.)  A call, so that its registers are not the kernel's.
template <int PerVec>
__device__ __noinline__ void add_repeats(const int32_t* tokens, const float* values, int b0, int b1, int slice0, int end,
                                         const int32_t* n_bias, float* sums) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int own0 = (tid - lane) * PerVec, own1 = min(own0 + 32 * PerVec, end);   // the warp's tokens, of the slice
    for (int64_t j0 = b0; j0 < b1; j0 += 32 * kAgain) {
        int64_t token[kAgain];
        float value[kAgain];
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
            const int64_t j = j0 + u * 32 + lane;
            token[u] = j < b1 ? (int64_t)tokens[j] - slice0 : -1;
            value[u] = j < b1 ? values[j] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
            const bool own = token[u] >= own0 && token[u] < own1;
            for (uint32_t hits = __ballot_sync(0xffffffffu, own && n_bias[own ? token[u] : 0] > 1); hits; hits &= hits - 1) {
                const int t = __shfl_sync(0xffffffffu, (int)token[u], __ffs(hits) - 1);
                const float v = __shfl_sync(0xffffffffu, value[u], __ffs(hits) - 1);
                if (t / PerVec == tid) sums[t] += v;
            }
        }
    }
}

// Bytes: 2 (bf16) or 4 (fp32) a logit; PerVec tokens in 16 bytes.  Lists: the call gives a history or biases.
template <int Bytes, bool Lists>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_adjust(const AdjustArgs a) {
    constexpr int kUnroll = unroll_of(Lists);
    constexpr int PerVec = 16 / Bytes;
    constexpr int kSlice = kThreads * PerVec;   // tokens of a block
    constexpr int kCounts = Lists ? kSlice : 4;
    __shared__ __align__(16) int32_t n_hist[kCounts];       // occurrences in the history
    __shared__ __align__(16) int32_t n_bias[kCounts];       // entries in the bias list
    __shared__ float one_bias[kCounts];                     // the value of the only one, else their sum
    __shared__ int32_t row_mask[kMaxRows];
    __shared__ uint2 expand[16];
    constexpr uint32_t kNegInf = Bytes == 2 ? 0xff80ff80u : 0xff800000u;
    dg::pdl_wait();
    dg::pdl_release();
    const int tid = threadIdx.x;
    const int64_t c = blockIdx.z;
    const int slice0 = (int)blockIdx.x * kSlice;
    const int v0 = slice0 + tid * PerVec;
    const int r0 = (int)blockIdx.y * a.rows, rows = min(a.L - r0, a.rows);
    const bool reports = blockIdx.x == 0 && blockIdx.y == 0 && tid == 0;

    // everything that depends on nothing else is read at once: the canvas's flag, its lists' bounds and
    // penalties, the rows' masks
    const uint32_t flags = a.params[c].flags;
    int h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    dg_penalties pen = {1.f, 0.f, 0.f};
    if (Lists && a.history) {
        h0 = a.cu_history[c];
        h1 = a.cu_history[c + 1];
        pen = a.penalties[c];
    }
    if (Lists && a.bias_tokens) {
        b0 = a.cu_bias[c];
        b1 = a.cu_bias[c + 1];
    }
    int m = -1;   // kMaxRows <= kThreads: a thread a row; -1 = none
    if (a.masks && tid < rows) m = a.mask_index[c * a.L + r0 + tid];
    if (!(flags & DG_ACTIVE)) return;
    const bool sound = h0 >= 0 && h1 >= h0 && h1 <= a.total_history && b0 >= 0 && b1 >= b0 && b1 <= a.total_bias &&
                       pen.repetition >= 0x1p-126f && pen.repetition <= 0x1p126f &&   // its reciprocal is a normal number
                       isfinite(pen.frequency) && isfinite(pen.presence);
    if (!sound) {
        if (reports) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        return;
    }
    if (m < -1 || m >= a.n_masks) {
        if (blockIdx.x == 0) dg::raise_status(a.status, DG_DEV_BAD_PARAM);
        m = -1;
    }
    if (tid < kMaxRows) row_mask[tid] = m;
    // what keeps an excluded token's logit: words of ones where four tokens' bits are set (bf16 pairs)
    if (Bytes == 2 && tid < 16)
        expand[tid] = make_uint2(((tid & 1) ? 0xffffu : 0u) | ((tid & 2) ? 0xffff0000u : 0u),
                                 ((tid & 4) ? 0xffffu : 0u) | ((tid & 8) ? 0xffff0000u : 0u));
    const bool listed = Lists && (h1 > h0 || b1 > b0);
    // a thread's first entries of the lists are on their way meanwhile
    int32_t early_h[kEarly], early_b[kEarly];
    float early_v[kEarly];
#pragma unroll
    for (int k = 0; Lists && k < kEarly; ++k) {
        const int64_t i = (int64_t)h0 + tid + k * kThreads, j = (int64_t)b0 + tid + k * kThreads;
        early_h[k] = i < h1 ? a.history[i] : -1;
        early_b[k] = j < b1 ? a.bias_tokens[j] : -1;
        early_v[k] = j < b1 ? a.bias_values[j] : 0.f;
    }
    if (listed) {
#pragma unroll
        for (int e = 0; e < PerVec / 4; ++e) {
            reinterpret_cast<int4*>(n_hist)[e * kThreads + tid] = make_int4(0, 0, 0, 0);
            if (b1 > b0) reinterpret_cast<int4*>(n_bias)[e * kThreads + tid] = make_int4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    // the first rows' masks and data are on their way while the lists are counted
    const bool in_place = a.out == a.x;
    const int n_mine = max(0, min(PerVec, a.V - v0));          // tokens of the vector inside the vocabulary
    const uint32_t mine = (1u << n_mine) - 1u;
    const unsigned char* mask_at = reinterpret_cast<const unsigned char*>(a.masks) + (v0 >> 3);
    const int64_t mask_pitch = a.mask_stride * 4;
    const unsigned char* src = a.x + (c * a.L + r0) * a.ld_bytes + (int64_t)v0 * Bytes;
    unsigned char* dst = a.out + (c * a.L + r0) * a.ld_out_bytes + (int64_t)v0 * Bytes;
    asm volatile("" : "+l"(src));   // no read of a row moves up past pdl_wait
    uint32_t keep[kUnroll], next[kUnroll];   // allowed tokens of the vector, for kUnroll rows
    uint4 x[kUnroll];
    auto masks_of = [&](int r) {             // row_mask is -1 past the last row
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int row = r + u < kMaxRows ? row_mask[r + u] : -1;
            next[u] = row >= 0 && n_mine > 0 ? (uint32_t)mask_at[row * mask_pitch] : 0xffu;
        }
    };
    auto load = [&](int r, bool only_mixed) {   // a vector that goes whole, or stays whole in place, is not read
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            keep[u] = (Bytes == 4 ? next[u] >> (v0 & 4) : next[u]) & mine;
            x[u] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
            if (r + u < rows && keep[u] != 0 && !(only_mixed && keep[u] == mine))
                x[u] = load16(src + u * a.ld_bytes);
        }
    };
    const int end = min(kSlice, a.V - slice0);
    auto count = [&](int32_t token) {
        const int64_t t = (int64_t)token - slice0;
        if (t >= 0 && t < end) atomicAdd(&n_hist[t], 1);
    };
    auto note = [&](int32_t token, float value) {
        const int64_t t = (int64_t)token - slice0;
        if (t < 0 || t >= end) return;
        atomicAdd(&n_bias[t], 1);
        one_bias[t] = value;
    };
    masks_of(0);
    if (listed) {
#pragma unroll
        for (int k = 0; k < kEarly; ++k) {
            count(early_h[k]);
            note(early_b[k], early_v[k]);
        }
    }
    load(0, in_place && !listed);
    if (listed) {
#pragma unroll 4
        for (int64_t i = (int64_t)h0 + kEarly * kThreads + tid; i < h1; i += kThreads) count(a.history[i]);
#pragma unroll 4
        for (int64_t i = (int64_t)b0 + kEarly * kThreads + tid; i < b1; i += kThreads)
            note(a.bias_tokens[i], a.bias_values[i]);
    }
    float add[PerVec];
    uint32_t penalised = 0, edited = 0;   // tokens with a count / with a count or a bias
#pragma unroll
    for (int e = 0; e < PerVec; ++e) add[e] = 0.f;
    if (listed) {
        __syncthreads();
        int nh[PerVec], nb[PerVec];
#pragma unroll
        for (int e = 0; e < PerVec; e += 4) {
            *reinterpret_cast<int4*>(&nh[e]) = *reinterpret_cast<const int4*>(&n_hist[tid * PerVec + e]);
            *reinterpret_cast<int4*>(&nb[e]) =
                b1 > b0 ? *reinterpret_cast<const int4*>(&n_bias[tid * PerVec + e]) : make_int4(0, 0, 0, 0);
        }
        bool several = false;   // some token of the thread has more than one bias
#pragma unroll
        for (int e = 0; e < PerVec; ++e) several |= nb[e] > 1;
        if (__any_sync(0xffffffffu, several)) {
#pragma unroll
            for (int e = 0; e < PerVec; ++e)
                if (nb[e] > 1) one_bias[tid * PerVec + e] = 0.f;
            add_repeats<PerVec>(a.bias_tokens, a.bias_values, b0, b1, slice0, end, n_bias, one_bias);
        }
#pragma unroll
        for (int e = 0; e < PerVec; ++e) {
            float b = nb[e] > 0 ? one_bias[tid * PerVec + e] : 0.f;
            if (nb[e] > 0) edited |= 1u << e;
            if (nh[e] > 0) {
                penalised |= 1u << e;
                b -= pen.frequency * (float)nh[e] + pen.presence;
            }
            add[e] = b;
        }
        edited |= penalised;
    }
    const uint32_t any = Lists ? __reduce_or_sync(0xffffffffu, edited) : 0u;
    if (n_mine == 0) return;
    const bool still = in_place && edited == 0;   // nothing to write where nothing is excluded
    const float down = 1.f / pen.repetition;
    for (int r = 0;;) {
        masks_of(r + kUnroll);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (r + u >= rows || (still && keep[u] == mine)) continue;
            if (any) edit<Bytes>(x[u], any, edited, penalised, down, pen.repetition, add);
            exclude<Bytes>(x[u], keep[u], expand);
            store<Bytes, Lists>(dst + u * a.ld_out_bytes, x[u], n_mine);
        }
        r += kUnroll;
        if (r >= rows) break;
        src += kUnroll * a.ld_bytes;
        dst += kUnroll * a.ld_out_bytes;
        load(r, still);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" dg_status dg_adjust_logits(const void* logits, dg_dtype dtype, int64_t ld, void* out, int64_t ld_out,
                                      int64_t n_canvas, int32_t L, int64_t V, const dg_canvas_params* params,
                                      const int32_t* history, const int32_t* cu_history, int64_t total_history,
                                      const dg_penalties* penalties, const int32_t* bias_tokens,
                                      const float* bias_values, const int32_t* cu_bias, int64_t total_bias,
                                      const uint32_t* masks, int64_t mask_stride, int32_t n_masks,
                                      const int32_t* mask_index, dg_stream_t stream) {
    if (dtype != DG_BF16 && dtype != DG_FP32) return DG_ERR_INVALID_ARG;
    if (n_canvas < 0 || n_canvas > 65535 || L < 1 || L > 1024 || V < 2 || V > 0x7fffffffLL || ld < V || ld_out < V ||
        total_history < 0 || total_history > 0x7fffffffLL || total_bias < 0 || total_bias > 0x7fffffffLL)
        return DG_ERR_INVALID_ARG;
    if (n_canvas == 0) return DG_OK;
    if (!logits || !out || !params) return DG_ERR_INVALID_ARG;
    if (history && (!cu_history || !penalties)) return DG_ERR_INVALID_ARG;
    if (bias_tokens && (!bias_values || !cu_bias)) return DG_ERR_INVALID_ARG;
    if (masks && (!mask_index || n_masks < 1 || mask_stride < (V + 31) / 32 || mask_stride > 0x7fffffffLL))
        return DG_ERR_INVALID_ARG;
    if (out == logits && ld_out != ld) return DG_ERR_INVALID_ARG;
    const int64_t es = dtype == DG_BF16 ? 2 : 4;
    if (!aligned(logits, 16) || !aligned(out, 16) || (ld * es) % 16 || (ld_out * es) % 16) return DG_ERR_ALIGNMENT;
    for (const void* p : {(const void*)params, (const void*)history, (const void*)cu_history, (const void*)penalties,
                          (const void*)bias_tokens, (const void*)bias_values, (const void*)cu_bias, (const void*)masks,
                          (const void*)mask_index})
        if (!aligned(p, 4)) return DG_ERR_ALIGNMENT;   // (records handed over as bytes may lie anywhere)
    if (V * es > 0x7fffffffLL) return DG_ERR_UNSUPPORTED;
    AdjustArgs a;
    a.x = static_cast<const unsigned char*>(logits);
    a.out = static_cast<unsigned char*>(out);
    a.ld_bytes = ld * es;
    a.ld_out_bytes = ld_out * es;
    a.L = L;
    a.V = (int32_t)V;
    a.params = params;
    a.history = history;
    a.cu_history = cu_history;
    a.penalties = penalties;
    a.bias_tokens = bias_tokens;
    a.bias_values = bias_values;
    a.cu_bias = cu_bias;
    a.masks = masks;
    a.mask_index = mask_index;
    a.total_history = total_history;
    a.total_bias = total_bias;
    a.mask_stride = mask_stride;
    a.n_masks = n_masks;
    a.status = dghost::status_word();
    const int sms = dghost::sm_count();
    if (sms <= 0) return DG_ERR_CUDA;
    const int64_t slice = kThreads * (16 / es), slices = (V + slice - 1) / slice;
    // rows of a block: up to 64, so that its lists are read for many rows, but few enough that the blocks
    // fill the places an SM has for them
    const bool lists = history || bias_tokens;
    const int64_t places = kBlocksPerSm * (int64_t)sms;
    const int64_t rows = (slices * n_canvas * L + places - 1) / places;
    a.rows = (int32_t)std::min<int64_t>(kMaxRows, (rows + 3) / 4 * 4);
    const dim3 grid((unsigned)slices, (unsigned)((L + a.rows - 1) / a.rows), (unsigned)n_canvas);
    const cudaError_t e = dghost::launch_pdl(es == 2 ? (lists ? k_adjust<2, true> : k_adjust<2, false>)
                                                     : (lists ? k_adjust<4, true> : k_adjust<4, false>), grid, dim3(kThreads), 0,
                                             (cudaStream_t)stream, a);
    dghost::count_launch();
    return dghost::cuda_status(e);
}
