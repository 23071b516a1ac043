// ep_moe_tokens.cu -- a whole mixture-of-experts layer for up to 64 tokens, in
// two kernels (and two small ones above 16 tokens or for large layers), without
// the dispatch / permute / combine round trip.
//
// Mathematics.  For token t with choices e = topk_idx[t][k], weights v[t][k]:
//   h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   out[t] = sum_k v[t][k] * W2[e] h[t,e].
// Kernel 1 leaves the sums Wg x and Wu x of every (token, expert) pair in fp32,
// kernel 2 forms h from them and the weighted sum.
//
// Bound.  Each weight byte of the experts that any token chose is read once;
// with one to a few tokens per expert that stream bounds the time.  So the
// weights are the 128 rows of the tensor-core product and go from memory to
// shared memory by tiled copies and nowhere else; the few tokens are its
// columns, written beside them by warps that convert them block by block:
//   fp8 weights: a token's 128 channels times a power of two, |v| < 256, are split
//     into e4m3 pieces, each the rest that the ones before leave, times 2^5 more
//     (a rest is at most 2^-5 of the range below 256, so that it fits again), and
//     each a column of its own.  A piece takes 5 bits and ends at 2^-9 of its power.
//     h, 24 bits: five pieces hold an element of 2^-13 of the block's largest or
//     more exactly, a smaller one to 2^-37 of the largest.  x, 8 bits: two pieces hold
//     an element of 2^-14 of the largest or more; what they leave of a smaller one is
//     at most 2^-15, and two more pieces, from 2^23 on, hold that.  An element of 2^-37
//     or more is exact, a smaller one off by at most 2^-45 (of the block's largest);
//   bf16 weights: x itself, and h as the sum of three bf16, which are its 24 bits.
// So the sums add x and h as a 32-bit form does.  Two pieces of x and three of h
// (two bf16) were off by up to 2^-21 of the largest and 2^-13 of h, which outputs
// that cancel show; 64 tokens took 694 us with them and take 754, bf16 417 / 418.
// For few tokens of a small layer each block converts what it needs; otherwise,
// where blocks would repeat much of it, the pieces are made once beforehand.
// A block of 128 channels is one accumulator; it leaves tensor memory, times its
// weight scale and the tokens' powers of two, for an fp32 sum in registers.
//
// Work items are (expert, 64 gate + 64 up channels, part of K) in kernel 1 and
// (128 output channels, expert, block of K) in kernel 2; each thread block takes
// its share, equal to within one.
//
// Measured: one token of 8 experts (H 7168, I 2048, fp8) 71 us, of which the
// weights' bytes take 53; 17 tokens, 75 experts, bf16 (H 4096, I 1408) 425 us, 6.1
// TB/s; 64 tokens, 99 experts 750 to 790 us, by its routing.
#include <atomic>

#include "ep_fp8.cuh"
#include "ep_tcgen05.cuh"

namespace ep {

constexpr int kTokMax = 64;        // tokens of a call: an expert's tokens are one 64-bit mask
constexpr int kTokThreads = 512;   // copy, mma, tensor-memory and spare warp; 8 that convert; 4 that sum
constexpr int kTokFillMost = 8;    // warps that convert tokens, at most
constexpr int kTokSlots = 16;      // tokens of a list entry: an expert with more has several, next to each other
constexpr int kTokRows = 128;      // weight rows of an item
constexpr int kTokBytes = 128;     // of a weight row per stage
constexpr int kTokScaleRing = 16;  // stages whose powers of two are kept: more than are ever between writer and reader
constexpr int kTokSplitMost = 4;   // parts of K in kernel 1, at most
constexpr int kTokChannelsMost = 1 << 28;  // hidden and inter: bytes and rows of a weight stay within 32 bits
constexpr int64_t kTokWaitNs = 2000000000ll;

template <bool kDown, bool kFp8>
struct TokShape {
    static constexpr int kPieces = kFp8 ? (kDown ? 5 : 4) : (kDown ? 3 : 1);  // columns of a token
    static constexpr int kCols = kTokSlots * kPieces;
    static constexpr int kAccCols = kCols <= 64 ? 64 : 128;  // tensor-memory columns of an accumulator
    // what piece z + 1 is multiplied by beyond piece z
    static constexpr float step(int z) { return !kFp8 ? 1.0f : !kDown && z == 1 ? 0x1p18f : 32.0f; }
    static constexpr int kStageA = kTokRows * kTokBytes, kStage = kStageA + kCols * kTokBytes;
    static constexpr int kStages = kDown ? (kFp8 ? 6 : 7) : (kFp8 ? 8 : 10);
    static constexpr int kChannels = kFp8 ? 128 : 64;  // of a stage
    // Each converting warp takes every kFill-th stage.  When it waits for the stage before its next one
    // to be done, it knows its own last one to be filled, so that stage kFill + kStages back is done; a
    // wait by parity is unambiguous if that is not later than 2 kStages back.
    static constexpr int kFill = kStages < kTokFillMost ? kStages : kTokFillMost;
    static_assert(kFill <= kStages, "a wait by parity could pass a whole round early");
};

struct TokArgs {
    const __nv_bfloat16* x;
    int64_t x_stride;
    const int64_t* topk_idx;
    const float* topk_weights;
    int T, K, E, H, I;
    const float* ws;        // scales of w13 in kernel 1, of w2 in kernel 2 (e4m3 only)
    int blocks_k;           // stages of a weight row
    int split;              // parts of K in kernel 1
    int list;               // entries of the expert list, at most
    float* sums;            // [split][T * K][2 I]: Wg x, then Wu x, of each pair
    float* part;            // [blocks][2][T][kTokRows]: sums of a tile that several blocks share
    uint32_t* done;         // [output tiles]: blocks that have written theirs; then the number of pairs
    uint8_t* formed;        // [T or pairs][blocks_k][pieces][kTokBytes]: pieces made beforehand, of x or of h
    float* powers;          // [T or pairs][blocks_k]: their powers of two (e4m3 only)
    __nv_bfloat16* out;
    int64_t out_stride;
    uint32_t* status;
};

struct TokBarriers {
    uint64_t copied[10], filled[10], done[10], acc_empty[2], drain;
    uint32_t tmem;
    int abort, last[2], entries;
    float scale[kTokScaleRing][kTokSlots];
};

struct TokLists {
    float* acc;        // [T][kTokRows] (kernel 2)
    float* weight;     // [pairs] (kernel 2)
    uint16_t* expert;  // [list]
    uint16_t* base;    // [list + 1]: pairs of entry i are base[i] .. base[i + 1] - 1
    uint8_t* token;    // [pairs]
};

template <bool kDown, bool kFp8>
constexpr size_t tok_smem(int T, int K, int list) {
    using Shape = TokShape<kDown, kFp8>;
    return 1024 + (size_t)Shape::kStages * Shape::kStage + (kDown ? sizeof(float) * T * (kTokRows + K) : 0) +
           sizeof(uint16_t) * (2 * list + 2) + (size_t)T * K + 16;
}

// The experts that some token chose, ascending, and their tokens, ascending, at
// most kTokSlots to an entry.  Every block builds the list for itself.  Returns
// the number of entries.
template <bool kDown>
__device__ __forceinline__ int build_list(const TokArgs& a, const TokLists& s, uint8_t* scratch) {
    constexpr int kWarps = kTokThreads / 32;
    __shared__ int scan[kWarps];
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(scratch);      // [E], 32 KB at most
    uint16_t* pair_expert = reinterpret_cast<uint16_t*>(mask + kMaxExperts);        // [pairs]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += kTokThreads) mask[e] = 0;
    __syncthreads();
    for (int p = tid; p < a.T * a.K; p += kTokThreads) {
        const int64_t e = a.topk_idx[p];
        if (e >= 0 && e < a.E) atomicOr(&mask[e], 1ull << (p / a.K));
        else if (e != -1 && a.status && blockIdx.x == 0 && !kDown) flag(a.status, FLAG_INVALID_TOPK);
    }
    __syncthreads();
    const int per = (a.E + kTokThreads - 1) / kTokThreads, e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
    int sum = 0;  // entries in the high half, pairs in the low: at most 2176 and 2048
    for (int e = e0; e < e1; ++e) {
        const int m = __popcll(mask[e]);
        sum += ((m + kTokSlots - 1) / kTokSlots << 16) + m;
    }
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += scan[w];
        total += scan[w];
    }
    for (int e = e0; e < e1; ++e) {
        unsigned long long m = mask[e];
        for (int z = 0; m; m &= m - 1, ++z, ++at) {
            const int p = at & 0xffff;
            if (z % kTokSlots == 0) {
                s.expert[at >> 16] = (uint16_t)e;
                s.base[at >> 16] = (uint16_t)p;
                at += 1 << 16;
            }
            s.token[p] = (uint8_t)(__ffsll(m) - 1);
            pair_expert[p] = (uint16_t)e;
        }
    }
    if (tid == 0) s.base[total >> 16] = (uint16_t)(total & 0xffff);
    __syncthreads();
    if constexpr (kDown) {  // a token that names an expert twice is one pair with both weights
        for (int p = tid; p < (total & 0xffff); p += kTokThreads) {
            const int64_t* idx = a.topk_idx + s.token[p] * a.K;
            float v = 0.0f;
            for (int k = 0; k < a.K; ++k)
                if (idx[k] == pair_expert[p]) v += a.topk_weights[s.token[p] * a.K + k];
            s.weight[p] = v;
        }
        for (int i = tid; i < a.T * kTokRows; i += kTokThreads) s.acc[i] = 0.0f;
    }
    __syncthreads();
    return total >> 16;
}

// The same for at most 32 pairs of at most kTokSlots tokens, by one warp: a pair
// per lane, so that a block waits for one load and no barrier (2.1 us for the
// general form, most of it barriers).  Entries in the order in which the pairs
// first name their experts.
template <bool kDown>
__device__ __forceinline__ void build_short_list(const TokArgs& a, const TokLists& s, int* entries) {
    const int lane = threadIdx.x & 31, pairs = a.T * a.K, t = lane / a.K;
    const int64_t e64 = lane < pairs ? a.topk_idx[lane] : -1;
    const float w = kDown && lane < pairs ? a.topk_weights[lane] : 0.0f;
    const bool ok = e64 >= 0 && e64 < a.E;
    if (!kDown && !ok && e64 != -1 && a.status && blockIdx.x == 0) flag(a.status, FLAG_INVALID_TOPK);
    const int e = ok ? (int)e64 : -1 - lane;  // its own group, left out below
    const uint32_t same = __match_any_sync(0xffffffffu, e), lower = lanemask_lt();
    const uint32_t token = __match_any_sync(0xffffffffu, t);
    // a token that names an expert again adds its weight to the first pair
    const bool first = ok && !(same & token & lower);
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    const bool leads = ok && !(same & lower);
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    // pairs of the entries of earlier leaders: every lane's entry is its group's leader's
    int base = 0;
    for (uint32_t m = leaders; m; m &= m - 1) {
        const int b = __ffs(m) - 1;
        const int n = __popc(__shfl_sync(0xffffffffu, same, b) & firsts);
        if (b < __ffs(same) - 1) base += n;
    }
    const int at = base + __popc(same & firsts & lower);
    if (leads) {
        const int i = __popc(leaders & lower);
        s.expert[i] = (uint16_t)e;
        s.base[i] = (uint16_t)base;
    }
    if (first) s.token[at] = (uint8_t)t;
    if constexpr (kDown) {
        float v = 0.0f;
        for (int b = 0; b < 32; ++b) {
            const float x = __shfl_sync(0xffffffffu, w, b);
            if (same & token & (1u << b)) v += x;
        }
        if (first) s.weight[at] = v;
    }
    if (lane == 0) {
        *entries = __popc(leaders);
        s.base[*entries] = (uint16_t)__popc(firsts);
    }
}

// The runs of one block: an entry's tile and a range of its blocks of K.
// Kernel 1 takes every `step`-th item, so that the tiles of one entry, and what
// they cost, are spread over the blocks.  Kernel 2 takes a contiguous range of
// the blocks of K, tile after tile, so that most of a tile's entries meet in
// one block's sum.
template <bool kDown>
struct TokRuns {
    int at, end, step, A, tiles, blocks_k, split;
    int ai, tile, k0, k1, part;
    __device__ __forceinline__ bool next() {
        if (at >= end) return false;
        if constexpr (kDown) {
            const int item = at / blocks_k;
            k0 = at - item * blocks_k;
            k1 = min(blocks_k, k0 + end - at);
            tile = item / A;
            ai = item - tile * A;
            part = 0;
            at += k1 - k0;
        } else {
            const int item = at / split;
            part = at - item * split;
            ai = item / tiles;
            tile = item - ai * tiles;
            k0 = part * blocks_k / split;
            k1 = (part + 1) * blocks_k / split;
            at += step;
        }
        return true;
    }
};

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    return (e4m3x2(a, b) & 0xffffu) | (e4m3x2(c, d) << 16);
}
// v[0..3] minus the values of their codes, times `step`: what the next piece holds.
__device__ __forceinline__ void next_piece(float* v, uint32_t codes, float step) {
    const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3)));
    const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16), __NV_E4M3)));
    v[0] = (v[0] - lo.x) * step;
    v[1] = (v[1] - lo.y) * step;
    v[2] = (v[2] - hi.x) * step;
    v[3] = (v[3] - hi.y) * step;
}

// kN consecutive 32-bit words.
template <int kN>
__device__ __forceinline__ void load_words(const float* p, float* v) {
    if constexpr (kN == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
    else if constexpr (kN == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p);
    else *v = *p;
}

// A lane's channels of a token's block as pieces, each handed to put(piece, 4 bytes).  Returns the
// power of two that the block's sums are multiplied by (e4m3 only).
template <bool kDown, bool kFp8, int kLane, class Put>
__device__ __forceinline__ float write_pieces(float (&v)[kLane], Put put) {
    using Shape = TokShape<kDown, kFp8>;
    constexpr int kPieces = Shape::kPieces;
    if constexpr (kFp8) {
        uint32_t top = 0;  // the largest magnitude's bits, above infinity's where one is NaN
#pragma unroll
        for (int z = 0; z < 4; ++z) top = max(top, __float_as_uint(v[z]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const int e = max((int)(top >> 23) - 127, -100);  // |v| < 2^(e + 1)
        const bool odd = top >= 0x7f800000u;
        const float up = odd ? 1.0f : __uint_as_float((uint32_t)(7 - e + 127) << 23);
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] *= up;
#pragma unroll
        for (int z = 0; z < kPieces; ++z) {
            const uint32_t c = pack_e4m3(v[0], v[1], v[2], v[3]);
            put(z, odd ? 0x7f7f7f7fu : c);  // an infinity or a NaN makes the token's whole block NaN
            if (z + 1 < kPieces) next_piece(v, c, Shape::step(z));
        }
        return odd ? 1.0f : __uint_as_float((uint32_t)(e - 7 + 127) << 23);
    } else {
#pragma unroll
        for (int z = 0; z < kPieces; ++z) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[0], v[1]);
            put(z, *reinterpret_cast<const uint32_t*>(&b));
            const float2 f = __bfloat1622float2(b);
            v[0] = isfinite(f.x) ? v[0] - f.x : 0.0f;
            v[1] = isfinite(f.y) ? v[1] - f.y : 0.0f;
        }
        return 1.0f;
    }
}

// A lane's channels of x, or of h from both sums.
template <bool kDown, int kLane>
__device__ __forceinline__ void values_of(const float* w, float (&v)[kLane]) {
    if constexpr (kDown) {
#pragma unroll
        for (int z = 0; z < kLane; ++z) v[z] = silu_mul(w[z], w[kLane + z]);
    } else {
#pragma unroll
        for (int z = 0; z < kLane; z += 2) {
            const uint32_t two = __float_as_uint(w[z / 2]);
            v[z] = __uint_as_float(two << 16);
            v[z + 1] = __uint_as_float(two & 0xffff0000u);
        }
    }
}

// The pieces of x (before kernel 1) or of h (between both), once for all blocks:
// a warp per token or pair and block of channels.
template <bool kDown, bool kFp8>
__global__ void __launch_bounds__(256) form_kernel(const TokArgs a) {
    using Shape = TokShape<kDown, kFp8>;
    constexpr int kPieces = Shape::kPieces, kLane = Shape::kChannels / 32, kRaw = kDown ? 2 * kLane : kLane / 2;
    grid_wait();  // kernel 1, or what ran before the call
    grid_launch_next();
    const int lane = threadIdx.x & 31;
    const int rows = kDown ? (int)a.done[(a.H + kTokRows - 1) / kTokRows] : a.T;
    for (int i = (blockIdx.x * 256 + threadIdx.x) >> 5; i < rows * a.blocks_k; i += gridDim.x * 8) {
        const int row = i / a.blocks_k, ch = (i - row * a.blocks_k) * Shape::kChannels + lane * kLane;
        float raw[kRaw] = {}, v[kLane];
        if (ch < (kDown ? a.I : a.H)) {
            if constexpr (kDown) {
                for (int z = 0; z < a.split; ++z) {
                    const float* p = a.sums + ((int64_t)z * a.T * a.K + row) * 2 * a.I + ch;
                    float more[kRaw];
                    load_words<kLane>(p, more);
                    load_words<kLane>(p + a.I, more + kLane);
#pragma unroll
                    for (int q = 0; q < kRaw; ++q) raw[q] += more[q];
                }
            } else {
                load_words<kRaw>(reinterpret_cast<const float*>(a.x + row * a.x_stride + ch), raw);
            }
        }
        values_of<kDown>(raw, v);
        uint8_t* to = a.formed + (int64_t)i * kPieces * kTokBytes + lane * 4;
        const float power = write_pieces<kDown, kFp8>(v, [&](int z, uint32_t w) { *reinterpret_cast<uint32_t*>(to + z * kTokBytes) = w; });
        if (kFp8 && lane == 0) a.powers[i] = power;
    }
}

// kDown: kernel 2.  kFp8: e4m3 weights with block scales, otherwise bf16.
// kParts: the sums come in several parts (few items, so few tokens); without
// them the next tokens' sums are loaded while these are converted, for which
// both forms in one kernel leave too few registers (64 tokens: 938 us instead of
// 904).  kFormed: the tokens' pieces were made beforehand and are copied.
template <bool kDown, bool kFp8, bool kParts, bool kFormed>
__global__ void __launch_bounds__(kTokThreads, 1) tok_kernel(const __grid_constant__ CUtensorMap map_w, const TokArgs a) {
    using Shape = TokShape<kDown, kFp8>;
    constexpr int kStages = Shape::kStages, kPieces = Shape::kPieces;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ TokBarriers sh;
    uint8_t* ring = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    TokLists s;
    s.acc = reinterpret_cast<float*>(ring + kStages * Shape::kStage);
    s.weight = s.acc + (kDown ? a.T * kTokRows : 0);
    s.expert = reinterpret_cast<uint16_t*>(s.weight + (kDown ? a.T * a.K : 0));
    s.base = s.expert + a.list;
    s.token = reinterpret_cast<uint8_t*>(s.base + a.list + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &sh.abort;
    const uint32_t copied = smem_u32(sh.copied), filled = smem_u32(sh.filled), done = smem_u32(sh.done);
    const uint32_t acc_empty = smem_u32(sh.acc_empty);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.copied[i], 1);
            mbar_init(&sh.filled[i], 1);
            mbar_init(&sh.done[i], 1);
        }
        mbar_init(&sh.acc_empty[0], 4);
        mbar_init(&sh.acc_empty[1], 4);
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_w);
    }
    if (warp == 2) tmem_alloc<1>(&sh.tmem, 2 * Shape::kAccCols);
    // What is above may run beside the end of the kernel before.  The first kernel of a call waits for what
    // ran before the call; the later ones start after that, and wait below, where they read their own.
    if constexpr (!kDown && !kFormed) grid_wait();
    grid_launch_next();
    if (!kDown && blockIdx.x == 0)
        for (int i = tid; i < (a.H + kTokRows - 1) / kTokRows; i += kTokThreads) a.done[i] = 0;
    int A = 0;
    const bool brief = a.T <= kTokSlots && a.T * a.K <= 32;
    if (brief) {
        if (warp == 3) build_short_list<kDown>(a, s, &sh.entries);
        if (kDown)
            for (int i = tid; i < a.T * kTokRows; i += kTokThreads) s.acc[i] = 0.0f;
    } else {
        A = build_list<kDown>(a, s, ring);
        fence_proxy_async_smem();  // the list's scratch becomes the ring
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (brief) A = sh.entries;
    if (!kDown && blockIdx.x == 0 && tid == 0) a.done[(a.H + kTokRows - 1) / kTokRows] = s.base[A];

    const int tiles = kDown ? (a.H + kTokRows - 1) / kTokRows : (a.I + kTokRows / 2 - 1) / (kTokRows / 2);
    const int total = A * tiles * (kDown ? a.blocks_k : a.split);
    // Blocks with work; the rest are idle.  In kernel 2 the blocks of a tile each stream per / n stages (0.4 us
    // each) and the last one adds n parts of T tokens (0.05 us for 4 tokens each, about): n as makes both equal.
    int most = gridDim.x;
    if constexpr (kDown) most = min(most, tiles * max(1, (int)sqrtf(8.0f * A * a.blocks_k / ((a.T + 3) / 4))));
    const int blocks = max(1, min(total, most));
    auto first_of = [&](int b) { return (int)((int64_t)total * b / blocks); };
    TokRuns<kDown> run;
    const bool idle = (int)blockIdx.x >= blocks;
    run.at = idle ? total : kDown ? first_of(blockIdx.x) : blockIdx.x;
    run.end = idle || !kDown ? total : first_of(blockIdx.x + 1);
    run.step = blocks;
    run.A = A;
    run.tiles = tiles;
    run.blocks_k = a.blocks_k;
    run.split = a.split;
    const int begin = run.at;

    if (warp == 0) {
        if (lane == 0) {
            // ---- weights: two boxes of 64 rows a stage ----------------------------
            uint32_t n = 0;
            bool ok = true;
            while (ok && run.next()) {
                const int e = s.expert[run.ai];
                const int r0 = kDown ? run.tile * kTokRows : run.tile * (kTokRows / 2), r1 = kDown ? r0 + 64 : a.I + r0;
                for (int k = run.k0; k < run.k1; ++k, ++n) {
                    const uint32_t u = n % kStages;
                    if (!mbar_wait_or_abort(done + u * 8, n / kStages & 1 ^ 1, kTokWaitNs, abort)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = ring + u * Shape::kStage;
                    mbar_arrive_expect_tx(&sh.copied[u], Shape::kStageA);
                    tma_load_3d<1>(st, &map_w, k * kTokBytes, r0, e, copied + u * 8);
                    tma_load_3d<1>(st + 64 * kTokBytes, &map_w, k * kTokBytes, r1, e, copied + u * 8);
                }
            }
            // no copy may be in flight when the block ends, also after a wait that ran out
            for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
                mbar_wait_bounded(&sh.copied[i % kStages], i / kStages & 1, kTokWaitNs);
        }
    } else if (warp == 1) {
        // ---- products: one block of K per accumulator, two accumulators ------------
        const uint32_t idesc = kFp8 ? idesc_e4m3(kTokRows, Shape::kCols) : idesc_bf16(kTokRows, Shape::kCols);
        const uint64_t d0 = smem_desc_sw128(ring);
        uint32_t n = 0;
        while (run.next()) {
#pragma unroll 1
            for (int k = run.k0; k < run.k1; ++k, ++n) {
                const uint32_t u = n % kStages, ph = n / kStages & 1;
                mbar_wait_warp(copied + u * 8, ph, kTokWaitNs, abort);
                mbar_wait_warp(filled + u * 8, ph, kTokWaitNs, abort);
                mbar_wait_warp(acc_empty + (n & 1) * 8, n >> 1 & 1 ^ 1, kTokWaitNs, abort);
                tc_fence_after();
                const uint64_t da = d0 + u * (Shape::kStage >> 4), db = da + (Shape::kStageA >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (kFp8) mma_e4m3<1>(tmem + (n & 1) * Shape::kAccCols, da + q * 2, db + q * 2, idesc, q > 0);
                        else mma_bf16_ss(tmem + (n & 1) * Shape::kAccCols, da + q * 2, db + q * 2, idesc, q > 0);
                    }
                    mma_commit<1>(done + u * 8);
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit<1>(smem_u32(&sh.drain));  // every product has finished before tensor memory is freed
        __syncwarp();
        mbar_wait_bounded(&sh.drain, 0, kTokWaitNs);
    } else if (warp >= 4 && warp < 4 + kTokFillMost) {
        // ---- tokens: warp w converts stages w, w + kFill, ... of the block ----------------
        constexpr uint32_t kFill = Shape::kFill;
        if (warp - 4 >= (int)kFill) run.at = run.end;
        if constexpr (kDown || kFormed) grid_wait();  // the sums of kernel 1, or the pieces
        uint32_t n0 = 0;
        while (run.next()) {
            const int p0 = s.base[run.ai], cnt = s.base[run.ai + 1] - p0, len = run.k1 - run.k0;
            for (int i = (warp - 4 + kFill - n0 % kFill) % kFill; i < len; i += kFill) {
                const uint32_t n = n0 + i, u = n % kStages;
                if constexpr (kFormed) {
                    // four rows (a piece of a token each) at a time, 16 bytes a lane
                    const int unit = lane & 7, k = run.k0 + i;
                    auto source = [&](int j) { return (int64_t)(kDown ? p0 + j : s.token[p0 + j]) * a.blocks_k + k; };
                    constexpr int kAt = Shape::kCols <= 48 ? Shape::kCols / 4 : Shape::kCols / 8;  // on their way at once
                    int4 w[kAt];
                    float power = 0.0f;
                    uint8_t* st = ring + u * Shape::kStage + Shape::kStageA;
                    auto load = [&](int r0) {
#pragma unroll
                        for (int q = 0; q < kAt; ++q) {
                            const int r = r0 + q * 4 + (lane >> 3), j = r / kPieces;
                            if (j < cnt)
                                w[q] = __ldcg(reinterpret_cast<const int4*>(a.formed + (source(j) * kPieces + r - j * kPieces) * kTokBytes) + unit);
                        }
                    };
                    auto store = [&](int r0) {
#pragma unroll
                        for (int q = 0; q < kAt; ++q) {
                            const int r = r0 + q * 4 + (lane >> 3);
                            if (r / kPieces < cnt) *reinterpret_cast<int4*>(st + r * kTokBytes + ((unit ^ (r & 7)) << 4)) = w[q];
                        }
                    };
                    load(0);
                    if (kFp8 && lane < cnt) power = __ldcg(a.powers + source(lane));
                    mbar_wait_warp(done + u * 8, n / kStages & 1 ^ 1, kTokWaitNs, abort);
                    store(0);
                    if (kAt * 4 < Shape::kCols && cnt * kPieces > kAt * 4) {
                        load(kAt * 4);
                        store(kAt * 4);
                    }
                    if (kFp8 && lane < cnt) sh.scale[n % kTokScaleRing][lane] = power;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(filled + u * 8);
                    continue;
                }
                constexpr int kLane = Shape::kChannels / 32;  // channels of a lane
                const int ch = (run.k0 + i) * Shape::kChannels + lane * kLane;
                const bool in = ch < (kDown ? a.I : a.H);
                uint8_t* st = ring + u * Shape::kStage + Shape::kStageA;
                // what a lane reads of a token: its channels of x, or of both sums
                constexpr int kRaw = kDown ? 2 * kLane : kLane / 2;
                const int64_t part = (int64_t)a.T * a.K * 2 * a.I;
                auto sums_of = [&](int j) { return a.sums + (int64_t)(p0 + j) * 2 * a.I + ch; };
                auto load = [&](int j0, float(&raw)[4][kRaw]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int z = 0; z < kRaw; ++z) raw[q][z] = 0.0f;
                        if (in && j0 + q < cnt) {
                            if constexpr (kDown) {
                                const float* p = sums_of(j0 + q);
                                load_words<kLane>(p, raw[q]);
                                load_words<kLane>(p + a.I, raw[q] + kLane);
                                if constexpr (kParts) {  // the other parts, all on their way at once
                                    float more[kTokSplitMost - 1][kRaw];
#pragma unroll
                                    for (int z = 0; z < kTokSplitMost - 1; ++z)
                                        if (z + 1 < a.split) {
                                            load_words<kLane>(p + (z + 1) * part, more[z]);
                                            load_words<kLane>(p + (z + 1) * part + a.I, more[z] + kLane);
                                        }
#pragma unroll
                                    for (int z = 0; z < kTokSplitMost - 1; ++z)
                                        if (z + 1 < a.split)
#pragma unroll
                                            for (int i = 0; i < kRaw; ++i) raw[q][i] += more[z][i];
                                }
                            } else {
                                load_words<kLane / 2>(
                                    reinterpret_cast<const float*>(a.x + s.token[p0 + j0 + q] * a.x_stride + ch), raw[q]);
                            }
                        }
                    }
                };
                auto convert = [&](int j0, float(&raw)[4][kRaw]) {
                    float v[4][kLane];
#pragma unroll
                    for (int q = 0; q < 4; ++q) values_of<kDown>(raw[q], v[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // four independent chains; a token too many is zeros
                        // piece z of the token is row col + z of the tile, 4 bytes a lane, 16-byte units
                        // exchanged by the 128-byte swizzle
                        const int col = (j0 + q) * kPieces;
                        const float power = write_pieces<kDown, kFp8>(v[q], [&](int z, uint32_t w) {
                            const int r = col + z;
                            *reinterpret_cast<uint32_t*>(st + r * kTokBytes + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) = w;
                        });
                        if (kFp8 && lane == 0) sh.scale[n % kTokScaleRing][j0 + q] = power;
                    }
                };
                float raw[kParts ? 1 : 2][4][kRaw];
                load(0, raw[0]);
                mbar_wait_warp(done + u * 8, n / kStages & 1 ^ 1, kTokWaitNs, abort);
                if constexpr (kParts) {
#pragma unroll 1
                    for (int j0 = 0; j0 < cnt; j0 += 4) {
                        if (j0 > 0) load(j0, raw[0]);
                        convert(j0, raw[0]);
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < kTokSlots / 4; ++b) {
                        if (b * 4 >= cnt) break;
                        if (b * 4 + 4 < cnt) load(b * 4 + 4, raw[(b + 1) & 1]);  // on their way while these are converted
                        convert(b * 4, raw[b & 1]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(filled + u * 8);
            }
            n0 += len;
        }
    } else if (warp >= 12) {
        // ---- sums: thread r owns weight row r of the tile ---------------------------------
        const int r = (warp - 12) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(warp - 12) << 21);
        if constexpr (kDown) grid_wait();  // the counters of kernel 1
        if (kDown && A == 0)
            for (int64_t i = blockIdx.x * 128ll + r; i < (int64_t)a.T * a.H; i += gridDim.x * 128ll)
                a.out[i / a.H * a.out_stride + i % a.H] = __float2bfloat16_rn(0.0f);
        uint32_t n = 0;
        while (run.next()) {
            const int p0 = s.base[run.ai], cnt = s.base[run.ai + 1] - p0;
            // the row's channel: kernel 1 has 64 gate rows, then the 64 up rows of the same channels
            const int ch = kDown ? run.tile * kTokRows + r : run.tile * (kTokRows / 2) + (r & 63);
            const int row = kDown ? ch : (r < 64 ? ch : a.I + ch);
            const float* ws = nullptr;
            if constexpr (kFp8)
                ws = a.ws + ((int64_t)s.expert[run.ai] * ((kDown ? a.H : 2 * a.I) / 128) + row / 128) * a.blocks_k;
            float acc[kTokSlots];
#pragma unroll
            for (int j = 0; j < kTokSlots; ++j) acc[j] = 0.0f;
            float sw = kFp8 ? ws[run.k0] : 1.0f;
#pragma unroll 1
            for (int k = run.k0; k < run.k1; ++k, ++n) {
                const float f = sw;
                if (kFp8 && k + 1 < run.k1) sw = ws[k + 1];
                mbar_wait_warp(done + n % kStages * 8, n / kStages & 1, kTokWaitNs, abort);
                tc_fence_after();
                const float* sc = sh.scale[n % kTokScaleRing];
                // the pieces of kAt tokens, in order, 16 columns at a time
                constexpr int kAt = kPieces > 3 ? kTokSlots / 2 : kTokSlots, kLoads = (kAt * kPieces + 15) / 16;
                const uint32_t ad = lane_base + (n & 1) * Shape::kAccCols;
#pragma unroll
                for (int j0 = 0; j0 < kTokSlots; j0 += kAt) {
                    if (j0 >= cnt) break;
                    float t[16 * kLoads];
#pragma unroll
                    for (int q = 0; q < kLoads; ++q)
                        if ((cnt - j0) * kPieces > q * 16) tmem_ld(ad + j0 * kPieces + q * 16, *reinterpret_cast<float(*)[16]>(t + q * 16));
#pragma unroll
                    for (int q = 0; q < kLoads; ++q) tmem_wait_ld(*reinterpret_cast<float(*)[16]>(t + q * 16));
                    if (j0 + kAt >= cnt) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_hand_back(acc_empty + (n & 1) * 8);
                    }
#pragma unroll
                    for (int j = 0; j < kAt; ++j) {
                        if ((j & 3) == 0 && j0 + j >= cnt) break;
                        float y = t[j * kPieces + kPieces - 1];
#pragma unroll
                        for (int z = kPieces - 2; z >= 0; --z) y = fmaf(y, 1.0f / Shape::step(z), t[j * kPieces + z]);
                        if constexpr (kFp8) acc[j0 + j] = fmaf(y, f * sc[j0 + j], acc[j0 + j]);
                        else acc[j0 + j] += y;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kTokSlots; ++j) {
                if (j >= cnt) break;
                const int pair = p0 + j;
                if constexpr (kDown) {
                    float* o = s.acc + s.token[pair] * kTokRows + r;
                    *o = fmaf(s.weight[pair], acc[j], *o);
                } else if (ch < a.I) {
                    a.sums[((int64_t)run.part * a.T * a.K + pair) * 2 * a.I + row] = acc[j];
                }
            }
            if constexpr (kDown) {
                const int per = A * a.blocks_k;  // units of a tile
                if (run.at < run.end && run.at / per == run.tile) continue;
                // The end of this block's part of a tile: its outputs, or, where other blocks share it, its part.
                // Only the block's first and last tile can be shared; both are joined at the block's end, so
                // that the sums between do not wait.
                const int lo = run.tile * per;
                const bool shared = begin > lo || run.end < lo + per;
                float* mine = a.part + ((int64_t)blockIdx.x * 2 + (run.tile != begin / per)) * a.T * kTokRows + r;
                for (int t = 0; t < a.T; ++t) {
                    const float v = s.acc[t * kTokRows + r];
                    if (shared) mine[t * kTokRows] = v;
                    else if (ch < a.H) a.out[t * a.out_stride + ch] = __float2bfloat16_rn(v);
                    s.acc[t * kTokRows + r] = 0.0f;
                }
            }
        }
        if constexpr (kDown) __threadfence();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free<1>(tmem, 2 * Shape::kAccCols);
    if constexpr (kDown) {
        // the block that leaves a tile's last part adds the parts in block order
        if (!idle && A > 0) {
            const int per = A * a.blocks_k, first = begin / per, last = (run.end - 1) / per;
            auto block_of = [&](int unit) { return (int)(((int64_t)(unit + 1) * blocks - 1) / total); };
            if (lane == 0 && warp < 2) {  // a warp for each of the two tiles
                const int tile = warp == 0 ? first : last, lo = tile * per;
                bool is_last = false;
                if ((warp == 0 || last > first) && (begin > lo || run.end < lo + per)) {
                    is_last = atomicAdd(&a.done[tile], 1u) == (uint32_t)(block_of(lo + per - 1) - block_of(lo));
                    __threadfence();
                }
                sh.last[warp] = is_last;
            }
            __syncthreads();
            for (int z = 0; z < 2; ++z) {
                if (!sh.last[z]) continue;
                // A warp per token, four rows a lane: four parts of two tokens on their way at a time.  The
                // later blocks began in this tile; the first one may have left another's part before.
                constexpr int kAt = 4, kWarps = kTokThreads / 32;
                const int tile = z ? last : first, lo = tile * per;
                const int b0 = block_of(lo), b1 = block_of(lo + per - 1), second = first_of(b0) < lo;
                auto from = [&](int b, int t) {
                    return __ldcg(reinterpret_cast<const float4*>(a.part + ((int64_t)(b * 2 + (b == b0 ? second : 0)) * a.T + t) * kTokRows) + lane);
                };
                for (int t = warp; t < a.T; t += 2 * kWarps) {
                    const bool two = t + kWarps < a.T;
                    float4 v[2] = {};
                    for (int q0 = b0; q0 <= b1; q0 += kAt) {
                        float4 x[kAt][2];
#pragma unroll
                        for (int q = 0; q < kAt; ++q)
                            if (q0 + q <= b1) {
                                x[q][0] = from(q0 + q, t);
                                if (two) x[q][1] = from(q0 + q, t + kWarps);
                            }
#pragma unroll
                        for (int q = 0; q < kAt; ++q)
                            if (q0 + q <= b1)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    v[i].x += x[q][i].x, v[i].y += x[q][i].y;
                                    v[i].z += x[q][i].z, v[i].w += x[q][i].w;
                                }
                    }
                    const int ch = tile * kTokRows + lane * 4;  // H is a multiple of 32
                    if (ch < a.H)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (i == 0 || two) {
                                __nv_bfloat16* o = a.out + (t + i * kWarps) * a.out_stride + ch;
                                o[0] = __float2bfloat16_rn(v[i].x);
                                o[1] = __float2bfloat16_rn(v[i].y);
                                o[2] = __float2bfloat16_rn(v[i].z);
                                o[3] = __float2bfloat16_rn(v[i].w);
                            }
                }
            }
        }
    }
    if (tid == 0 && *abort && a.status) flag(a.status, FLAG_TIMEOUT);
}

// Whether the pieces are made beforehand: two launches and their hand-over, 4 to 5 us of the host's time or of a
// short call's, against a conversion by every block that meets the token (us, by each block / beforehand).  fp8, 128
// experts, top-8, H 7168, I 2048: one token 74.8 / 71.4, 8 373 / 366, 16 569 / 558, 32 780 / 759, 64 986 / 861, skewed
// 942 / 605; 32 experts, top-4, H 2048, I 768: 2 24.7 / 26.8, 8 39.4 / 38.3, 16 52.4 / 48.2; 16 experts, top-2, H 4096,
// I 1408: 1 23.9 / 26.7, 2 30.1 / 31.0, 4 38.5 / 37.9, 16 64.7 / 60.8, 64 129 / 83; H 2048, I 768: 8 27.4 / 28.2, 16
// 32.9 / 33.0, 17 35.5 / 34.9; 8 experts, H 1024, I 512: 16 22.5 / 26.0, 17 25.0 / 25.7, 32 35.4 / 27.5.  So above 16
// tokens, and where the chosen experts' weights have 100 MB, so that the call hides the launches.  bf16 halves only h:
// 16 experts, 17 tokens 95.5 / 98.1, 32 114 / 108, 64 142 / 117; 75 experts, top-6, 64 tokens 404 / 410.
static bool tok_formed(int T, int K, int E, int H, int I, bool fp8) {
    if (!fp8) return T > kTokSlots && T * K >= 6 * E;
    return T > kTokSlots || (int64_t)(E < T * K ? E : T * K) * H * I >= 100000000 / 3;
}

// Entries of the expert list, at most: one for each expert that is chosen, and one more for every kTokSlots pairs.
static int tok_list(int T, int K, int E) { return (E < T * K ? E : T * K) + T * K / kTokSlots; }

struct TokWorkspace {
    int split;
    int64_t part, done, formed_x, formed_h, powers, bytes;
};
// The parts of K in kernel 1: enough items that the blocks' shares differ little,
// each with a few stages left.
static TokWorkspace tok_workspace(int T, int K, int E, int H, int I, bool fp8, int sms) {
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int blocks_k = (H * (fp8 ? 1 : 2) + kTokBytes - 1) / kTokBytes;
    const int64_t items = (int64_t)(E < T * K ? E : T * K) * ((I + kTokRows / 2 - 1) / (kTokRows / 2));
    int64_t split = (6 * sms + items - 1) / items;
    if (split > kTokSplitMost) split = kTokSplitMost;
    if (split > blocks_k / 4) split = blocks_k / 4;
    TokWorkspace w;
    w.split = split < 1 ? 1 : (int)split;
    w.part = up((int64_t)w.split * T * K * 2 * I * 4);
    w.done = w.part + up((int64_t)sms * 2 * T * kTokRows * 4);
    w.formed_x = w.formed_h = w.powers = w.bytes = w.done + up((int64_t)((H + kTokRows - 1) / kTokRows + 1) * 4);
    if (tok_formed(T, K, E, H, I, fp8)) {
        const int64_t blocks_x = fp8 ? (int64_t)T * blocks_k : 0;
        const int64_t blocks_h = (int64_t)T * K * ((I * (fp8 ? 1 : 2) + kTokBytes - 1) / kTokBytes);
        w.formed_h = w.formed_x + blocks_x * TokShape<false, true>::kPieces * kTokBytes;
        w.powers = w.formed_h + blocks_h * (fp8 ? TokShape<true, true>::kPieces : TokShape<true, false>::kPieces) * kTokBytes;
        w.bytes = w.powers + up((blocks_x > blocks_h ? blocks_x : blocks_h) * 4);
    }
    return w;
}

static ep_status tok_map(CUtensorMap* m, const void* w, int64_t row_bytes, int64_t rows, int experts, const char* fn) {
    const cuuint64_t dims[3] = {(cuuint64_t)row_bytes, (cuuint64_t)rows, (cuuint64_t)experts};
    const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)(row_bytes * rows)};
    const cuuint32_t box[3] = {kTokBytes, 64, 1};
    return encode_rows(m, w, 3, dims, strides, box, fn);
}

template <bool kFp8>
static ep_status launch_tokens(TokArgs a, const ep_moe_weights* w, int sms, const TokWorkspace& ws, uint8_t* mem, cudaStream_t st) {
    const char* fn = "ep_moe_tokens";
    int dev = 0;
    EP_CUDA(cudaGetDevice(&dev));
    static std::atomic<bool> known[kMaxDevicesTracked];  // devices whose launch attributes are set
    if (dev >= kMaxDevicesTracked || !known[dev].load(std::memory_order_relaxed)) {
        constexpr int kMost = kTokMax * kMaxTopk + kTokMax * kMaxTopk / kTokSlots;
        auto allow = [](auto* kernel, size_t bytes) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        };
        static_assert(tok_smem<false, kFp8>(kTokMax, kMaxTopk, kMost) + sizeof(TokBarriers) + 128 <= 227 * 1024 &&
                      tok_smem<true, kFp8>(kTokMax, kMaxTopk, kMost) + sizeof(TokBarriers) + 128 <= 227 * 1024, "shared memory");
        const size_t most1 = tok_smem<false, kFp8>(kTokMax, kMaxTopk, kMost), most2 = tok_smem<true, kFp8>(kTokMax, kMaxTopk, kMost);
        EP_CUDA(allow(tok_kernel<false, kFp8, false, false>, most1));
        if constexpr (kFp8) EP_CUDA(allow(tok_kernel<false, true, false, true>, most1));
        EP_CUDA(allow(tok_kernel<true, kFp8, false, false>, most2));
        EP_CUDA(allow(tok_kernel<true, kFp8, true, false>, most2));
        EP_CUDA(allow(tok_kernel<true, kFp8, false, true>, most2));
        if (dev < kMaxDevicesTracked) known[dev].store(true, std::memory_order_relaxed);
    }
    constexpr int kByte = kFp8 ? 1 : 2;
    CUtensorMap m13, m2;
    ep_status rc = tok_map(&m13, w->w13, (int64_t)a.H * kByte, 2 * (int64_t)a.I, a.E, fn);
    if (rc == EP_OK) rc = tok_map(&m2, w->w2, (int64_t)a.I * kByte, a.H, a.E, fn);
    if (rc != EP_OK) return rc;
    const int tiles1 = (a.I + kTokRows / 2 - 1) / (kTokRows / 2), tiles2 = (a.H + kTokRows - 1) / kTokRows;
    const int k1 = (a.H * kByte + kTokBytes - 1) / kTokBytes, k2 = (a.I * kByte + kTokBytes - 1) / kTokBytes;
    a.split = ws.split;
    a.sums = reinterpret_cast<float*>(mem);
    a.part = reinterpret_cast<float*>(mem + ws.part);
    a.done = reinterpret_cast<uint32_t*>(mem + ws.done);
    a.blocks_k = k1;
    a.ws = w->w13_scales;
    const int64_t items1 = (int64_t)a.list * tiles1 * a.split, items2 = (int64_t)a.list * tiles2 * k2;
    // Each kernel starts while the one before drains: its list and first weights depend on none of the call's.
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    auto config = [&](int64_t blocks, int threads, size_t smem) {
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3((unsigned)blocks);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = st;
        c.attrs = &early;
        c.numAttrs = 1;
        return c;
    };
    auto at_most = [](int64_t n, int64_t most) { return n < most ? n : most; };
    const bool formed = tok_formed(a.T, a.K, a.E, a.H, a.I, kFp8);
    const auto c1 = config(at_most(items1, sms), kTokThreads, tok_smem<false, kFp8>(a.T, a.K, a.list));
    if (kFp8 && formed) {
        a.formed = mem + ws.formed_x;
        a.powers = reinterpret_cast<float*>(mem + ws.powers);
        const auto c0 = config(at_most(((int64_t)a.T * k1 + 7) / 8, 4 * sms), 256, 0);
        if constexpr (kFp8) {
            EP_CUDA(cudaLaunchKernelEx(&c0, form_kernel<false, true>, a));
            EP_CUDA(cudaLaunchKernelEx(&c1, tok_kernel<false, true, false, true>, m13, a));
        }
    } else {
        EP_CUDA(cudaLaunchKernelEx(&c1, tok_kernel<false, kFp8, false, false>, m13, a));
    }
    a.blocks_k = k2;
    a.ws = w->w2_scales;
    const auto c2 = config(at_most(items2, sms), kTokThreads, tok_smem<true, kFp8>(a.T, a.K, a.list));
    if (formed) {
        a.formed = mem + ws.formed_h;
        a.powers = reinterpret_cast<float*>(mem + ws.powers);
        const auto cf = config(at_most(((int64_t)a.T * a.K * k2 + 7) / 8, 4 * sms), 256, 0);
        EP_CUDA(cudaLaunchKernelEx(&cf, form_kernel<true, kFp8>, a));
        EP_CUDA(cudaLaunchKernelEx(&c2, tok_kernel<true, kFp8, false, true>, m2, a));
    } else {
        EP_CUDA(cudaLaunchKernelEx(&c2, a.split > 1 ? tok_kernel<true, kFp8, true, false> : tok_kernel<true, kFp8, false, false>, m2, a));
    }
    return EP_OK;
}

static int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

}  // namespace ep

using namespace ep;

// The sizes that the operator takes; what it refuses needs no workspace.
static ep_status check_sizes(const char* fn, int num_tokens, int num_topk, const ep_moe_weights* w) {
    if (!w) return set_error(EP_ERR_INVALID_ARG, "%s: null weights", fn);
    const int unit = w->w13_scales ? 128 : 32;
    if (num_tokens < 0 || num_tokens > kTokMax) return set_error(EP_ERR_INVALID_ARG, "%s: %d tokens outside 0..%d", fn, num_tokens, kTokMax);
    if (num_topk < 1 || num_topk > kMaxTopk) return set_error(EP_ERR_INVALID_ARG, "%s: top-k %d outside 1..%d", fn, num_topk, kMaxTopk);
    if (w->experts < 1 || w->experts > kMaxExperts) return set_error(EP_ERR_INVALID_ARG, "%s: %d experts", fn, w->experts);
    if (w->hidden < unit || w->hidden % unit || w->inter < unit || w->inter % unit)
        return set_error(EP_ERR_INVALID_ARG, "%s: hidden %d and inter %d must be multiples of %d", fn, w->hidden, w->inter, unit);
    if ((w->w2_scales != nullptr) != (w->w13_scales != nullptr))
        return set_error(EP_ERR_INVALID_ARG, "%s: scales for both weights, or for none", fn);
    // the kernels count channels and work items in 32 bits
    const int list = tok_list(num_tokens, num_topk, w->experts);
    const int64_t bytes1 = (int64_t)w->hidden * (w->w13_scales ? 1 : 2), bytes2 = (int64_t)w->inter * (w->w13_scales ? 1 : 2);
    const int64_t tiles1 = ((int64_t)w->inter + kTokRows / 2 - 1) / (kTokRows / 2), tiles2 = ((int64_t)w->hidden + kTokRows - 1) / kTokRows;
    if (w->hidden > kTokChannelsMost || w->inter > kTokChannelsMost || list * tiles1 * kTokSplitMost > 0x7fffffff ||
        list * tiles2 * ((bytes2 + kTokBytes - 1) / kTokBytes) > 0x7fffffff || num_tokens * ((bytes1 + kTokBytes - 1) / kTokBytes) > 0x7fffffff)
        return set_error(EP_ERR_INVALID_ARG, "%s: %d x %d channels of %d experts are too many", fn, w->hidden, w->inter, list);
    return EP_OK;
}

extern "C" int64_t ep_moe_tokens_workspace(int32_t num_tokens, int32_t num_topk, const ep_moe_weights* w) {
    const int sms = sm_count();
    if (check_sizes("ep_moe_tokens_workspace", num_tokens, num_topk, w) != EP_OK || num_tokens == 0 || sms < 1) return 0;
    return tok_workspace(num_tokens, num_topk, w->experts, w->hidden, w->inter, w->w13_scales != nullptr, sms).bytes;
}

extern "C" ep_status ep_moe_tokens(const void* x, int64_t x_stride, int32_t num_tokens, const int64_t* topk_idx,
                                   const float* topk_weights, int32_t num_topk, const ep_moe_weights* w, void* out,
                                   int64_t out_stride, void* workspace, int64_t workspace_bytes, uint32_t* status_out,
                                   void* stream) {
    const char* fn = "ep_moe_tokens";
    const ep_status sizes = check_sizes(fn, num_tokens, num_topk, w);
    if (sizes != EP_OK) return sizes;
    const bool fp8 = w->w13_scales != nullptr;
    const int H = w->hidden, I = w->inter;
    if (num_tokens == 0) return EP_OK;
    if (!x || !topk_idx || !topk_weights || !out || !w->w13 || !w->w2 || !aligned16(x) || !aligned16(w->w13) || !aligned16(w->w2))
        return set_error(EP_ERR_INVALID_ARG, "%s: null or unaligned (16 bytes: x, weights) pointer", fn);
    if (!aligned_to(topk_idx, 8) || !aligned_to(topk_weights, 4) || !aligned_to(out, 2) || !aligned_to(w->w13_scales, 4) ||
        !aligned_to(w->w2_scales, 4) || !aligned_to(status_out, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: a pointer is not aligned to its elements", fn);
    if (x_stride < H || x_stride % 8 || out_stride < H)
        return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld (a multiple of 8), %lld for %d channels", fn, (long long)x_stride,
                         (long long)out_stride, H);
    const int sms = sm_count();
    if (sms < 1) return set_error(EP_ERR_CUDA, "%s: no CUDA device", fn);
    const TokWorkspace ws = tok_workspace(num_tokens, num_topk, w->experts, H, I, fp8, sms);
    if (!workspace || !aligned16(workspace) || workspace_bytes < ws.bytes)
        return set_error(EP_ERR_CAPACITY, "%s: workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes, (long long)ws.bytes);
    TokArgs a{};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.x_stride = x_stride;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.T = num_tokens;
    a.K = num_topk;
    a.E = w->experts;
    a.H = H;
    a.I = I;
    a.list = tok_list(a.T, a.K, a.E);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_stride = out_stride;
    a.status = status_out;
    uint8_t* mem = static_cast<uint8_t*>(workspace);
    return fp8 ? launch_tokens<true>(a, w, sms, ws, mem, as_stream(stream)) : launch_tokens<false>(a, w, sms, ws, mem, as_stream(stream));
}
