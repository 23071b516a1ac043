// ep_router.cu -- the router around dispatch: logits to topk_idx and topk_weights, the balance loss
// with its per-expert counts, and the gradient of the logits.
//
// A warp per token.  Lane i holds experts i V .. i V + V - 1 of the row in registers, so that the lowest
// expert of equal ones is the first of the lowest lane.
//
// Choice.  key = fp32(logit + bias) or fp32(score + bias), compared as integers in the same order (NaN the largest,
// -inf and what closed groups hold never chosen).  Lane k ends with choice k.  Without a bias and without sums
// over a group both keys choose alike, since the scores grow with the logits; with either they do not.
//
// Balance.  With c_se the choices of expert e in sequence s, m_s = sum_e c_se, n_s the tokens that chose:
//   F_se = coef E c_se / (S m_s n_s),   loss = sum_s sum_e F_se sum_t q_ste,   q: softmax, or sigmoid / its sum
// F is held constant in the gradient, and sum_e q_e = 1, so that F less its mean over e gives the same
// gradient; F - mean = coef (E c_se - m_s) / (S m_s n_s) is formed from integers, and keeps its bits where
// the load is nearly balanced.
//   softmax:  dl_e = q_e (F_e - sum_j F_j q_j);   sigmoid (p, p' = p (1 - p)):  dl_e = p'_e (F_e - sum_j F_j q_j) / sum p
//
// Bound.  Not memory yet (256 experts, fp32: 1 KB a token), but the instructions of a token, some 365 for a choice
// of 8, 570 by groups with a bias, 400 for the gradient, and with that the warps that wait for loads meanwhile:
// route 32768 tokens, 4 of 8 groups, 21 us (79 by maxima over the warp, one choice at a time; issue slots 72 % full),
// by scores 24 (some 610 instructions); without groups 14.5, by scores 18;
// 65536 tokens of 32 sequences: route 29 us, loss 24, gradient 35.  What brought it there: whole sectors a lane (two
// halves of each twice: gradient 49 -> 44), grids of one wave (loss 31 -> 24), two tokens' loads together.  Teams of
// 8 or 16 lanes a token share a row's sums among tokens, but hold 32 or 16 experts a lane, and the registers of that
// cost more than it saves (loss 31 -> 47, 39).
#include <climits>
#include <initializer_list>

#include "ep_tcgen05.cuh"

namespace ep {

constexpr int kRouterThreads = 256, kRouterWarps = kRouterThreads / 32;
constexpr int kRouterMaxExperts = 1024, kRouterMaxGroups = 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // the ordered key of -inf
constexpr uint32_t kAll = 0xffffffffu;
// Blocks that a processor holds at least, which the grids are made for: one more wave costs as much as the first.
template <int V>
constexpr int kPerSm = V <= 8 ? 5 : V == 16 ? 3 : 2;
constexpr int blocks_per_sm(int experts) { return experts <= 256 ? kPerSm<8> : experts <= 512 ? kPerSm<16> : kPerSm<32>; }
constexpr int balance_per_sm(int experts) { return experts <= 256 ? 4 : blocks_per_sm(experts); }

struct RouterArgs {
    const void* logits;
    int64_t stride;
    uint32_t tokens;  // below 2^31, so that a step past them stays within 32 bits
    int E, K, groups, topk_groups;
    int group_size, lanes_log;  // lanes_log: a group is 1 << lanes_log whole lanes; -1: it is not
    bool group_sums;            // a group counts its two largest keys, not the largest alone
    bool normalize;
    int vec;
    float scale;
    const float* bias;
    const uint8_t* mask;
    int64_t* idx;
    float* weights;
};

// Ordered as the floats are.  Adding +0 makes both zeros alike and every NaN the one that sums give, 0x7fffffff,
// whose key is the largest.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : kAll));  // kAll comes back as a NaN
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {  // a NaN counts only where all are
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// This lane's V logits of a row; -inf past the last expert.  vec: the bytes a lane may take at once.  Plain loads: the
// gradient may overwrite the logits.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, int vec, float (&v)[V]) {
    auto unpack = [&](const uint32_t* u, int words, int at) {
#pragma unroll
        for (int i = 0; i < words; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[at + i] = __uint_as_float(u[i]);
            } else {
                v[at + 2 * i] = __uint_as_float(u[i] << 16);
                v[at + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    };
    if constexpr (V * sizeof(T) >= 16) {
        if (vec >= 16) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = -INFINITY;
            constexpr int kWide = V * sizeof(T) >= 32 ? 32 : 16;
            if (kWide == 32 && vec == 32) {
                constexpr int kPer = 32 / sizeof(T);
#pragma unroll
                for (int c = 0; c < V; c += kPer)
                    if (lane * V + c < E) {
                        uint32_t u[8];
                        ld_global_32(row + lane * V + c, u);
                        unpack(u, 8, c);
                    }
            } else {
                constexpr int kPer = 16 / sizeof(T);
#pragma unroll
                for (int c = 0; c < V; c += kPer)
                    if (lane * V + c < E) {
                        const int4 r = ld_na_v4(row + lane * V + c);
                        const uint32_t u[4] = {(uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w};
                        unpack(u, 4, c);
                    }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lane * V + i < E ? (float)row[lane * V + i] : -INFINITY;
}

// e^x for x <= 0.  Rounding x * log2(e) moves the result by |x| 2^-24 of itself, log2(e)'s own rounding by less, and
// the approximate power by 2 units of 2^-23: (|x| + 4) 2^-23 covers it.  Below 2^-126 the result is 0.
__device__ __forceinline__ float exp_of(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}
// sigmoid(l) and its slope, from e^-|l|: neither cancels.
__device__ __forceinline__ float sigmoid_of(float l, float* slope) {
    const float e = exp_of(-fabsf(l)), r = __fdividef(1.0f, 1.0f + e);
    *slope = e * r * r;
    return l < 0.0f ? e * r : r;  // a NaN stays one: r
}

// The scores of a row (-inf past the last expert gives 0): softmax, with *top the largest logit and *by 1 / sum of
// e^(l - top); or sigmoid and its slope, with *by 1 / its sum (0 for a sum of 0).
template <int V, bool kSigmoid>
__device__ __forceinline__ void scores(const float (&l)[V], float (&p)[V], float (&slope)[V], float* top, float* by) {
    if constexpr (kSigmoid) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = sigmoid_of(l[i], &slope[i]);
            s += p[i];
        }
        s = warp_sum(s);
        *by = s != 0.0f ? __fdividef(1.0f, s) : 0.0f;
    } else {
        float m = l[0], s = 0.0f;
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = exp_of(l[i] - m);
            s += p[i];
        }
        s = __fdividef(1.0f, warp_sum(s));
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] *= s;
        *top = m;
        *by = s;
    }
}

// Whether this lane's group stays; a group counts the sum of its two largest keys, or the largest.  Lanes that hold whole parts of
// groups (V divides the group, a power of two of lanes each): the lanes' two largest are merged.
template <int V>
__device__ __forceinline__ bool keep_group(const uint32_t (&key)[V], const RouterArgs& a, int lane) {
    uint32_t hi = key[0], lo = 0;
#pragma unroll
    for (int i = 1; i < V; ++i) {
        lo = max(lo, min(hi, key[i]));
        hi = max(hi, key[i]);
    }
    for (int o = 1; o < 1 << a.lanes_log; o <<= 1) {
        const uint32_t h = __shfl_xor_sync(kAll, hi, o), l = __shfl_xor_sync(kAll, lo, o);
        lo = max(max(lo, l), min(hi, h));
        hi = max(hi, h);
    }
    const uint32_t score = a.group_sums ? ordered(unordered(hi) + unordered(lo)) : hi;
    // lane g: group g's score, taken out as it is chosen
    uint32_t left = __shfl_sync(kAll, score, lane << a.lanes_log & 31);
    if (lane >= a.groups) left = 0;
    bool taken = false;
    for (int i = 0; i < a.topk_groups; ++i) {
        const uint32_t most = __reduce_max_sync(kAll, left);
        if (lane == __ffs(__ballot_sync(kAll, left == most)) - 1) {
            left = 0;
            taken = true;
        }
    }
    return __ballot_sync(kAll, taken) >> (lane >> a.lanes_log) & 1;
}
// Any other groups, one after the other: bit g of the result.
template <int V>
__device__ __forceinline__ uint32_t choose_groups(const uint32_t (&key)[V], const RouterArgs& a, int lane) {
    const int size = a.group_size;
    uint32_t score = 0;  // lane g: group g's
    for (int g = 0; g < a.groups; ++g) {
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i - g * size;
            const uint32_t k = e >= 0 && e < size ? key[i] : 0;
            lo = max(lo, min(hi, k));
            hi = max(hi, k);
        }
        const uint32_t top = __reduce_max_sync(kAll, hi);
        const bool owner = lane == __ffs(__ballot_sync(kAll, hi == top)) - 1;
        const uint32_t next = __reduce_max_sync(kAll, owner ? lo : hi);
        const uint32_t s = a.group_sums ? ordered(unordered(top) + unordered(next)) : top;
        if (lane == g) score = s;
    }
    uint32_t kept = 0;
    for (int i = 0; i < a.topk_groups; ++i) {
        const uint32_t top = __reduce_max_sync(kAll, score);
        const int g = __ffs(__ballot_sync(kAll, score == top)) - 1;
        if (lane == g) score = 0;
        kept |= 1u << g;
    }
    return kept;
}

// The K largest keys by K warp-wide maxima, the first owner giving up its first: any number of candidates.
template <int V>
__device__ __forceinline__ int choose_one_by_one(uint32_t (&key)[V], int K, int lane) {
    int expert = -1;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t most = __reduce_max_sync(kAll, best);
        if (most <= kKeyNegInf) break;
        const int owner = __ffs(__ballot_sync(kAll, best == most)) - 1;
        const int e = __shfl_sync(kAll, lane * V + at, owner);
        if (lane == k) expert = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i == e) key[i] = 0;
    }
    return expert;
}

// Choice k's expert, in lane k: the K-th largest of the lanes' best keys bounds the K-th largest key from below, so that
// the keys from there on, mostly K and a few, are all that has to be ranked: they are listed, a lane each, and a
// candidate's rank is the number of larger ones (a looser bound in fewer steps, the least of the best of 8 runs of lanes,
// leaves 17 of them and takes 31 us for 29).  Equal candidates show as two that want the same place; then the lower
// experts among them count as larger.  Where there are more than 32, the choices are made one by one.
struct RouteList {
    uint32_t key[32];
    int expert[32];
};
template <int V>
__device__ __forceinline__ int choose(uint32_t (&key)[V], int K, int lane, RouteList& list) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    uint32_t least = 0;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {  // equal ones go at once, which only lowers the bound
        least = __reduce_max_sync(kAll, best);
        if (best == least) best = 0;
    }
    least = max(least, kKeyNegInf + 1);
    int total = 0;
    list.key[lane] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool on = key[i] >= least;
        const uint32_t all = __ballot_sync(kAll, on);
        const int to = total + __popc(all & lanemask_lt());
        if (on && to < 32) {
            list.key[to] = key[i];
            list.expert[to] = lane * V + i;
        }
        total += __popc(all);
    }
    if (total > 32) return choose_one_by_one(key, K, lane);
    __syncwarp();
    const uint32_t mine = list.key[lane];
    const int expert = list.expert[lane];
    int rank = 0;
    for (int i = 0; i < total; i += 4) {
        const uint4 other = *reinterpret_cast<const uint4*>(list.key + i);
        rank += other.x > mine;
        rank += other.y > mine;
        rank += other.z > mine;
        rank += other.w > mine;
    }
    __syncwarp();
    if (lane < total) list.expert[rank] = expert;
    __syncwarp();
    const bool lost = lane < total && list.expert[rank] != expert;
    if (__any_sync(kAll, lost)) {
        for (int i = 0; i < total; ++i) {
            const uint32_t other = __shfl_sync(kAll, mine, i);
            const int e = __shfl_sync(kAll, expert, i);
            rank += other == mine && e < expert;
        }
        __syncwarp();
        if (lane < total) list.expert[rank] = expert;
        __syncwarp();
    }
    return lane < total && lane < K ? list.expert[lane] : -1;
}

// What the keys are made of.  By scores, groups are chosen first where topk_groups says so.
enum KeyKind { kByLogits, kByLogitsOfGroups, kByScores };

template <typename T, int V, bool kSigmoid, int kKind>
__global__ void __launch_bounds__(kRouterThreads, kPerSm<V>) route_kernel(const RouterArgs a) {
    __shared__ __align__(16) RouteList lists[kRouterWarps];
    const int lane = threadIdx.x & 31;
    grid_wait();
    grid_launch_next();
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias && lane * V + i < a.E ? a.bias[lane * V + i] : 0.0f;
    for (uint32_t t = blockIdx.x * kRouterWarps + (threadIdx.x >> 5); t < a.tokens; t += gridDim.x * kRouterWarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.stride;
        float l[V];
        load_logits(row, a.E, lane, a.vec, l);
        if (a.mask && !a.mask[t]) {
            if (lane < a.K) {
                a.idx[(int64_t)t * a.K + lane] = -1;
                a.weights[(int64_t)t * a.K + lane] = 0.0f;
            }
            continue;
        }
        uint32_t key[V];  // kKeyNegInf past the last expert
        float most, by;   // of a softmax
        if constexpr (kKind == kByScores) {
            float p[V], slope[V];
            scores<V, kSigmoid>(l, p, slope, &most, &by);
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = l[i] == -INFINITY ? kKeyNegInf : ordered(p[i] + bias[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = ordered(l[i] + bias[i]);  // -inf stays past the last expert
        }
        if (kKind == kByLogitsOfGroups || (kKind == kByScores && a.topk_groups < a.groups)) {
            if (a.lanes_log >= 0) {
                if (!keep_group(key, a, lane))
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = 0;
            } else {
                const uint32_t kept = choose_groups(key, a, lane);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!(kept >> min((lane * V + i) / a.group_size, 31) & 1)) key[i] = 0;
            }
        }
        const int expert = choose(key, a.K, lane, lists[threadIdx.x >> 5]);
        const float logit = expert >= 0 ? (float)row[expert] : -INFINITY;
        float w;
        if (kSigmoid) {
            float slope;
            w = expert >= 0 ? sigmoid_of(logit, &slope) : 0.0f;
            if (a.normalize) w = __fdividef(w, warp_sum(w) + 1e-20f);
        } else if (a.normalize) {
            const float m = warp_max(logit);
            w = expert >= 0 ? exp_of(logit - m) : 0.0f;
            w = __fdividef(w, warp_sum(w));
        } else {
            if constexpr (kKind != kByScores) {
                float p[V], slope[V];
                scores<V, false>(l, p, slope, &most, &by);
            }
            w = exp_of(logit - most) * by;
        }
        if (lane < a.K) {
            a.idx[(int64_t)t * a.K + lane] = expert;
            a.weights[(int64_t)t * a.K + lane] = expert >= 0 ? w * a.scale : 0.0f;
        }
    }
}

// ---- balance loss -------------------------------------------------------------------
struct BalanceArgs {
    const void* logits;
    const int64_t* idx;
    int64_t stride, T;  // tokens of a sequence
    int S, E, K, blocks;  // blocks of a sequence
    int vec;
    float coef;
    // workspace: [S][blocks][E] sums of q and choices, [S][blocks] tokens, [S] losses, the counter of the last block
    float* part;
    int* part_counts;
    int* part_tokens;
    float* seq_loss;
    uint32_t* ticket;
    float* loss;
    int32_t* counts;
    float* factors;
    uint32_t* status;
};

template <typename T, int V, bool kSigmoid>
__global__ void __launch_bounds__(kRouterThreads, V <= 8 ? 4 : kPerSm<V>) balance_kernel(const BalanceArgs a) {
    __shared__ float sums[kRouterMaxExperts];
    __shared__ int hist[kRouterMaxExperts];
    __shared__ int used_tokens;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_wait();
    grid_launch_next();
    for (int e = threadIdx.x; e < a.E; e += kRouterThreads) hist[e] = 0;
    if (threadIdx.x == 0) used_tokens = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    __syncthreads();
    const int s = blockIdx.x / a.blocks, b = blockIdx.x - s * a.blocks;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    int tokens = 0;
    bool bad = false;
    // two tokens at a time, where registers allow it: their loads and sums wait together
    constexpr int kU = V <= 8 ? 2 : 1;
    const int64_t step = (int64_t)a.blocks * kRouterWarps;
    for (int64_t t0 = (int64_t)b * kRouterWarps + warp; t0 < a.T; t0 += kU * step) {
        float l[kU][V], p[V], slope[V], top, by;
        int64_t e[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t t = t0 + u * step, row = s * a.T + t;
            e[u] = -1;
            if (t < a.T) {
                load_logits(static_cast<const T*>(a.logits) + row * a.stride, a.E, lane, a.vec, l[u]);
                if (lane < a.K) e[u] = a.idx[row * a.K + lane];
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const bool chose = e[u] >= 0 && e[u] < a.E;
            bad |= e[u] < -1 || e[u] >= a.E;
            if (chose) atomicAdd(&hist[(int)e[u]], 1);
            if (!__any_sync(kAll, chose)) continue;
            ++tokens;
            scores<V, kSigmoid>(l[u], p, slope, &top, &by);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += kSigmoid ? p[i] * by : p[i];
        }
    }
    if (lane == 0 && tokens) atomicAdd(&used_tokens, tokens);
    for (int w = 0; w < kRouterWarps; ++w) {  // in warp order
        if (warp == w)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                if (e < a.E) sums[e] = w ? sums[e] + acc[i] : acc[i];
            }
        __syncthreads();
    }
    const int64_t at = (int64_t)blockIdx.x * a.E;
    for (int e = threadIdx.x; e < a.E; e += kRouterThreads) {
        a.part[at + e] = sums[e];
        a.part_counts[at + e] = hist[e];
    }
    if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = used_tokens;
    if (bad && a.status) flag(a.status, FLAG_INVALID_TOPK);
}

constexpr int kFinishThreads = 1024;

template <typename T>
__device__ __forceinline__ T warp_total(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// A block per sequence: its counts, factors and loss; the last block to end adds the losses in order.  A thread adds
// every (threads / width)-th block's part of one expert, width: the experts rounded up to a power of two.
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(const BalanceArgs a, int width) {
    __shared__ long long pairs_of[32], tokens_of[32];  // by warp
    __shared__ float loss_of[32];
    __shared__ float sums[kFinishThreads];
    __shared__ int hist[kFinishThreads];
    __shared__ long long all_pairs;
    __shared__ float unit;
    grid_wait();
    grid_launch_next();
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, e = tid & (width - 1);
    const int parts = blockDim.x / width;
    float p = 0.0f;
    int c = 0;
    if (e < a.E)
#pragma unroll 4
        for (int b = tid / width; b < a.blocks; b += parts) {
            const int64_t at = ((int64_t)s * a.blocks + b) * a.E + e;
            p += a.part[at];
            c += a.part_counts[at];
        }
    long long tokens = 0;
    for (int b = tid; b < a.blocks; b += blockDim.x) tokens += a.part_tokens[(int64_t)s * a.blocks + b];
    sums[tid] = p;
    hist[tid] = c;
    const long long pairs = warp_total((long long)c);
    tokens = warp_total(tokens);
    if (lane == 0) {
        pairs_of[warp] = pairs;
        tokens_of[warp] = tokens;
    }
    __syncthreads();
    if (warp == 0) {
        const long long m = warp_total(lane < warps ? pairs_of[lane] : 0ll), n = warp_total(lane < warps ? tokens_of[lane] : 0ll);
        if (lane == 0) {  // coef / (S m n), the same for every expert: in 64 bits, which one thread is enough for
            all_pairs = m;
            unit = m ? (float)((double)a.coef / ((double)a.S * (double)m * (double)n)) : 0.0f;
        }
    }
    __syncthreads();
    float loss = 0.0f;
    if (tid < a.E) {  // the first part's thread
        for (int i = tid + width; i < (int)blockDim.x; i += width) {
            p += sums[i];
            c += hist[i];
        }
        a.counts[(int64_t)s * a.E + e] = c;
        a.factors[(int64_t)s * a.E + e] = unit * (float)((long long)c * a.E - all_pairs);
        loss = unit * (float)((long long)c * a.E) * p;
    }
    loss = warp_total(loss);
    if (lane == 0) loss_of[warp] = loss;
    __syncthreads();
    if (warp != 0) return;
    loss = warp_total(lane < warps ? loss_of[lane] : 0.0f);
    bool last = false;
    if (lane == 0) {
        a.seq_loss[s] = loss;
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == (uint32_t)a.S - 1;
    }
    if (!__any_sync(kAll, last)) return;
    __threadfence();
    float sum = 0.0f;
    for (int i = lane; i < a.S; i += 32) sum += __ldcg(a.seq_loss + i);
    sum = warp_total(sum);
    if (lane == 0) *a.loss = sum;
}

// ---- gradient of the logits -----------------------------------------------------------
struct RouterBackArgs {
    const void* logits;
    const int64_t* idx;
    const float* dweights;  // null: none
    const float* factors;   // null: no balance loss
    const float* dloss;
    void* dlogits;
    int64_t stride, dstride;
    uint32_t tokens, T;
    int E, K;
    bool normalize;
    int vec, dvec, fvec;
    float scale;
    uint32_t* status;
};

template <typename T, int V>
__device__ __forceinline__ void store_logits(T* row, int E, int lane, int vec, const float (&v)[V]) {
    constexpr int kWords = V * sizeof(T) / 4;
    if constexpr (V * sizeof(T) >= 16) {
        if (vec >= 16) {
            uint32_t u[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) {
                    u[i] = __float_as_uint(v[i]);
                } else {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
            if (kWords >= 8 && vec == 32) {
                constexpr int kPer = 32 / sizeof(T);
#pragma unroll
                for (int c = 0; c < kWords / 8; ++c)
                    if (lane * V + c * kPer < E) st_global_32(row + lane * V + c * kPer, u + c * 8);
            } else {
                constexpr int kPer = 16 / sizeof(T);
#pragma unroll
                for (int c = 0; c < kWords / 4; ++c)
                    if (lane * V + c * kPer < E)
                        st_na_v4(row + lane * V + c * kPer, make_int4((int)u[4 * c], (int)u[4 * c + 1], (int)u[4 * c + 2], (int)u[4 * c + 3]));
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < E) row[lane * V + i] = (T)v[i];
}

template <int V>
__device__ __forceinline__ void add_shared(const float* p, float (&d)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            d[i] += v.x, d[i + 1] += v.y, d[i + 2] += v.z, d[i + 3] += v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += p[i];
    }
}

// This lane's V factors; 0 past the last expert.  Cached: a sequence's tokens share them.  Plain loads: the kernel before
// may still write them when this one is launched.
template <int V>
__device__ __forceinline__ void load_factors(const float* row, int E, int lane, int vec, float (&f)[V]) {
    if constexpr (V % 4 == 0) {
        if (vec >= 16) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int e = lane * V + i;
                const float4 v = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = lane * V + i < E ? row[lane * V + i] : 0.0f;
}

template <typename T, int V, bool kSigmoid>
__global__ void __launch_bounds__(kRouterThreads, V <= 8 ? 4 : kPerSm<V>) router_backward_kernel(const RouterBackArgs a) {
    __shared__ __align__(16) float rows[kRouterWarps][32 * V];
    const int lane = threadIdx.x & 31;
    float* mine = rows[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i * 32 + lane] = 0.0f;
    __syncwarp();
    grid_wait();
    grid_launch_next();
    const float dloss = a.factors ? *a.dloss : 0.0f;
    // softmax of the whole row, or sigmoid: for the balance loss, and for weights that are not normalised
    const bool whole = a.factors || (!kSigmoid && !a.normalize);
    bool bad = false;
    // two tokens at a time, where registers allow it: their loads wait together
    constexpr int kU = V <= 8 ? 2 : 1;
    const uint32_t step = gridDim.x * kRouterWarps;
    for (uint32_t t0 = blockIdx.x * kRouterWarps + (threadIdx.x >> 5); t0 < a.tokens; t0 += kU * step) {
      float rows_l[kU][V], rows_g[kU], rows_logit[kU];
      int rows_e[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t t = t0 + u * step;
        rows_e[u] = -1;
        rows_g[u] = 0.0f;
        if (t >= a.tokens) continue;
        if (whole) load_logits(static_cast<const T*>(a.logits) + t * a.stride, a.E, lane, a.vec, rows_l[u]);
        if (lane < a.K) {
            const int64_t i = a.idx[(int64_t)t * a.K + lane];
            bad |= i < -1 || i >= a.E;
            rows_e[u] = i >= 0 && i < a.E ? (int)i : -1;
            if (a.dweights) rows_g[u] = a.dweights[(int64_t)t * a.K + lane] * a.scale;
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        rows_logit[u] = a.dweights && rows_e[u] >= 0 ? (float)static_cast<const T*>(a.logits)[(t0 + u * step) * a.stride + rows_e[u]] : -INFINITY;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t t = t0 + u * step;
        if (t >= a.tokens) break;
        const float(&l)[V] = rows_l[u];
        const int e = rows_e[u];
        const float logit = rows_logit[u], g = e >= 0 ? rows_g[u] : 0.0f;
        T* out = static_cast<T*>(a.dlogits) + t * a.dstride;
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = 0.0f;
        if (!__any_sync(kAll, e >= 0)) {  // a padded token
            store_logits(out, a.E, lane, a.dvec, d);
            continue;
        }
        // the chosen experts' share of the gradient, in lane k for choice k
        float near = 0.0f, inner = 0.0f;
        if (whole) {
            float p[V], slope[V], top, by;
            scores<V, kSigmoid>(l, p, slope, &top, &by);
            if (a.factors) {
                float fv[V], sum = 0.0f;
                load_factors(a.factors + (int64_t)(t / a.T) * a.E, a.E, lane, a.fvec, fv);
#pragma unroll
                for (int i = 0; i < V; ++i) sum = fmaf(fv[i], p[i], sum);
                sum = warp_sum(sum) * (kSigmoid ? by : 1.0f);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] = dloss * (fv[i] - sum) * (kSigmoid ? slope[i] * by : p[i]);
            }
            if (!kSigmoid && !a.normalize && a.dweights) {
                near = e >= 0 ? exp_of(logit - top) * by * g : 0.0f;
                inner = warp_sum(near);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] -= p[i] * inner;
            }
        }
        if (a.dweights && (kSigmoid || a.normalize)) {
            if (kSigmoid) {
                float slope = 0.0f;
                float w = e >= 0 ? sigmoid_of(logit, &slope) : 0.0f;
                if (e < 0) slope = 0.0f;
                if (a.normalize) {
                    const float by = __fdividef(1.0f, warp_sum(w) + 1e-20f);
                    inner = warp_sum(g * w * by);
                    near = slope * (g - inner) * by;
                } else {
                    near = slope * g;
                }
            } else {
                const float m = warp_max(logit);
                float w = e >= 0 ? exp_of(logit - m) : 0.0f;
                w = __fdividef(w, warp_sum(w));
                inner = warp_sum(w * g);
                near = w * (g - inner);
            }
            if (e < 0) near = 0.0f;
        }
        if (a.dweights) {
            // choice k's share to the lane that holds its expert, by a row of shared memory that is 0 between tokens;
            // a token that names an expert twice adds the shares in the order of the choices
            if (e >= 0) mine[e] = __int_as_float(lane);
            __syncwarp();
            const bool twice = e >= 0 && __float_as_int(mine[e]) != lane;
            __syncwarp();
            if (!__any_sync(kAll, twice)) {
                if (e >= 0) mine[e] = near;
            } else {
                if (e >= 0) mine[e] = 0.0f;
                for (int k = 0; k < a.K; ++k) {
                    __syncwarp();
                    if (lane == k && e >= 0) mine[e] += near;
                }
            }
            __syncwarp();
            add_shared<V>(mine + lane * V, d);
            __syncwarp();
            if (e >= 0) mine[e] = 0.0f;
            __syncwarp();
        }
        store_logits(out, a.E, lane, a.dvec, d);
      }
    }
    if (bad && a.status) flag(a.status, FLAG_INVALID_TOPK);
}

// ---- host -------------------------------------------------------------------------
// The kernel for these experts (lanes hold 1, 2, 4, .. 32 each), type of logits and scoring.
#define EP_BY_EXPERTS(kernel, T, sig, E)                                                     \
    ((E) <= 32    ? kernel<T, 1, sig>                                                        \
     : (E) <= 64  ? kernel<T, 2, sig>                                                        \
     : (E) <= 128 ? kernel<T, 4, sig>                                                        \
     : (E) <= 256 ? kernel<T, 8, sig>                                                        \
     : (E) <= 512 ? kernel<T, 16, sig>                                                       \
                  : kernel<T, 32, sig>)
#define EP_ROUTER_KERNEL(kernel, r)                                                                                     \
    ((r)->logits_type == EP_F32                                                                                         \
         ? ((r)->scoring == EP_SIGMOID ? EP_BY_EXPERTS(kernel, float, true, (r)->experts)                               \
                                       : EP_BY_EXPERTS(kernel, float, false, (r)->experts))                             \
         : ((r)->scoring == EP_SIGMOID ? EP_BY_EXPERTS(kernel, __nv_bfloat16, true, (r)->experts)                       \
                                       : EP_BY_EXPERTS(kernel, __nv_bfloat16, false, (r)->experts)))

template <typename T, int V, bool kSigmoid>
constexpr auto route_all = route_kernel<T, V, kSigmoid, kByLogits>;
template <typename T, int V, bool kSigmoid>
constexpr auto route_groups = route_kernel<T, V, kSigmoid, kByLogitsOfGroups>;
template <typename T, int V, bool kSigmoid>
constexpr auto route_scores = route_kernel<T, V, kSigmoid, kByScores>;

static ep_status check_router(const char* fn, const ep_router* r, const void* logits, int64_t stride) {
    if (!r) return set_error(EP_ERR_INVALID_ARG, "%s: null descriptor", fn);
    if (r->experts < 1 || r->experts > kRouterMaxExperts || r->topk < 1 || r->topk > kMaxTopk || r->topk > r->experts)
        return set_error(EP_ERR_INVALID_ARG, "%s: %d of %d experts (at most %d of %d)", fn, r->topk, r->experts, kMaxTopk, kRouterMaxExperts);
    if (r->tokens < 0 || r->tokens > (int64_t)INT_MAX) return set_error(EP_ERR_INVALID_ARG, "%s: %lld tokens", fn, (long long)r->tokens);
    if (r->logits_type < 0 || r->logits_type > EP_F32 || r->scoring < 0 || r->scoring > EP_SIGMOID)
        return set_error(EP_ERR_INVALID_ARG, "%s: type %d, scoring %d", fn, r->logits_type, r->scoring);
    if (r->tokens > 0 && (!logits || !aligned_to(logits, r->logits_type == EP_F32 ? 4 : 2) || (r->tokens > 1 && stride < r->experts)))
        return set_error(EP_ERR_INVALID_ARG, "%s: logits, rows %lld elements apart for %d experts", fn, (long long)stride, r->experts);
    return EP_OK;
}
// Bytes that a lane may take of these rows at once: 32, 16, or one expert's.
static int by_vectors(int experts, int type, const void* p, int64_t stride) {
    const int size = type == EP_F32 ? 4 : 2;
    for (const int bytes : {32, 16})
        if (aligned_to(p, bytes) && stride * size % bytes == 0 && experts * size % bytes == 0) return bytes;
    return size;
}
static ep_status router_blocks(const ep_router* r, int per_sm, int64_t* blocks) {
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const int64_t most = (int64_t)sms * per_sm, need = (r->tokens + kRouterWarps - 1) / kRouterWarps;
    *blocks = need < most ? need : most;
    return EP_OK;
}

// Blocks of one sequence: one wave over all of them (928 blocks for 912 places: 31 us for 24), each with two tokens a
// warp or more.
static int balance_blocks(int64_t S, int64_t T, int experts, int sms) {
    int64_t b = (int64_t)sms * balance_per_sm(experts) / S;
    const int64_t most = (T + 2 * kRouterWarps - 1) / (2 * kRouterWarps);
    if (b > most) b = most;
    return b < 1 ? 1 : (int)b;
}
static int64_t balance_bytes(int64_t S, int blocks, int E) { return (S * blocks * (2 * (int64_t)E + 1) + S + 1) * 4; }

}  // namespace ep

using namespace ep;

extern "C" ep_status ep_route(const ep_router* r, const void* logits, int64_t logits_stride, const float* bias, const uint8_t* mask,
                              int64_t* topk_idx, float* topk_weights, void* stream) {
    const char* fn = "ep_route";
    EP_TRY(check_router(fn, r, logits, logits_stride));
    if (r->groups < 1 || r->groups > kRouterMaxGroups || r->experts % r->groups || r->topk_groups < 1 || r->topk_groups > r->groups ||
        r->topk > r->topk_groups * (r->experts / r->groups))
        return set_error(EP_ERR_INVALID_ARG, "%s: %d of %d groups (at most %d) of %d experts for %d choices", fn, r->topk_groups, r->groups,
                         kRouterMaxGroups, r->experts, r->topk);
    if (r->keys < 0 || r->keys > EP_KEYS_SCORES || r->group_keys < 0 || r->group_keys > 2)
        return set_error(EP_ERR_INVALID_ARG, "%s: keys %d, %d keys of a group", fn, r->keys, r->group_keys);
    if (r->tokens == 0) return EP_OK;
    if (!topk_idx || !topk_weights || !aligned_to(topk_idx, 8) || !aligned_to(topk_weights, 4) || !aligned_to(bias, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: topk_idx, topk_weights and bias aligned to their elements", fn);
    int64_t blocks = 0;
    EP_TRY(router_blocks(r, blocks_per_sm(r->experts), &blocks));
    int held = 1, lanes_log = -1;  // experts a lane holds, as EP_BY_EXPERTS
    while (32 * held < r->experts) held *= 2;
    const int size = r->experts / r->groups;
    if (size % held == 0 && (size / held & (size / held - 1)) == 0)
        for (lanes_log = 0; held << lanes_log < size;) ++lanes_log;
    const RouterArgs a = {logits, logits_stride, (uint32_t)r->tokens, r->experts, r->topk, r->groups, r->topk_groups, size, lanes_log,
                          size > 1 && r->group_keys != 1, r->normalize != 0,
                          by_vectors(r->experts, r->logits_type, logits, logits_stride), r->scale, bias, mask, topk_idx, topk_weights};
    return launch_next(r->keys == EP_KEYS_SCORES    ? EP_ROUTER_KERNEL(route_scores, r)
                       : r->topk_groups < r->groups ? EP_ROUTER_KERNEL(route_groups, r)
                                                    : EP_ROUTER_KERNEL(route_all, r),
                       blocks, kRouterThreads, stream, a);
}

extern "C" int64_t ep_balance_loss_workspace(const ep_router* r, int32_t sequences) {
    int dev = 0, sms = 0;
    if (!r || sequences < 1 || r->experts < 1 || r->experts > kRouterMaxExperts || r->tokens < 0 || r->tokens > INT_MAX ||
        cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return balance_bytes(sequences, balance_blocks(sequences, r->tokens / sequences, r->experts, sms), r->experts);
}

extern "C" ep_status ep_balance_loss(const ep_router* r, const void* logits, int64_t logits_stride, const int64_t* topk_idx,
                                     int32_t sequences, float coef, float* loss, int32_t* counts, float* factors, void* workspace,
                                     int64_t workspace_bytes, uint32_t* status_out, void* stream) {
    const char* fn = "ep_balance_loss";
    EP_TRY(check_router(fn, r, logits, logits_stride));
    if (sequences < 1 || r->tokens % sequences)
        return set_error(EP_ERR_INVALID_ARG, "%s: %lld tokens in %d sequences", fn, (long long)r->tokens, sequences);
    if ((r->tokens > 0 && !topk_idx) || !loss || !counts || !factors || !aligned_to(topk_idx, 8) || !aligned_to(loss, 4) ||
        !aligned_to(counts, 4) || !aligned_to(factors, 4) || !aligned_to(status_out, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: topk_idx, loss, counts and factors, aligned to their elements", fn);
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const int64_t T = r->tokens / sequences;
    const int blocks = balance_blocks(sequences, T, r->experts, sms);
    const int64_t need = balance_bytes(sequences, blocks, r->experts);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
        return set_error(EP_ERR_INVALID_ARG, "%s: workspace of %lld bytes (16-byte aligned), %lld needed", fn, (long long)workspace_bytes, (long long)need);
    if (r->tokens * r->topk > INT_MAX) return set_error(EP_ERR_INVALID_ARG, "%s: %lld tokens with %d choices", fn, (long long)r->tokens, r->topk);
    if ((int64_t)sequences * blocks > INT_MAX) return set_error(EP_ERR_INVALID_ARG, "%s: %d sequences", fn, sequences);
    const int64_t n = (int64_t)sequences * blocks * r->experts;
    float* ws = static_cast<float*>(workspace);
    const BalanceArgs a = {logits, topk_idx, logits_stride, T, sequences, r->experts, r->topk, blocks, by_vectors(r->experts, r->logits_type, logits, logits_stride), coef,
                           ws, reinterpret_cast<int*>(ws + n), reinterpret_cast<int*>(ws + 2 * n),
                           ws + 2 * n + (int64_t)sequences * blocks, reinterpret_cast<uint32_t*>(ws + 2 * n + (int64_t)sequences * blocks + sequences),
                           loss, counts, factors, status_out};
    EP_TRY(launch_next(EP_ROUTER_KERNEL(balance_kernel, r), (int64_t)sequences * blocks, kRouterThreads, stream, a));
    int width = 32, parts = 1;
    while (width < r->experts) width *= 2;
    while (parts < blocks && width * parts < kFinishThreads) parts *= 2;
    return launch_next(balance_finish_kernel, sequences, width * parts, stream, a, width);
}

extern "C" ep_status ep_router_backward(const ep_router* r, const void* logits, int64_t logits_stride, const int64_t* topk_idx,
                                        const float* dweights, const float* factors, int32_t sequences, const float* dloss, void* dlogits,
                                        int64_t dlogits_stride, uint32_t* status_out, void* stream) {
    const char* fn = "ep_router_backward";
    EP_TRY(check_router(fn, r, logits, logits_stride));
    if (r->tokens == 0) return EP_OK;
    if (!factors != !dloss) return set_error(EP_ERR_INVALID_ARG, "%s: factors come with the loss's gradient", fn);
    if (!factors && !dweights) return set_error(EP_ERR_INVALID_ARG, "%s: no gradient comes in", fn);
    if (factors && (sequences < 1 || r->tokens % sequences))
        return set_error(EP_ERR_INVALID_ARG, "%s: %lld tokens in %d sequences", fn, (long long)r->tokens, sequences);
    if (!topk_idx || !dlogits || !aligned_to(topk_idx, 8) || !aligned_to(dweights, 4) || !aligned_to(factors, 4) || !aligned_to(dloss, 4) ||
        !aligned_to(dlogits, r->logits_type == EP_F32 ? 4 : 2) || !aligned_to(status_out, 4) || (r->tokens > 1 && dlogits_stride < r->experts))
        return set_error(EP_ERR_INVALID_ARG, "%s: topk_idx, gradients and dlogits (rows %lld elements apart), aligned to their elements", fn,
                         (long long)dlogits_stride);
    int64_t blocks = 0;
    EP_TRY(router_blocks(r, balance_per_sm(r->experts), &blocks));
    const RouterBackArgs a = {logits, topk_idx, dweights, factors, dloss, dlogits, logits_stride, dlogits_stride, (uint32_t)r->tokens,
                              (uint32_t)(factors ? r->tokens / sequences : 1), r->experts, r->topk, r->normalize != 0, by_vectors(r->experts, r->logits_type, logits, logits_stride),
                              by_vectors(r->experts, r->logits_type, dlogits, dlogits_stride), by_vectors(r->experts, EP_F32, factors, r->experts), r->scale, status_out};
    return launch_next(EP_ROUTER_KERNEL(router_backward_kernel, r), blocks, kRouterThreads, stream, a);
}
