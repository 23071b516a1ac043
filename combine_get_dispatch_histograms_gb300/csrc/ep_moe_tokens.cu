// ep_moe_tokens.cu -- a whole mixture-of-experts layer for up to 64 tokens, in
// two kernels, without the dispatch / permute / combine round trip.
//
// Mathematics.  For token t with choices e = topk_idx[t][k], weights v[t][k]:
//   h[t,e] = silu(Wg[e] x[t]) * (Wu[e] x[t]),   out[t] = sum_k v[t][k] * W2[e] h[t,e].
// Kernel 1 computes h for every (token, expert) pair, kernel 2 the weighted sum.
//
// Bound.  Each weight byte of the experts that any token chose is read once;
// with one to a few tokens per expert the operations are far below the tensor
// cores' rate, so the kernels are bound by that stream.  One block per SM,
// every thread feeds itself through a private ring of asynchronous 16-byte
// copies (no barrier between copy and use), and 16 warps split the channels of
// the reduction.  The product is the register-operand m16n8k16 form with the
// weights as its 16 rows and up to 8 tokens as its columns: a warp's weights go
// from shared memory through registers (e4m3 to bf16, exact) straight into it,
// where a tensor-memory product would need them back in shared memory.  The
// order of k inside a product is free, so each thread's 16 consecutive bytes
// of a weight row are its fragments and no data moves between threads.
//
// Work items are (expert, 16 channels of gate and up) and (32 output channels,
// expert); each block takes a contiguous run of them, equal to within one.
#include <atomic>
#include <type_traits>

#include "ep_fp8.cuh"

namespace ep {

constexpr int kTokMax = 64;                 // tokens of a call: an expert's tokens are one 64-bit mask
constexpr int kTokThreads = 512;
constexpr int kTokWarps = kTokThreads / 32;
constexpr int kTokRing = 4;                 // copies in flight per thread: kTokRing - 1 stages
constexpr int kTokStage = 64;               // bytes of a weight row per stage
constexpr int kTokRows = 32;                // weight rows of an item
constexpr int kTokSlots = 16;               // tokens of a pass over an item's weights
constexpr int kPartStride = kTokSlots + 1;  // floats: consecutive rows fall into other banks
constexpr int kPartFloats = kTokWarps * kTokRows * kPartStride;

struct TokArgs {
    const __nv_bfloat16* x;
    int64_t x_stride;
    const int64_t* topk_idx;
    const float* topk_weights;
    int T, K, E, H, I;
    const uint8_t* w;       // w13 in kernel 1, w2 in kernel 2
    const float* ws;        // their scales (e4m3 only)
    int stages;             // of a weight row
    int warps;              // that share a row's stages
    int list;               // entries of the expert list: min(E, T * K)
    __nv_bfloat16 *h_hi, *h_lo;  // [pairs][I]: h as the sum of two bf16, 16 bits of mantissa
    float* part;            // [blocks][2][T][kTokRows] sums of a chunk that several blocks share
    uint32_t* done;         // [H / kTokRows] blocks that have written theirs
    __nv_bfloat16* out;
    int64_t out_stride;
    uint32_t* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 codes to two bf16 pairs; exact, as bf16 holds every e4m3 value.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
    const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
    const __nv_bfloat162 ba = __floats2bfloat162_rn(fa.x, fa.y), bb = __floats2bfloat162_rn(fb.x, fb.y);
    lo = *reinterpret_cast<const uint32_t*>(&ba);
    hi = *reinterpret_cast<const uint32_t*>(&bb);
}

struct TokShared {
    uint8_t* ring;      // [kTokRing][4][kTokThreads] 16-byte pieces
    float* part;        // [2][kPartFloats]
    float* acc;         // [T][kTokRows] (kernel 2)
    float* weight;      // [pairs] (kernel 2)
    uint16_t* expert;   // [list]
    uint16_t* base;     // [list + 1]: pairs of entry i are base[i] .. base[i + 1] - 1
    uint8_t* token;     // [pairs]
};

__host__ __device__ inline size_t tok_smem(int T, int K, int list) {
    const size_t pairs = (size_t)T * K;
    return (size_t)kTokRing * 4 * 16 * kTokThreads + 2 * sizeof(float) * kPartFloats + sizeof(float) * T * kTokRows +
           sizeof(float) * pairs + sizeof(uint16_t) * (2 * list + 2) + pairs + 16;
}

// The experts that some token chose, ascending, and their tokens, ascending.
// Every block builds the list for itself.  Returns the number of experts.
template <bool kDown>
__device__ __forceinline__ int build_list(const TokArgs& a, const TokShared& s) {
    __shared__ int scan[kTokWarps];
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(s.part);       // [E], 32 KB at most
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
    int sum = 0;  // experts in the high half, pairs in the low: both at most 2048
    for (int e = e0; e < e1; ++e) sum += mask[e] ? (1 << 16) + __popcll(mask[e]) : 0;
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
    for (int w = 0; w < kTokWarps; ++w) {
        if (w < warp) at += scan[w];
        total += scan[w];
    }
    for (int e = e0; e < e1; ++e) {
        unsigned long long m = mask[e];
        if (!m) continue;
        const int i = at >> 16;
        int p = at & 0xffff;
        s.expert[i] = (uint16_t)e;
        s.base[i] = (uint16_t)p;
        at += (1 << 16) + __popcll(m);
        for (; m; m &= m - 1, ++p) {
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

// kDown: kernel 2.  kFp8: e4m3 weights with block scales, otherwise bf16.
template <bool kDown, bool kFp8>
__global__ void __launch_bounds__(kTokThreads, 1) tok_kernel(const TokArgs a) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ int last;
    TokShared s;
    s.ring = dyn;
    s.part = reinterpret_cast<float*>(dyn + kTokRing * 4 * 16 * kTokThreads);
    s.acc = s.part + 2 * kPartFloats;
    s.weight = s.acc + a.T * kTokRows;
    s.expert = reinterpret_cast<uint16_t*>(s.weight + a.T * a.K);
    s.base = s.expert + a.list;
    s.token = reinterpret_cast<uint8_t*>(s.base + a.list + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;

    if constexpr (!kDown) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (blockIdx.x == 0)
            for (int i = tid; i < a.H / kTokRows; i += kTokThreads) a.done[i] = 0;
    }
    const int A = build_list<kDown>(a, s);

    const int chunks = kDown ? a.H / kTokRows : a.I / (kTokRows / 2);
    const int64_t total = (int64_t)A * chunks;
    const int64_t blocks = total < gridDim.x ? (total > 0 ? total : 1) : gridDim.x;  // each has an item; the rest are idle
    const bool idle = blockIdx.x >= blocks;
    const int64_t i0 = idle ? total : total * blockIdx.x / blocks, i1 = idle ? total : total * (blockIdx.x + 1) / blocks;
    const int64_t row_bytes = (int64_t)a.stages * kTokStage;
    const int64_t rows = kDown ? a.H : 2 * (int64_t)a.I;  // of one expert
    const int KB = (a.stages + 1) / 2;                    // scale blocks of a row (e4m3)
    const int outer = kDown ? A : chunks;                 // length of the inner index of an item
    const int my_stages = warp < a.warps ? (a.stages - warp + a.warps - 1) / a.warps : 0;

    // ---- copies: stage after stage of pass after pass of item after item ----------
    int64_t c_item = i0;
    int c_hi = outer ? (int)(i0 / outer) : 0, c_lo = outer ? (int)(i0 % outer) : 0, c_pass = 0, c_j = 0, c_slot = 0;
    const uint8_t* c_row = nullptr;
    auto locate = [&] {  // the thread's first weight row of the item, at its 16 bytes of a stage
        const int e = s.expert[kDown ? c_lo : c_hi], chunk = kDown ? c_hi : c_lo;
        c_row = a.w + ((int64_t)e * rows + chunk * (kDown ? 32 : 16) + g) * row_bytes + q * 16;
    };
    if (c_item < i1) locate();
    const int64_t up = kDown ? 8 * row_bytes : a.I * row_bytes;   // rows 8..15 of a product
    const int64_t next = kDown ? 16 * row_bytes : 8 * row_bytes;  // the second product's rows
    const uint32_t ring = smem_u32(s.ring) + tid * 16;
    auto copy = [&] {
        if (c_item < i1 && my_stages > 0) {
            const uint8_t* p = c_row + (int64_t)(warp + c_j * a.warps) * kTokStage;
            const uint32_t d = ring + c_slot * (4 * 16 * kTokThreads);
            cp_async16(d, p);
            cp_async16(d + 16 * kTokThreads, p + up);
            cp_async16(d + 32 * kTokThreads, p + next);
            cp_async16(d + 48 * kTokThreads, p + next + up);
            c_slot = c_slot + 1 == kTokRing ? 0 : c_slot + 1;
            if (++c_j == my_stages) {
                c_j = 0;
                const int i = kDown ? c_lo : c_hi;
                if (++c_pass * kTokSlots >= s.base[i + 1] - s.base[i]) {
                    c_pass = 0;
                    ++c_item;
                    if (++c_lo == outer) {
                        c_lo = 0;
                        ++c_hi;
                    }
                    if (c_item < i1) locate();
                }
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < kTokRing - 1; ++i) copy();

    if constexpr (kDown) asm volatile("griddepcontrol.wait;" ::: "memory");  // h and the counters of kernel 1

    if (kDown && A == 0)
        for (int64_t i = blockIdx.x * (int64_t)kTokThreads + tid; i < (int64_t)a.T * a.H; i += (int64_t)gridDim.x * kTokThreads)
            a.out[i / a.H * a.out_stride + i % a.H] = __float2bfloat16_rn(0.0f);

    int slot = 0, buf = 0;
    int hi = outer ? (int)(i0 / outer) : 0, lo = outer ? (int)(i0 % outer) : 0;
    for (int64_t item = i0; item < i1; ++item) {
        const int ai = kDown ? lo : hi, chunk = kDown ? hi : lo;
        const int e = s.expert[ai], p0 = s.base[ai], m = s.base[ai + 1] - p0;
        const float* sc = nullptr;
        int64_t sc_up = 0;
        if constexpr (kFp8) {
            sc = a.ws + ((int64_t)e * (rows / 128) + (kDown ? chunk * 32 : chunk * 16) / 128) * KB;
            sc_up = kDown ? 0 : (int64_t)(a.I / 128) * KB;
        }
        for (int first = 0; first < m; first += kTokSlots) {
            const int cnt = min(kTokSlots, m - first);
            float tot[2][2][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) (&tot[0][0][0])[i] = 0.0f;

            auto pass = [&](auto nt_tag) {
                constexpr int NT = decltype(nt_tag)::value;
                constexpr int kElems = kFp8 ? 16 : 8;          // of a thread's 16 bytes
                constexpr int kB = kDown ? 2 : 1;              // h comes as two bf16
                const __nv_bfloat16* xb[NT][kB];
                bool have[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    have[n] = g + 8 * n < cnt;
                    const int pair = p0 + first + (have[n] ? g + 8 * n : 0);
                    if constexpr (kDown) {
                        xb[n][0] = a.h_hi + (int64_t)pair * a.I + q * kElems;
                        xb[n][1] = a.h_lo + (int64_t)pair * a.I + q * kElems;
                    } else {
                        xb[n][0] = a.x + s.token[pair] * a.x_stride + q * kElems;
                    }
                }
                for (int j = 0; j < my_stages; ++j) {
                    const int u = warp + j * a.warps;
                    uint32_t b[NT][kB][kElems / 2];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int z = 0; z < kB; ++z)
#pragma unroll
                            for (int i = 0; i < kElems / 8; ++i) {
                                int4 v = make_int4(0, 0, 0, 0);
                                if (have[n]) v = *reinterpret_cast<const int4*>(xb[n][z] + u * (4 * kElems) + i * 8);
                                b[n][z][4 * i] = v.x;
                                b[n][z][4 * i + 1] = v.y;
                                b[n][z][4 * i + 2] = v.z;
                                b[n][z][4 * i + 3] = v.w;
                            }
                    float s0 = 1.0f, s1 = 1.0f;
                    if constexpr (kFp8) {
                        s0 = __ldg(sc + (u >> 1));
                        s1 = kDown ? s0 : __ldg(sc + sc_up + (u >> 1));
                    }
                    cp_async_wait<kTokRing - 2>();
                    const uint8_t* src = s.ring + slot * (4 * 16 * kTokThreads) + tid * 16;
                    slot = slot + 1 == kTokRing ? 0 : slot + 1;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int4 r0 = *reinterpret_cast<const int4*>(src + (2 * t) * 16 * kTokThreads);
                        const int4 r1 = *reinterpret_cast<const int4*>(src + (2 * t + 1) * 16 * kTokThreads);
                        const uint32_t w0[4] = {(uint32_t)r0.x, (uint32_t)r0.y, (uint32_t)r0.z, (uint32_t)r0.w};
                        const uint32_t w1[4] = {(uint32_t)r1.x, (uint32_t)r1.y, (uint32_t)r1.z, (uint32_t)r1.w};
                        if constexpr (kFp8) {
                            float blk[NT][4] = {};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_bf16(w0[k], a0, a2);
                                e4m3x4_to_bf16(w1[k], a1, a3);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int z = 0; z < kB; ++z)
                                        mma_bf16(blk[n], a0, a1, a2, a3, b[n][z][2 * k], b[n][z][2 * k + 1]);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i) tot[t][n][i] = fmaf(blk[n][i], i < 2 ? s0 : s1, tot[t][n][i]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int z = 0; z < kB; ++z)
                                        mma_bf16(tot[t][n], w0[2 * k], w1[2 * k], w0[2 * k + 1], w1[2 * k + 1],
                                                 b[n][z][2 * k], b[n][z][2 * k + 1]);
                        }
                    }
                    copy();
                }
            };
            if (cnt > 8) pass(std::integral_constant<int, 2>{});
            else pass(std::integral_constant<int, 1>{});

            // the warps' sums of this item meet in shared memory, added in warp order
            float* part = s.part + buf * kPartFloats;
            buf ^= 1;
            if (warp < a.warps) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            part[(warp * kTokRows + t * 16 + (i >> 1) * 8 + g) * kPartStride + n * 8 + 2 * q + (i & 1)] =
                                tot[t][n][i];
            }
            __syncthreads();
            if constexpr (!kDown) {
                const int ch = tid & 15, at = tid >> 4;
                if (at < cnt) {
                    const float* p = part + ((ch >> 3) * 16 + (ch & 7)) * kPartStride + at;
                    float gate = 0.0f, upv = 0.0f;
                    for (int w = 0; w < a.warps; ++w) {
                        gate += p[w * kTokRows * kPartStride];
                        upv += p[(w * kTokRows + 8) * kPartStride];
                    }
                    const float h = gate / (1.0f + expf(-gate)) * upv;
                    const __nv_bfloat16 top = __float2bfloat16_rn(h);
                    const float rest = isfinite(__bfloat162float(top)) ? h - __bfloat162float(top) : 0.0f;
                    const int64_t o = (int64_t)(p0 + first + at) * a.I + chunk * 16 + ch;
                    a.h_hi[o] = top;
                    a.h_lo[o] = __float2bfloat16_rn(rest);
                }
            } else {
                const int r = tid & 31, at = tid >> 5;
                if (at < cnt) {
                    const float* p = part + r * kPartStride + at;
                    float y = 0.0f;
                    for (int w = 0; w < a.warps; ++w) y += p[w * kTokRows * kPartStride];
                    const int pair = p0 + first + at;
                    float* acc = s.acc + s.token[pair] * kTokRows + r;
                    *acc = fmaf(s.weight[pair], y, *acc);
                }
            }
        }
        if (++lo == outer || (kDown && item + 1 == i1)) {
            if constexpr (kDown) {
                // the end of this block's part of a chunk: write the chunk, or leave the part
                // where the block that finishes the chunk last adds the parts in block order
                __syncthreads();
                const int64_t lo0 = (int64_t)chunk * A, hi1 = lo0 + A;
                const bool whole = i0 <= lo0 && i1 >= hi1;
                float* mine = a.part + ((int64_t)blockIdx.x * 2 + (chunk != i0 / A)) * a.T * kTokRows;
                if (tid == 0) last = 1;
                if (!whole) {
                    for (int i = tid; i < a.T * kTokRows; i += kTokThreads) mine[i] = s.acc[i];
                    __threadfence();
                    __syncthreads();
                    const int64_t b0 = ((lo0 + 1) * blocks - 1) / total, b1 = (hi1 * blocks - 1) / total;
                    if (tid == 0) {
                        last = atomicAdd(&a.done[chunk], 1u) == (uint32_t)(b1 - b0);
                        __threadfence();
                    }
                    __syncthreads();
                    if (last)
                        for (int i = tid; i < a.T * kTokRows; i += kTokThreads) {
                            float v = 0.0f;
                            for (int64_t b = b0; b <= b1; ++b)
                                v += __ldcg(a.part + (b * 2 + (chunk != (total * b / blocks) / A)) * a.T * kTokRows + i);
                            s.acc[i] = v;
                        }
                }
                __syncthreads();
                for (int i = tid; i < a.T * kTokRows; i += kTokThreads) {
                    if (last) a.out[i / kTokRows * a.out_stride + chunk * kTokRows + i % kTokRows] = __float2bfloat16_rn(s.acc[i]);
                    s.acc[i] = 0.0f;
                }
                __syncthreads();
            }
            if (lo == outer) {
                lo = 0;
                ++hi;
            }
        }
    }
    cp_async_wait<0>();
}

struct TokWorkspace {
    int64_t h_lo, part, done, bytes;
};
static TokWorkspace tok_workspace(int T, int K, int H, int I, int blocks) {
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    TokWorkspace w;
    w.h_lo = up((int64_t)T * K * I * 2);
    w.part = 2 * w.h_lo;
    w.done = w.part + up((int64_t)blocks * 2 * T * kTokRows * 4);
    w.bytes = w.done + up((int64_t)(H / kTokRows) * 4);
    return w;
}

template <bool kFp8>
static ep_status launch_tokens(TokArgs a, const ep_moe_weights* w, int sms, const TokWorkspace& ws, uint8_t* mem, cudaStream_t st) {
    const size_t smem = tok_smem(a.T, a.K, a.list);
    int dev = 0;
    EP_CUDA(cudaGetDevice(&dev));
    static std::atomic<bool> known[kMaxDevicesTracked];  // devices whose launch attributes are set
    if (dev >= kMaxDevicesTracked || !known[dev].load(std::memory_order_relaxed)) {
        const int most = (int)tok_smem(kTokMax, kMaxTopk, kTokMax * kMaxTopk);
        EP_CUDA(cudaFuncSetAttribute(tok_kernel<false, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        EP_CUDA(cudaFuncSetAttribute(tok_kernel<true, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        if (dev < kMaxDevicesTracked) known[dev].store(true, std::memory_order_relaxed);
    }
    a.h_hi = reinterpret_cast<__nv_bfloat16*>(mem);
    a.h_lo = reinterpret_cast<__nv_bfloat16*>(mem + ws.h_lo);
    a.part = reinterpret_cast<float*>(mem + ws.part);
    a.done = reinterpret_cast<uint32_t*>(mem + ws.done);
    // the fewest rounds of kTokWarps warps over a row's stages, then the fewest warps with that many
    auto split = [&](int channels) {
        a.stages = channels * (kFp8 ? 1 : 2) / kTokStage;
        const int rounds = (a.stages + kTokWarps - 1) / kTokWarps;
        a.warps = (a.stages + rounds - 1) / rounds;
    };
    split(a.H);
    a.w = static_cast<const uint8_t*>(w->w13);
    a.ws = w->w13_scales;
    const int64_t items1 = (int64_t)a.list * (a.I / 16), items2 = (int64_t)a.list * (a.H / kTokRows);
    tok_kernel<false, kFp8><<<(int)(items1 < sms ? items1 : sms), kTokThreads, smem, st>>>(a);
    EP_CHECK_LAUNCH("ep_moe_tokens");
    split(a.I);
    a.w = static_cast<const uint8_t*>(w->w2);
    a.ws = w->w2_scales;
    // kernel 2 starts while kernel 1 drains: its list and first weights do not depend on h
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items2 < sms ? items2 : sms));
    cfg.blockDim = dim3(kTokThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    EP_CUDA(cudaLaunchKernelEx(&cfg, tok_kernel<true, kFp8>, a));
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

extern "C" int64_t ep_moe_tokens_workspace(int32_t num_tokens, int32_t num_topk, int32_t hidden, int32_t inter) {
    if (num_tokens < 1 || num_tokens > kTokMax || num_topk < 1 || num_topk > kMaxTopk || hidden < 32 || inter < 32) return 0;
    return tok_workspace(num_tokens, num_topk, hidden, inter, sm_count()).bytes;
}

extern "C" ep_status ep_moe_tokens(const void* x, int64_t x_stride, int32_t num_tokens, const int64_t* topk_idx,
                                   const float* topk_weights, int32_t num_topk, const ep_moe_weights* w, void* out,
                                   int64_t out_stride, void* workspace, int64_t workspace_bytes, uint32_t* status_out,
                                   void* stream) {
    const char* fn = "ep_moe_tokens";
    if (!w) return set_error(EP_ERR_INVALID_ARG, "%s: null weights", fn);
    const bool fp8 = w->w13_scales != nullptr;
    const int H = w->hidden, I = w->inter, unit = fp8 ? 128 : 32;
    if (num_tokens < 0 || num_tokens > kTokMax) return set_error(EP_ERR_INVALID_ARG, "%s: %d tokens outside 0..%d", fn, num_tokens, kTokMax);
    if (num_topk < 1 || num_topk > kMaxTopk) return set_error(EP_ERR_INVALID_ARG, "%s: top-k %d outside 1..%d", fn, num_topk, kMaxTopk);
    if (w->experts < 1 || w->experts > kMaxExperts) return set_error(EP_ERR_INVALID_ARG, "%s: %d experts", fn, w->experts);
    if (H < unit || H % unit || I < unit || I % unit)
        return set_error(EP_ERR_INVALID_ARG, "%s: hidden %d and inter %d must be multiples of %d", fn, H, I, unit);
    if ((w->w2_scales != nullptr) != fp8) return set_error(EP_ERR_INVALID_ARG, "%s: scales for both weights, or for none", fn);
    if (num_tokens == 0) return EP_OK;
    if (!x || !topk_idx || !topk_weights || !out || !w->w13 || !w->w2 || !aligned16(x) || !aligned16(w->w13) || !aligned16(w->w2))
        return set_error(EP_ERR_INVALID_ARG, "%s: null or unaligned (16 bytes: x, weights) pointer", fn);
    if (x_stride < H || x_stride % 8 || out_stride < H)
        return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld (a multiple of 8), %lld for %d channels", fn, (long long)x_stride,
                         (long long)out_stride, H);
    const int sms = sm_count();
    if (sms < 1) return set_error(EP_ERR_CUDA, "%s: no CUDA device", fn);
    const TokWorkspace ws = tok_workspace(num_tokens, num_topk, H, I, sms);
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
    a.list = a.E < a.T * a.K ? a.E : a.T * a.K;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_stride = out_stride;
    a.status = status_out;
    uint8_t* mem = static_cast<uint8_t*>(workspace);
    return fp8 ? launch_tokens<true>(a, w, sms, ws, mem, as_stream(stream)) : launch_tokens<false>(a, w, sms, ws, mem, as_stream(stream));
}
