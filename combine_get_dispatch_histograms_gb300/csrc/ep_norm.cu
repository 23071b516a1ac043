// ep_norm.cu -- RMS norm with the residual's addition, out as bf16 and as the
// FP8 rows that dispatch carries, and its backward pass.
//
// Mathematics.  Per row of H channels, h = x + residual rounded to the residual's type:
//   s = (sum_c h_c^2 / H + eps)^-1/2,   n_c = h_c s w_c
//   y = bf16(n);  FP8: per 128 channels scale = max|n| / 448, code = e4m3(n / scale), from the
//   32-bit n, so that the codes are rounded once
// and backward, with g = dy w and d the gradient that reaches h from elsewhere:
//   dh_c = d_c + s (g_c - h_c s^2 (sum_j g_j h_j) / H),   dw_c = sum over rows of dy_c h_c s
//
// Both are bound by memory: every array is read or written once.  Forward, a row stays in the registers
// of one block (of one warp up to 1024 channels) between its sum and its outputs, with the next row's loads
// on their way: 32768 rows of 7168 with a bf16 residual, bf16 and FP8 out, 335 us (6.3 TB/s of 6.8 measured for
// a copy); with an fp32 residual two vectors a thread and more blocks, since four take 108 registers (4099
// rows of 4104: 42 -> 33.5 us, 6.0 TB/s).  A single row of 7168 takes 2.9 us.  Backward, rows come by bulk
// copies into shared memory, up to four ahead, and two blocks or more share a processor, since a block's
// two sums a row wait for each other (16384 rows of 7168: by registers alone 187 us, one block a processor
// 184, two 161: 5.8 TB/s).
#include <atomic>

#include "ep_fp8.cuh"
#include "ep_tcgen05.cuh"

namespace ep {

constexpr int kNormMaxHidden = 16384;

struct NormArgs {
    const __nv_bfloat16* x;
    const void* residual;
    const void* weight;
    void* residual_out;
    __nv_bfloat16* y;
    uint8_t* fp8;
    int64_t x_stride, r_stride, ro_stride, y_stride, fp8_stride;  // elements; fp8: bytes
    int64_t rows;
    int hidden;
    float eps;
    bool weight_f32;
};

struct NormBackArgs {
    const __nv_bfloat16* dy;
    const void *h, *dres;
    const void* weight;
    void* dx;
    float* part;  // [blocks][hidden]
    int64_t dy_stride, h_stride, dres_stride, dx_stride;
    int64_t rows;
    int hidden;
    float eps;
    bool weight_f32;
};

// 8 channels at a time.  Plain loads: an output may be the input's own memory.
template <typename T>
struct Raw8;  // 8 channels as they lie in memory
template <>
struct Raw8<__nv_bfloat16> {
    int4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_na_v4(p); }
    __device__ __forceinline__ void get(float* v) const {
        const uint32_t u[4] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    // rounds v to the type, v included
    __device__ __forceinline__ void round(float* v) {
        int* o = &a.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            o[i] = *reinterpret_cast<const int*>(&b);
        }
        get(v);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { st_na_v4(p, a); }
};
template <>
struct Raw8<float> {
    uint32_t u[8];
    __device__ __forceinline__ void load(const float* p) {
        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
            ld_global_32(p, u);
        } else {
            const int4 a = ld_na_v4(p), b = ld_na_v4(p + 4);
            u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
        }
    }
    __device__ __forceinline__ void get(float* v) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    }
    __device__ __forceinline__ void round(float* v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[i]);
    }
    __device__ __forceinline__ void store(float* p) const {
        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
            st_global_32(p, u);
        } else {
            st_na_v4(p, make_int4((int)u[0], (int)u[1], (int)u[2], (int)u[3]));
            st_na_v4(p + 4, make_int4((int)u[4], (int)u[5], (int)u[6], (int)u[7]));
        }
    }
};

__device__ __forceinline__ void load_weight8(const void* w, bool f32, int at, float* v) {
    if (f32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        Raw8<__nv_bfloat16> r;
        r.a = *reinterpret_cast<const int4*>(static_cast<const __nv_bfloat16*>(w) + at);
        r.get(v);
    }
}

// Sums of the threads that share a row, the same in each: one barrier a row, by two buffers in turn.
template <bool kWarp, int kN>
__device__ __forceinline__ void row_sums(float (&s)[kN], float (&buf)[2][kN][32], int turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if constexpr (kWarp) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < kN; ++i) buf[turn & 1][i][warp] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = lane < warps ? buf[turn & 1][i][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
}

// The 8 channels of a lane as e4m3; 16 neighbouring lanes hold a block of 128.  Whole warps call it.
__device__ __forceinline__ int2 quantize8(const float* n, float* scale_out) {
    float v[16] = {}, m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = n[i];
        m = max_or_nan(m, fabsf(n[i]));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    *scale_out = __fdiv_rn(m, 448.0f);
    const int4 c = quantize16_by(v, *scale_out);
    return make_int2(c.x, c.y);
}

// kV: vectors of 8 channels a thread; kMax: threads of a block at most; kWarp: a warp a row.
// kRes: 0 no residual, 1 bf16, 2 fp32.
template <int kRes>
using ResType = std::conditional_t<kRes == 2, float, __nv_bfloat16>;

template <int kV, int kMax, bool kWarp, int kRes>
__global__ void __launch_bounds__(kMax) norm_kernel(const NormArgs a) {
    using T = ResType<kRes>;
    __shared__ float buf[2][1][32];
    grid_wait();
    grid_launch_next();
    const int team = kWarp ? 32 : blockDim.x, me = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const int per = kWarp ? blockDim.x >> 5 : 1;
    const int64_t step = (int64_t)gridDim.x * per;
    const int vecs = a.hidden >> 3;
    // the next row's loads are in flight while this one is summed and written
    Raw8<__nv_bfloat16> px[kV];
    Raw8<T> pr[kV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = me + i * team;
            if (v < vecs) {
                px[i].load(a.x + row * a.x_stride + v * 8);
                if (kRes) pr[i].load(static_cast<const T*>(a.residual) + row * a.r_stride + v * 8);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * per + (kWarp ? threadIdx.x >> 5 : 0);
    if (row < a.rows) fetch(row);
    for (int turn = 0; row < a.rows; row += step, ++turn) {
        float h[kV][8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = me + i * team;
            if (v < vecs) {
                px[i].get(h[i]);
                if (kRes) {
                    float r[8];
                    pr[i].get(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += r[j];
                    Raw8<T> o;
                    o.round(h[i]);
                    o.store(static_cast<T*>(a.residual_out) + row * a.ro_stride + v * 8);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(h[i][j], h[i][j], sum[0]);
        }
        if (row + step < a.rows) fetch(row + step);
        row_sums<kWarp>(sum, buf, turn);
        const float s = rsqrtf(sum[0] / (float)a.hidden + a.eps);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = me + i * team;
            if (v < vecs) {
                float w[8];
                load_weight8(a.weight, a.weight_f32, v * 8, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * s * w[j];
                if (a.y) {
                    Raw8<__nv_bfloat16> o;
                    float n[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) n[j] = h[i][j];
                    o.round(n);
                    o.store(a.y + row * a.y_stride + v * 8);
                }
            }
            if (a.fp8) {
                float scale;
                const int2 c = quantize8(h[i], &scale);
                uint8_t* o = a.fp8 + row * a.fp8_stride;
                if (v < vecs) {
                    *reinterpret_cast<int2*>(o + v * 8) = c;
                    if ((v & 15) == 0) *reinterpret_cast<float*>(o + a.hidden + (v >> 4) * 4) = scale;
                }
            }
        }
    }
}

// The 8 channels' share of a row's sums, and then of its outputs.
struct BackRow {
    float s, c;  // the row's scale, and s^2 mean(g h)
};
__device__ __forceinline__ void back_sums(const float* h, const float* g, const float* w, float (&sum)[2]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sum[0] = fmaf(h[j], h[j], sum[0]);
        sum[1] = fmaf(g[j] * w[j], h[j], sum[1]);
    }
}
__device__ __forceinline__ BackRow back_row(const float (&sum)[2], const NormBackArgs& a) {
    BackRow r;
    r.s = rsqrtf(sum[0] / (float)a.hidden + a.eps);
    r.c = r.s * r.s * (sum[1] / (float)a.hidden);
    return r;
}
__device__ __forceinline__ void back_outputs(const BackRow& r, const float* h, const float* g, const float* w, float* d, float* dw) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        d[j] = fmaf(r.s, fmaf(-h[j], r.c, g[j] * w[j]), d[j]);
        dw[j] = fmaf(g[j], h[j] * r.s, dw[j]);
    }
}

// Up to 1024 channels: a warp a row, which stays in its registers.
template <int kV, int kRes>
__global__ void __launch_bounds__(256) norm_backward_warps(const NormBackArgs a) {
    using T = ResType<kRes>;
    __shared__ float block_dw[kV * 256];
    grid_wait();
    grid_launch_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int vecs = a.hidden >> 3;
    float dw[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * 8 + warp; row < a.rows; row += (int64_t)gridDim.x * 8) {
        Raw8<__nv_bfloat16> pg[kV];
        Raw8<T> ph[kV], pd[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = lane + i * 32;
            if (v < vecs) {
                pg[i].load(a.dy + row * a.dy_stride + v * 8);
                ph[i].load(static_cast<const T*>(a.h) + row * a.h_stride + v * 8);
                if (a.dres) pd[i].load(static_cast<const T*>(a.dres) + row * a.dres_stride + v * 8);
            }
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = lane + i * 32;
            if (v < vecs) {
                float h[8], g[8], w[8];
                ph[i].get(h);
                pg[i].get(g);
                load_weight8(a.weight, a.weight_f32, v * 8, w);
                back_sums(h, g, w, sum);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
            sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
        }
        const BackRow r = back_row(sum, a);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int v = lane + i * 32;
            if (v < vecs) {
                float h[8], g[8], w[8], d[8] = {};
                ph[i].get(h);
                pg[i].get(g);
                load_weight8(a.weight, a.weight_f32, v * 8, w);
                if (a.dres) pd[i].get(d);
                back_outputs(r, h, g, w, d, dw[i]);
                Raw8<T> o;
                o.round(d);
                o.store(static_cast<T*>(a.dx) + row * a.dx_stride + v * 8);
            }
        }
    }
    // the block's part of dw, its warps' in order
    for (int w = 0; w < 8; ++w) {
        if (warp == w)
#pragma unroll
            for (int i = 0; i < kV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float* p = &block_dw[(lane + i * 32) * 8 + j];
                    *p = w ? *p + dw[i][j] : dw[i][j];
                }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.hidden; c += 256) a.part[(int64_t)blockIdx.x * a.hidden + c] = block_dw[c];
}

// More channels: a block a row.  The rows to come are on their way into shared memory by bulk copies (a stage holds dy, h
// and d of one row, up to kBackStages of them), so that loads go on while a row is summed and written; a thread's
// registers hold its 16 channels of dw.
constexpr int kBackStages = 4;
constexpr int64_t kBackWaitNs = 2000000000ll;

template <typename T>
__device__ __forceinline__ void shared8(const T* p, float* v) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
        r.a = *reinterpret_cast<const int4*>(p);
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 4);
        r.u[0] = x.x, r.u[1] = x.y, r.u[2] = x.z, r.u[3] = x.w, r.u[4] = y.x, r.u[5] = y.y, r.u[6] = y.z, r.u[7] = y.w;
    }
    r.get(v);
}

template <int kRes>
__global__ void __launch_bounds__(1024) norm_backward_block(const NormBackArgs a, int stages) {
    using T = ResType<kRes>;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kBackStages];
    __shared__ float buf[2][2][32];
    __shared__ int abort[2];  // of the rows in turn: all threads of the block leave the loop at the same row
    const int tid = threadIdx.x, vecs = a.hidden >> 3;
    const uint32_t dy_bytes = a.hidden * 2, h_bytes = a.hidden * sizeof(T);
    const uint32_t stage = dy_bytes + (a.dres ? 2 : 1) * h_bytes;
    if (tid == 0) {
        for (int s = 0; s < kBackStages; ++s) mbar_init(&full[s], 1);
        abort[0] = abort[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_wait();
    grid_launch_next();
    auto issue = [&](int64_t row, int s) {
        uint8_t* d = ring + s * stage;
        mbar_arrive_expect_tx(&full[s], stage);
        bulk_g2s(d, a.dy + row * a.dy_stride, dy_bytes, &full[s]);
        bulk_g2s(d + dy_bytes, static_cast<const T*>(a.h) + row * a.h_stride, h_bytes, &full[s]);
        if (a.dres) bulk_g2s(d + dy_bytes + h_bytes, static_cast<const T*>(a.dres) + row * a.dres_stride, h_bytes, &full[s]);
    };
    int64_t next = blockIdx.x;  // the next row to copy
    if (tid == 0)
        for (int s = 0; s < stages && next < a.rows; ++s, next += gridDim.x) issue(next, s);
    float dw[2][8] = {};
    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool gave_up = false;
    int64_t row = blockIdx.x;
    for (; row < a.rows; row += gridDim.x, ++turn) {
        // a copy that does not come ends the row loop for the whole block
        if (!mbar_wait_bounded(&full[s], phase, kBackWaitNs)) abort[turn & 1] = 1;
        const uint8_t* p = ring + s * stage;
        const __nv_bfloat16* sg = reinterpret_cast<const __nv_bfloat16*>(p);
        const T* sh = reinterpret_cast<const T*>(p + dy_bytes);
        const T* sd = reinterpret_cast<const T*>(p + dy_bytes + h_bytes);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = tid + i * blockDim.x;
            if (v < vecs) {
                float h[8], g[8], w[8];
                shared8(sh + v * 8, h);
                shared8(sg + v * 8, g);
                load_weight8(a.weight, a.weight_f32, v * 8, w);
                back_sums(h, g, w, sum);
            }
        }
        row_sums<false>(sum, buf, turn);
        gave_up = *static_cast<volatile int*>(&abort[turn & 1]);
        if (gave_up) break;
        // every thread has left the row before: its stage takes the next copy
        if (tid == 0 && turn > 0 && stages > 1 && next < a.rows) {
            issue(next, s == 0 ? stages - 1 : s - 1);
            next += gridDim.x;
        }
        const BackRow r = back_row(sum, a);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = tid + i * blockDim.x;
            if (v < vecs) {
                float h[8], g[8], w[8], d[8] = {};
                shared8(sh + v * 8, h);
                shared8(sg + v * 8, g);
                load_weight8(a.weight, a.weight_f32, v * 8, w);
                if (a.dres) shared8(sd + v * 8, d);
                back_outputs(r, h, g, w, d, dw[i]);
                Raw8<T> o;
                o.round(d);
                o.store(static_cast<T*>(a.dx) + row * a.dx_stride + v * 8);
            }
        }
        if (stages == 1) {
            __syncthreads();
            if (tid == 0 && next < a.rows) {
                issue(next, 0);
                next += gridDim.x;
            }
        }
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    // Then its part of dw is NaN, and so is dx from that row on: whoever reads either sees it.
    const float bad = gave_up ? __int_as_float(0x7fffffff) : 0.0f;
    if (gave_up) {
        if (tid == 0)  // no copy may be in flight when the block ends
            for (int i = 0; i < stages; ++i) mbar_wait_bounded(&full[i], i < s ? phase ^ 1 : phase, kBackWaitNs);
        for (; row < a.rows; row += gridDim.x)
            for (int v = tid; v < vecs; v += blockDim.x) {
                float d[8] = {bad, bad, bad, bad, bad, bad, bad, bad};
                Raw8<T> o;
                o.round(d);
                o.store(static_cast<T*>(a.dx) + row * a.dx_stride + v * 8);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int v = tid + i * blockDim.x;
        if (v < vecs) {
            float* p = a.part + (int64_t)blockIdx.x * a.hidden + v * 8;
            *reinterpret_cast<float4*>(p) = make_float4(dw[i][0] + bad, dw[i][1] + bad, dw[i][2] + bad, dw[i][3] + bad);
            *reinterpret_cast<float4*>(p + 4) = make_float4(dw[i][4] + bad, dw[i][5] + bad, dw[i][6] + bad, dw[i][7] + bad);
        }
    }
}

// dw[c] = sum over blocks of part[block][c], in an order that depends on the number of blocks alone: 32 rows of threads
// take every 32nd block each, then their sums are added as a tree.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, int blocks, int hidden, float* dw) {
    __shared__ float sums[32][33];
    grid_wait();
    grid_launch_next();
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < hidden)
#pragma unroll 8
        for (int b = r; b < blocks; b += 32) s += part[(int64_t)b * hidden + c];
    sums[r][lane] = s;
    __syncthreads();
    s = sums[lane][r];  // warp r: column r
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && blockIdx.x * 32 + r < hidden) dw[blockIdx.x * 32 + r] = s;
}

// ---- host -------------------------------------------------------------------------
static ep_status sm_count(int* sms) {
    int dev = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
    return EP_OK;
}

// Who works on a row of the forward pass: `kind` 0..2: a warp with 1, 2 or 4 vectors a lane; 3: a block with one vector a
// thread; 4: a block of up to 256 threads with 4; 5: of up to 1024 with 2.
constexpr int kNormPerSm = 6;  // blocks of up to 256 threads
struct NormShape {
    int kind, threads, blocks;
};
static NormShape norm_shape(int64_t rows, int hidden, int sms, bool wide) {
    const int vecs = hidden / 8;
    NormShape s;
    int64_t units = rows, per_sm = kNormPerSm;
    if (vecs <= 128) {
        s.kind = vecs <= 32 ? 0 : vecs <= 64 ? 1 : 2;
        s.threads = 256;
        units = (rows + 7) / 8;
    } else {
        s.kind = vecs > 1024 ? 5 : rows <= sms ? 3 : wide ? 5 : 4;
        const int v = s.kind == 3 ? 1 : s.kind == 4 ? 4 : 2;
        s.threads = ((vecs + v - 1) / v + 31) / 32 * 32;
        per_sm = s.kind == 3 ? 1 : s.kind == 5 ? 1024 / s.threads : kNormPerSm;
    }
    s.blocks = (int)(units < sms * per_sm ? units : sms * per_sm);
    return s;
}

template <int kRes>
static ep_status launch_norm(const NormArgs& a, const NormShape& s, void* stream) {
    switch (s.kind) {
        case 0: return launch_next(norm_kernel<1, 256, true, kRes>, s.blocks, s.threads, stream, a);
        case 1: return launch_next(norm_kernel<2, 256, true, kRes>, s.blocks, s.threads, stream, a);
        case 2: return launch_next(norm_kernel<4, 256, true, kRes>, s.blocks, s.threads, stream, a);
        case 3: return launch_next(norm_kernel<1, 1024, false, kRes>, s.blocks, s.threads, stream, a);
        case 4: return launch_next(norm_kernel<4, 256, false, kRes>, s.blocks, s.threads, stream, a);
        default: return launch_next(norm_kernel<2, 1024, false, kRes>, s.blocks, s.threads, stream, a);
    }
}

// Blocks of the backward pass, each with a part of dw, at most: by warps three a processor; by blocks as many as its
// registers hold, up to 8.
static int back_threads(int hidden) { return ((hidden / 8 + 1) / 2 + 31) / 32 * 32; }
static int back_blocks(int64_t rows, int hidden, int sms) {
    const int per_sm = hidden <= 1024 ? 3 : 1024 / back_threads(hidden) < 8 ? 1024 / back_threads(hidden) : 8;
    const int64_t units = hidden <= 1024 ? (rows + 7) / 8 : rows, most = (int64_t)per_sm * sms;
    return (int)(units < most ? units : most);
}

template <int kRes>
static ep_status launch_back(const NormBackArgs& a, int sms, int* blocks, void* stream) {
    const int vecs = a.hidden / 8;
    if (vecs <= 32) return launch_next(norm_backward_warps<1, kRes>, *blocks, 256, stream, a);
    if (vecs <= 64) return launch_next(norm_backward_warps<2, kRes>, *blocks, 256, stream, a);
    if (vecs <= 128) return launch_next(norm_backward_warps<4, kRes>, *blocks, 256, stream, a);
    // A block's sums wait for each other, so that two blocks or more share a processor where two rows each fit.
    const int threads = back_threads(a.hidden), stage = a.hidden * (2 + (a.dres ? 2 : 1) * (int)sizeof(ResType<kRes>));
    constexpr int kMost = 208 * 1024;
    int per_sm = 1024 / threads < 8 ? 1024 / threads : 8;
    while (per_sm > 1 && per_sm * 2 * stage > kMost) --per_sm;
    const int fit = kMost / per_sm / stage, stages = fit < kBackStages ? fit : kBackStages;
    if (*blocks > per_sm * sms) *blocks = per_sm * sms;
    int dev = 0;
    EP_CUDA(cudaGetDevice(&dev));
    static std::atomic<bool> known[kMaxDevicesTracked];  // devices whose launch attribute is set
    if (dev >= kMaxDevicesTracked || !known[dev].load(std::memory_order_relaxed)) {
        EP_CUDA(cudaFuncSetAttribute(norm_backward_block<kRes>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost));
        if (dev < kMaxDevicesTracked) known[dev].store(true, std::memory_order_relaxed);
    }
    return launch_next(norm_backward_block<kRes>, *blocks, threads, stream, Shared{(size_t)stages * stage}, a, stages);
}

static int type_bytes(int type) { return type == EP_F32 ? 4 : 2; }

// A row array: there, 16-byte aligned, rows far enough apart and on 16 bytes.
static ep_status check_rows(const char* fn, const char* what, const void* p, int64_t stride, int64_t rows, int hidden, int type) {
    if (!p || !aligned16(p)) return set_error(EP_ERR_INVALID_ARG, "%s: %s is required, 16-byte aligned", fn, what);
    if (stride * type_bytes(type) % 16 || (rows > 1 && stride < hidden))
        return set_error(EP_ERR_INVALID_ARG, "%s: %s: rows %lld elements apart for %d channels (whole 16 bytes)", fn, what, (long long)stride, hidden);
    return EP_OK;
}
static ep_status check_norm(const char* fn, int64_t rows, int hidden, float eps, int residual_type, const void* weight, int weight_type) {
    if (rows < 0 || rows > 0x7fffffff) return set_error(EP_ERR_INVALID_ARG, "%s: %lld rows", fn, (long long)rows);
    if (hidden < 8 || hidden % 8 || hidden > kNormMaxHidden)
        return set_error(EP_ERR_INVALID_ARG, "%s: %d channels (a multiple of 8, at most %d)", fn, hidden, kNormMaxHidden);
    if (!(eps > 0.0f) || eps > 3.0e38f) return set_error(EP_ERR_INVALID_ARG, "%s: eps must be positive", fn);
    if (residual_type < 0 || residual_type > EP_F32 || weight_type < 0 || weight_type > EP_F32)
        return set_error(EP_ERR_INVALID_ARG, "%s: types %d, %d", fn, residual_type, weight_type);
    if (!weight || !aligned16(weight)) return set_error(EP_ERR_INVALID_ARG, "%s: weight is required, 16-byte aligned", fn);
    return EP_OK;
}

}  // namespace ep

using namespace ep;

extern "C" ep_status ep_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                 int32_t residual_type, const void* weight, int32_t weight_type, float eps, int64_t rows,
                                 int32_t hidden, void* residual_out, int64_t residual_out_stride, void* y, int64_t y_stride,
                                 uint8_t* fp8_rows, int64_t fp8_stride, void* stream) {
    const char* fn = "ep_rms_norm";
    EP_TRY(check_norm(fn, rows, hidden, eps, residual_type, weight, weight_type));
    if (fp8_rows && hidden % 128) return set_error(EP_ERR_INVALID_ARG, "%s: FP8 rows of %d channels (a multiple of 128)", fn, hidden);
    if (rows == 0) return EP_OK;
    if (!y && !fp8_rows) return set_error(EP_ERR_INVALID_ARG, "%s: no output", fn);
    if (!residual != !residual_out) return set_error(EP_ERR_INVALID_ARG, "%s: a residual comes with its output", fn);
    EP_TRY(check_rows(fn, "x", x, x_stride, rows, hidden, EP_BF16));
    if (y) EP_TRY(check_rows(fn, "y", y, y_stride, rows, hidden, EP_BF16));
    if (residual) {
        EP_TRY(check_rows(fn, "residual", residual, residual_stride, rows, hidden, residual_type));
        EP_TRY(check_rows(fn, "residual_out", residual_out, residual_out_stride, rows, hidden, residual_type));
    }
    if (fp8_rows && (!aligned16(fp8_rows) || fp8_stride % 16 || (rows > 1 && fp8_stride < ep_fp8_row_bytes(hidden))))
        return set_error(EP_ERR_INVALID_ARG, "%s: FP8 rows (16-byte aligned) %lld bytes apart", fn, (long long)fp8_stride);
    int sms = 0;
    EP_TRY(sm_count(&sms));
    const NormArgs a = {static_cast<const __nv_bfloat16*>(x), residual, weight, residual_out, static_cast<__nv_bfloat16*>(y), fp8_rows,
                        x_stride, residual_stride, residual_out_stride, y_stride, fp8_stride, rows, hidden, eps, weight_type == EP_F32};
    const NormShape s = norm_shape(rows, hidden, sms, residual && residual_type == EP_F32);
    return !residual ? launch_norm<0>(a, s, stream) : residual_type == EP_BF16 ? launch_norm<1>(a, s, stream) : launch_norm<2>(a, s, stream);
}

extern "C" int64_t ep_rms_norm_backward_workspace(int64_t rows, int32_t hidden) {
    int sms = 0;
    if (rows <= 0 || rows > 0x7fffffff || hidden < 8 || hidden % 8 || hidden > kNormMaxHidden || sm_count(&sms) != EP_OK) return 0;
    return (int64_t)back_blocks(rows, hidden, sms) * hidden * 4;
}

extern "C" ep_status ep_rms_norm_backward(const void* dy, int64_t dy_stride, const void* h, int64_t h_stride, int32_t h_type,
                                          const void* weight, int32_t weight_type, float eps, const void* dresidual,
                                          int64_t dresidual_stride, int64_t rows, int32_t hidden, void* dx, int64_t dx_stride,
                                          float* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "ep_rms_norm_backward";
    EP_TRY(check_norm(fn, rows, hidden, eps, h_type, weight, weight_type));
    if (!dweight || !aligned_to(dweight, 4)) return set_error(EP_ERR_INVALID_ARG, "%s: dweight is required", fn);
    int blocks = 0;
    if (rows > 0) {
        EP_TRY(check_rows(fn, "dy", dy, dy_stride, rows, hidden, EP_BF16));
        EP_TRY(check_rows(fn, "h", h, h_stride, rows, hidden, h_type));
        EP_TRY(check_rows(fn, "dx", dx, dx_stride, rows, hidden, h_type));
        if (dresidual) EP_TRY(check_rows(fn, "dresidual", dresidual, dresidual_stride, rows, hidden, h_type));
        int sms = 0;
        EP_TRY(sm_count(&sms));
        blocks = back_blocks(rows, hidden, sms);
        if (!workspace || !aligned16(workspace) || workspace_bytes < (int64_t)blocks * hidden * 4)
            return set_error(EP_ERR_INVALID_ARG, "%s: workspace of %lld bytes (16-byte aligned), %lld needed", fn,
                             (long long)workspace_bytes, (long long)blocks * hidden * 4);
        const NormBackArgs a = {static_cast<const __nv_bfloat16*>(dy), h, dresidual, weight, dx, static_cast<float*>(workspace),
                                dy_stride, h_stride, dresidual_stride, dx_stride, rows, hidden, eps, weight_type == EP_F32};
        EP_TRY(h_type == EP_BF16 ? launch_back<1>(a, sms, &blocks, stream) : launch_back<2>(a, sms, &blocks, stream));
    }
    return launch_next(norm_weight_kernel, (hidden + 31) / 32, 1024, stream, static_cast<const float*>(workspace), blocks, hidden, dweight);
}
