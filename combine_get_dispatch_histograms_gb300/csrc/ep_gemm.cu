// ep_gemm.cu -- the experts' products on FP8 rows: y = x w^T per group of rows,
// and the first product with its activation and requantisation fused.
//
// Mathematics.  Row r, output channel n, blocks b of 128 along K:
//   y[r][n] = sum_b sx[r][b] * sw[g][n/128][b] * sum_{k in b} x[r][k] * w[g][n][k]
// with e4m3 codes x, w.  The inner sum is a tensor-core product (the codes'
// products are exact in fp32); its scales change with every block, so the
// block's accumulator leaves tensor memory and is added, times sx * sw, to an
// fp32 sum in registers.  One thread owns one row and 128 columns of the tile,
// so that factor is one scalar per thread and block.
#include <cstdlib>

#include "ep_fp8.cuh"
#include "ep_tcgen05.cuh"

namespace ep {

constexpr int kBM = 128;               // rows of a tile
constexpr int kBN = 256;               // weight rows of a tile
constexpr int kBK = 128;               // one scale block of K
constexpr int kStageA = kBM * kBK;     // bytes
constexpr int kStageB = kBN * kBK;
constexpr int kStages = 4;
constexpr int kBoxRows = 32;           // rows of one copy of x: a short group copies only the boxes it has rows in
constexpr int kGemmThreads = 384;      // copy, mma, tensor-memory and spare warp; two warpgroups that sum
constexpr int kMaxGroups = 4096;
constexpr int kChunkM = 16;            // row tiles that share a pass over the weight's tiles
constexpr int64_t kGemmWaitNs = 2000000000ll;

struct GemmArgs {
    const float* x_scales;
    int64_t x_sstride;
    const float* w_scales;
    int64_t w_sgroup;   // floats of one group's scales
    int G, N, K, KB, n_tiles;
    const int32_t *counts, *offsets, *bases;
    int per_base;
    int64_t group_stride, rows;
    void* out;          // bf16 rows, or e4m3 codes
    int64_t out_stride; // elements
    float* out_scales;
    int64_t out_sstride;
    bool out_vec;
    uint32_t* status;
};

struct GemmShared {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], amax_full[2], drain;
    uint32_t tmem;
    int abort;
    int scan[kGemmThreads / 32];
    float amax[2][2][kBM];
};

struct GemmTile {
    int g, n;       // group, column tile
    int64_t row0;   // first row
    int rows;       // 1..kBM
};

__device__ __forceinline__ int64_t group_first(const GemmArgs& a, int g) {
    int64_t r = a.offsets ? (int64_t)a.offsets[g] : (int64_t)g * a.group_stride;
    if (a.bases) r += a.bases[g / a.per_base];
    return r;
}
// Rows of group g inside the arrays: what lies past their end is cut off and flagged.
__device__ __forceinline__ int group_rows(const GemmArgs& a, int g, bool* cut) {
    int64_t n = a.counts ? (int64_t)a.counts[g] : a.group_stride;
    const int64_t f = group_first(a, g);
    if (n <= 0) return 0;
    if (f < 0 || f >= a.rows) {
        *cut = true;
        return 0;
    }
    if (f + n > a.rows) {
        *cut = true;
        n = a.rows - f;
    }
    return (int)n;
}

// Tile t of the launch: groups in order; inside a group, chunks of kChunkM row
// tiles, column tiles inside a chunk, row tiles innermost, so that what runs at
// the same time shares a chunk of rows and few weight tiles.
__device__ __forceinline__ GemmTile find_tile(const GemmArgs& a, const int* start, int t) {
    int lo = 0, hi = a.G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
    }
    bool cut = false;
    const int rows = group_rows(a, lo, &cut);
    const int mt = (rows + kBM - 1) / kBM;
    int r = t - start[lo];
    const int chunk = r / (kChunkM * a.n_tiles);
    r -= chunk * kChunkM * a.n_tiles;
    const int m0 = chunk * kChunkM, mc = min(kChunkM, mt - m0);
    GemmTile tile;
    tile.g = lo;
    tile.n = r / mc;
    const int m = m0 + r % mc;
    tile.row0 = group_first(a, lo) + (int64_t)m * kBM;
    tile.rows = min(kBM, rows - m * kBM);
    return tile;
}

// kSwiglu: the tile's 256 weight rows are 128 gate rows and the 128 up rows of
// the same channels; otherwise 256 consecutive rows.
template <bool kSwiglu>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ GemmShared sh;
    uint8_t* tiles = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    int* start = reinterpret_cast<int*>(tiles + kStages * (kStageA + kStageB));  // [G + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &sh.abort;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], 8);
            mbar_init(&sh.amax_full[b], 8);
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
    }
    if (warp == 2) tmem_alloc(&sh.tmem, 512);

    // first tile of every group: each thread sums a run of groups, one scan over the threads
    {
        const int per = (a.G + kGemmThreads - 1) / kGemmThreads, g0 = tid * per;
        int sum = 0;
        bool cut = false;
        for (int g = g0; g < min(a.G, g0 + per); ++g) {
            const int n = (group_rows(a, g, &cut) + kBM - 1) / kBM * a.n_tiles;
            start[g] = sum;
            sum += n;
        }
        if (cut && a.status && blockIdx.x == 0) flag(a.status, FLAG_CAPACITY);
        int inc = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sh.scan[warp] = inc;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        int before = inc - sum;
        for (int w = 0; w < warp; ++w) before += sh.scan[w];
        for (int g = g0; g < min(a.G, g0 + per); ++g) start[g] += before;
        if (tid == kGemmThreads - 1) start[a.G] = before + sum;
        __syncthreads();
    }
    const int total = start[a.G];
    const uint32_t tmem = sh.tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            // ---- copies: kStages blocks of K ahead of the products --------------
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const GemmTile tile = find_tile(a, start, t);
                const int boxes = (tile.rows + kBoxRows - 1) / kBoxRows;
                const uint32_t bytes = boxes * kBoxRows * kBK + kStageB;
                const int w0 = kSwiglu ? tile.n * 128 : tile.n * kBN;
                const int w1 = kSwiglu ? a.N / 2 + tile.n * 128 : w0 + 128;
                for (int kb = 0; kb < a.KB; ++kb) {
                    if (!mbar_wait_or_abort(&sh.empty[stage], phase ^ 1, kGemmWaitNs, abort)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = tiles + stage * (kStageA + kStageB);
                    uint8_t* sb = sa + kStageA;
                    mbar_arrive_expect_tx(&sh.full[stage], bytes);
                    tma_load_3d(sb, &map_w, kb * kBK, w0, tile.g, &sh.full[stage]);
                    tma_load_3d(sb + kStageB / 2, &map_w, kb * kBK, w1, tile.g, &sh.full[stage]);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(sa + b * kBoxRows * kBK, &map_x, kb * kBK, (int)tile.row0 + b * kBoxRows, &sh.full[stage]);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // no copy may be in flight when the block ends, also after a wait that ran out
            for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                mbar_wait_bounded(&sh.full[i % kStages], (i / kStages) & 1, kGemmWaitNs);
        } else if (warp == 1 && lane == 0) {
            // ---- products: one block of K per accumulator, two accumulators ------
            const uint32_t idesc = idesc_e4m3(kBM, kBN);
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                for (int kb = 0; kb < a.KB; ++kb) {
                    if (!mbar_wait_or_abort(&sh.full[stage], phase, kGemmWaitNs, abort) ||
                        !mbar_wait_or_abort(&sh.acc_empty[buf], bphase ^ 1, kGemmWaitNs, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t* sa = tiles + stage * (kStageA + kStageB);
                    const uint64_t da = smem_desc_sw128(sa), db = smem_desc_sw128(sa + kStageA);
#pragma unroll
                    for (int k = 0; k < kBK / 32; ++k)
                        mma_e4m3(tmem + buf * kBN, da + k * 2, db + k * 2, idesc, k > 0);
                    mma_commit(&sh.empty[stage]);
                    mma_commit(&sh.acc_full[buf]);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    if ((buf ^= 1) == 0) bphase ^= 1;
                }
            }
            mma_commit(&sh.drain);  // every product has finished before tensor memory is freed
            mbar_wait_bounded(&sh.drain, 0, kGemmWaitNs);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // ---- sums: warpgroup `half` adds its 128 columns of every block ----------
        const int half = (warp - 4) >> 2, r = ((warp & 3) << 5) + lane;
        // swiglu: 64 gate columns and the 64 up columns of the same channels
        const uint32_t c0 = kSwiglu ? half * 64 : half * 128, c1 = kSwiglu ? 128 + half * 64 : half * 128 + 64;
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);
        int buf = 0, mbuf = 0;
        uint32_t bphase = 0, mphase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const GemmTile tile = find_tile(a, start, t);
            const bool valid = r < tile.rows;
            const int64_t row = tile.row0 + (valid ? r : 0);
            const float* xs = a.x_scales + row * a.x_sstride;
            const int nb = (kSwiglu ? a.N / 2 : a.N) / 128;
            const int b0 = kSwiglu ? tile.n : min(tile.n * 2 + half, (a.N - 1) / 128);
            const float* ws0 = a.w_scales + tile.g * a.w_sgroup + (int64_t)b0 * a.KB;
            const float* ws1 = kSwiglu ? ws0 + (int64_t)nb * a.KB : ws0;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
            float sx = __ldg(xs), s0 = __ldg(ws0), s1 = __ldg(ws1);
            for (int kb = 0; kb < a.KB; ++kb) {
                const float f0 = sx * s0, f1 = kSwiglu ? sx * s1 : f0;
                if (kb + 1 < a.KB) {  // the next block's scales, used after the next wait
                    sx = __ldg(xs + kb + 1);
                    s0 = __ldg(ws0 + kb + 1);
                    if (kSwiglu) s1 = __ldg(ws1 + kb + 1);
                }
                ok = mbar_wait_or_abort(&sh.acc_full[buf], bphase, kGemmWaitNs, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ad = lane_base + buf * kBN;
                float v[2][32];
                tmem_ld32(ad + c0, v[0]);
                tmem_wait_ld(v[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q < 3) tmem_ld32(ad + (q + 1 < 2 ? c0 + 32 : c1 + (q - 1) * 32), v[(q + 1) & 1]);
                    const float f = q < 2 ? f0 : f1;
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[q * 32 + i] = fmaf(v[q & 1][i], f, acc[q * 32 + i]);
                    if (q < 3) tmem_wait_ld(v[(q + 1) & 1]);
                    if (q == 2) {  // all four loads are in registers: the accumulator is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
                    }
                }
                if ((buf ^= 1) == 0) bphase ^= 1;
            }
            if (!ok) break;
            if constexpr (kSwiglu) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float gate = acc[i];
                    acc[i] = gate / (1.0f + expf(-gate)) * acc[64 + i];
                    m = fmaxf(m, fabsf(acc[i]));
                }
                // the block's maximum over both warpgroups' channels; two buffers: a
                // warp writes one again only after every warp has passed the other
                sh.amax[mbuf][half][r] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.amax_full[mbuf]);
                ok = mbar_wait_or_abort(&sh.amax_full[mbuf], mphase, kGemmWaitNs, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                m = fmaxf(m, sh.amax[mbuf][half ^ 1][r]);
                if ((mbuf ^= 1) == 0) mphase ^= 1;
                const float scale = __fdiv_rn(m, 448.0f);
                if (valid) {
                    uint8_t* o = reinterpret_cast<uint8_t*>(a.out) + row * a.out_stride + tile.n * 128 + half * 64;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<int4*>(o + q * 16) = quantize16_by(&acc[q * 16], scale);
                    if (half == 0) a.out_scales[row * a.out_sstride + tile.n] = scale;
                }
            } else if (valid) {
                const int n0 = tile.n * kBN + half * 128;
                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.out_stride + n0;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    if (a.out_vec && n0 + q * 8 + 8 <= a.N) {
                        __nv_bfloat162 p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(acc[q * 8 + 2 * i], acc[q * 8 + 2 * i + 1]);
                        *reinterpret_cast<int4*>(o + q * 8) = *reinterpret_cast<const int4*>(p);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (n0 + q * 8 + i < a.N) o[q * 8 + i] = __float2bfloat16_rn(acc[q * 8 + i]);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free(tmem, 512);
    if (tid == 0 && *abort && a.status) flag(a.status, FLAG_TIMEOUT);
}

// ---- host -------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

static ep_status encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                        const cuuint32_t* box, const char* what) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(EP_ERR_INVALID_ARG, "%s: the tensor map was refused (%d)", what, (int)r);
    return EP_OK;
}

static ep_status check_products(const char* fn, const ep_fp8_rows* x, const ep_row_groups* g, const ep_fp8_weight* w) {
    if (!x || !g || !w) return set_error(EP_ERR_INVALID_ARG, "%s: null descriptor", fn);
    if (w->groups < 1 || w->groups > kMaxGroups)
        return set_error(EP_ERR_INVALID_ARG, "%s: groups %d outside 1..%d", fn, w->groups, kMaxGroups);
    if (w->n < 1 || w->k < 128 || w->k % 128)
        return set_error(EP_ERR_INVALID_ARG, "%s: weight rows %d, channels %d (a multiple of 128)", fn, w->n, w->k);
    if (!w->codes || !w->scales || !aligned16(w->codes))
        return set_error(EP_ERR_INVALID_ARG, "%s: weight codes (16-byte aligned) and scales are required", fn);
    if (x->rows < 0 || x->rows > 0x7fffffff - kBM)
        return set_error(EP_ERR_INVALID_ARG, "%s: %lld rows", fn, (long long)x->rows);
    if (x->rows > 0) {
        if (!x->codes || !x->scales || !aligned16(x->codes))
            return set_error(EP_ERR_INVALID_ARG, "%s: row codes (16-byte aligned) and scales are required", fn);
        if (x->code_stride < w->k || x->code_stride % 16 || x->scale_stride < w->k / 128)
            return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld, %lld for %d channels", fn, (long long)x->code_stride,
                             (long long)x->scale_stride, w->k);
    }
    if (g->bases && g->per_base < 1) return set_error(EP_ERR_INVALID_ARG, "%s: groups per base %d", fn, g->per_base);
    if (g->stride < 0) return set_error(EP_ERR_INVALID_ARG, "%s: group stride %lld", fn, (long long)g->stride);
    return EP_OK;
}

template <bool kSwiglu>
static ep_status launch_gemm(const char* fn, const ep_fp8_rows* x, const ep_row_groups* g, const ep_fp8_weight* w,
                             GemmArgs a, void* stream) {
    a.x_scales = x->scales;
    a.x_sstride = x->scale_stride;
    a.w_scales = w->scales;
    a.G = w->groups;
    a.N = w->n;
    a.K = w->k;
    a.KB = w->k / kBK;
    a.w_sgroup = (int64_t)((w->n + 127) / 128) * a.KB;
    a.n_tiles = kSwiglu ? w->n / kBN : (w->n + kBN - 1) / kBN;
    a.counts = g->counts;
    a.offsets = g->offsets;
    a.bases = g->bases;
    a.per_base = g->per_base;
    a.group_stride = g->stride;
    a.rows = x->rows;
    // the tiles are counted in 32 bits: every group's last tile may be partial
    const int64_t most = ((x->rows + kBM - 1) / kBM + w->groups) * (int64_t)a.n_tiles;
    if (most > 0x7fffffff) return set_error(EP_ERR_INVALID_ARG, "%s: %lld tiles", fn, (long long)most);

    CUtensorMap map_x, map_w;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)w->k, (cuuint64_t)x->rows};
        const cuuint64_t strides[1] = {(cuuint64_t)x->code_stride};
        const cuuint32_t box[2] = {kBK, kBoxRows};
        const ep_status st = encode(&map_x, x->codes, 2, dims, strides, box, fn);
        if (st != EP_OK) return st;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)w->k, (cuuint64_t)w->n, (cuuint64_t)w->groups};
        const cuuint64_t strides[2] = {(cuuint64_t)w->k, (cuuint64_t)w->k * (cuuint64_t)w->n};
        const cuuint32_t box[3] = {kBK, 128, 1};
        const ep_status st = encode(&map_w, w->codes, 3, dims, strides, box, fn);
        if (st != EP_OK) return st;
    }
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const size_t smem = 1024 + kStages * (kStageA + kStageB) + sizeof(int) * (a.G + 1);
    EP_CUDA(cudaFuncSetAttribute(gemm_kernel<kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    gemm_kernel<kSwiglu><<<(int)(most < sms ? most : sms), kGemmThreads, smem, as_stream(stream)>>>(map_x, map_w, a);
    EP_CHECK_LAUNCH(fn);
    return EP_OK;
}

}  // namespace ep

using namespace ep;

extern "C" ep_status ep_expert_gemm(const ep_fp8_rows* x, const ep_row_groups* groups, const ep_fp8_weight* w, void* out,
                                    int64_t out_stride, uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_gemm";
    const ep_status st = check_products(fn, x, groups, w);
    if (st != EP_OK) return st;
    if (x->rows == 0) return EP_OK;
    if (!out || out_stride < w->n) return set_error(EP_ERR_INVALID_ARG, "%s: output stride %lld for %d channels", fn, (long long)out_stride, w->n);
    if (reinterpret_cast<uintptr_t>(out) & 1) return set_error(EP_ERR_INVALID_ARG, "%s: output is not 2-byte aligned", fn);
    GemmArgs a{};
    a.out = out;
    a.out_stride = out_stride;
    a.out_vec = aligned16(out) && out_stride % 8 == 0;
    a.status = status_out;
    return launch_gemm<false>(fn, x, groups, w, a, stream);
}

extern "C" ep_status ep_expert_swiglu(const ep_fp8_rows* x, const ep_row_groups* groups, const ep_fp8_weight* w13, uint8_t* out,
                                      int64_t out_stride, float* out_scales, int64_t out_scale_stride,
                                      uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_swiglu";
    const ep_status st = check_products(fn, x, groups, w13);
    if (st != EP_OK) return st;
    if (w13->n % 256) return set_error(EP_ERR_INVALID_ARG, "%s: %d weight rows (gate and up, each a multiple of 128)", fn, w13->n);
    if (x->rows == 0) return EP_OK;
    const int inter = w13->n / 2;
    if (!out || !out_scales || !aligned16(out) || out_stride < inter || out_stride % 16 || out_scale_stride < inter / 128)
        return set_error(EP_ERR_INVALID_ARG, "%s: output rows (16-byte aligned, strides %lld, %lld) for %d channels", fn,
                         (long long)out_stride, (long long)out_scale_stride, inter);
    GemmArgs a{};
    a.out = out;
    a.out_stride = out_stride;
    a.out_scales = out_scales;
    a.out_sstride = out_scale_stride;
    a.status = status_out;
    return launch_gemm<true>(fn, x, groups, w13, a, stream);
}
