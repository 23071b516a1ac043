// ep_gemm.cu -- the experts' products on FP8 rows: y = x w^T per group of rows,
// and the first product with its activation and requantisation fused.
//
// Mathematics.  Row r, output channel n, blocks b of 128 along K:
//   y[r][n] = sum_b sx[r][b] * sw[g][n/128][b] * sum_{k in b} x[r][k] * w[g][n][k]
// with e4m3 codes x, w.  The inner sum is a tensor-core product (the codes'
// products are exact in fp32); its scales change with every block, so the
// block's accumulator leaves tensor memory and is added, times sx * sw, to an
// fp32 sum in registers.  A thread owns one row and 64 columns of the tile, so
// that factor is one scalar per thread and block (gate and up: two).
//
// Shape.  256 weight rows a tile: tensor memory then holds two accumulators, so
// that one fills while the other is added.  One warp copies, one issues the
// products, one announces tiles and stages scales, 16 add; each has what it
// needs in shared memory and none waits for global memory in the loop over K.
//
// Bound.  With long groups not the tensor cores: a block of K takes them 517
// cycles (128 x 256 x 128 of each SM) and the kernel 860 to 1000, by the clock that
// power leaves.  What holds it there is not settled.  The adding takes its share:
// a warp adds for about 600 cycles (365 while no products run; 292 are the 32,768
// multiply-adds), hands its accumulator back half way through, and waits 220 for
// the next one; a third accumulator has no room, nor have the registers for loading
// all of one before adding it.  But a variant that read no accumulator and handed
// each back at once kept 88 % of the time (K 8192: 964 us of 1099, 882 cycles a
// block of 1005 at the same clock), so that the copies (32 KB per SM and block,
// 11.7 TB/s out of the second-level cache at that rate) or the issue of both must
// come close to it.  Halves of the tile handed back on their own (two issuing warps)
// read the rows' tile twice from shared memory and are slower (1163 -> 1305 us).
// The warps with 32 registers spill some 130 to 140 bytes.  Sustained, power: 1360
// of 1400 W, and the clock falls to 1.7 - 1.76 GHz.  Measured: second product, 262144
// rows, K 2048, N 7168, 256 groups, 3.42 ms from a cool start (2.25 PFLOP/s) and
// 3.74 sustained (2.06); first product, 498304 rows, K 4096, 2I 2816, 4.41 ms (2.6)
// and 4.84 (2.4).  With short groups the weights' bytes: 64 rows a group run at
// 6.6 TB/s (second product 0.60 ms, first 1.13 ms of 256 groups).
#include <atomic>
#include <initializer_list>

#include "ep_fp8.cuh"
#include "ep_groups.cuh"

namespace ep {

constexpr int kBM = 128;               // rows of a tile in each block
constexpr int kBN = 256;               // weight rows of a tile
constexpr int kBK = 128;               // one scale block of K
constexpr int kStages = 4;             // blocks of K in flight; the loops over K are unrolled by it
constexpr int kBoxRows = 32;           // rows of one copy of x: a short group copies only the boxes it has rows in
constexpr int kSumGroups = 4;          // warpgroups that sum, each a quarter of the tile's columns
constexpr int kSumWarps = 4 * kSumGroups;
constexpr int kGemmThreads = 128 + 128 * kSumGroups;  // copy, mma, tensor-memory and tile warp first

// The two shapes of the kernel.  kCtas = 2: a pair of blocks makes a tile of 256
// rows; each copies half of the weight's rows, so that a block moves 32 KB per
// block of K instead of 48.  kCtas = 1: tiles of 128 rows, for groups too short
// to fill both halves, where the weight's bytes bound the time.
template <int kCtas>
struct GemmShape {
    static constexpr int kTileM = kCtas * kBM;
    static constexpr int kStageA = kBM * kBK;          // bytes in each block
    static constexpr int kStageB = kBN / kCtas * kBK;
    static constexpr int kStage = kStageA + kStageB;
    // of a warp's output on its way: 32 rows of 64 columns, or (48 KB stages leave no room) of 8
    static constexpr int kOut = kCtas == 2 ? 32 * 128 : 32 * 16;
    static constexpr size_t kSmem = 1024 + kStages * kStage + kSumWarps * kOut;
};
constexpr int kTileRing = 4;            // tiles announced ahead
constexpr int kScaleChunk = 8;          // blocks of K whose scales are staged together
constexpr int kScaleRing = 2;
constexpr int kSplitStride = kBN + 4;  // floats of a row of sums: rows fall into other banks
constexpr int64_t kGemmWaitNs = 2000000000ll;

struct GemmArgs : TileArgs {
    const float* x_scales;
    int64_t x_sstride;
    const float* w_scales;
    int64_t w_sgroup;   // floats of one group's scales
    int N, K, KB;
    void* out;          // bf16 rows, or e4m3 codes
    int64_t out_stride; // elements
    float* out_scales;
    int64_t out_sstride;
    bool out_vec;       // 16-byte stores
    bool out_wide;      // 32-byte stores
    bool out_clip;      // rows end at a multiple of 16 bytes, so that a tiled copy that crosses their end is cut there
    bool x_vec;         // 16-byte loads of row scales
    uint32_t* status;
};

struct GemmShared {
    // done: the products of a stage's block have finished; frees the stage and hands over its accumulator
    uint64_t full[kStages], done[kStages], acc_empty[2], amax_full[2];
    uint64_t tile_full[kTileRing], tile_empty[kTileRing], scale_full[kScaleRing], scale_empty[kScaleRing], drain;
    uint32_t tmem;
    int abort;
    GemmTile tile[kTileRing];
    float amax[2][kSumGroups][kBM];
    // sx * sw of a chunk of blocks: [block][first or second weight block of the tile][row]
    float scale[kScaleRing][kScaleChunk][2][kBM];
};

// The stages and accumulators need none: every tile starts at stage 0 and
// accumulator 0, so that in the unrolled loops both are constants, and bit u of
// a mask is the parity of slot u's next phase.

// kSwiglu: the tile's 256 weight rows are 128 gate rows and the 128 up rows of
// the same channels; otherwise 256 consecutive rows.
// kSplit (with kCtas = 1): the blocks of a cluster make one tile, each from its
// share of the blocks of K.  For launches with fewer tiles than SMs, where one
// block alone would walk all of K; every cluster has at most one tile.
template <bool kSwiglu, int kCtas, bool kSplit>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
            const __grid_constant__ CUtensorMap map_out, const GemmArgs a) {
    using Shape = GemmShape<kCtas>;
    constexpr int kTileM = Shape::kTileM, kStage = Shape::kStage, kStageA = Shape::kStageA;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ GemmShared sh;
    uint8_t* tiles = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    uint8_t* out_stage = tiles + kStages * kStage;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
    const int part = kSplit ? (int)cluster_rank() : 0, parts = kSplit ? cluster_size() : 1;
    const int unit = blockIdx.x / (kCtas * parts), units = gridDim.x / (kCtas * parts);
    const int k0 = kSplit ? part * a.KB / parts : 0, k1 = kSplit ? (part + 1) * a.KB / parts : a.KB;
    volatile int* abort = &sh.abort;
    const uint32_t full = smem_u32(sh.full), done = smem_u32(sh.done), acc_empty = smem_u32(sh.acc_empty);
    const uint32_t tile_full = smem_u32(sh.tile_full), tile_empty = smem_u32(sh.tile_empty);
    const uint32_t scale_full = smem_u32(sh.scale_full), scale_empty = smem_u32(sh.scale_empty);

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.done[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_empty[b], kCtas * kSumWarps);
            mbar_init(&sh.amax_full[b], kSumWarps);
        }
        for (int b = 0; b < kTileRing; ++b) {
            mbar_init(&sh.tile_full[b], 1);
            mbar_init(&sh.tile_empty[b], kSumWarps + 1 + (rank == 0));
        }
        for (int b = 0; b < kScaleRing; ++b) {
            mbar_init(&sh.scale_full[b], 1);
            mbar_init(&sh.scale_empty[b], kSumWarps);
        }
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < kTileRing; ++i) sh.tile[i].rows = 0;
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
        if (kCtas == 2 && (kSwiglu || a.out_vec)) tma_prefetch_desc(&map_out);
    }
    if (warp == 2) tmem_alloc<kCtas>(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();  // both blocks' barriers are ready
    tc_fence_after();
    // All above may run beside the end of the kernel before; the kernel after may do the same.
    grid_wait();
    grid_launch_next();
    const uint32_t tmem = sh.tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == 3) {
            // ---- tiles and scales: announces each tile, then stages its blocks' scales, so that the
            // other warps never wait for global memory themselves
            TileWalk<kTileM> walk;
            RingPos<kTileRing> tr;
            RingPos<kScaleRing> sr;
            for (int t = unit;; t += units) {
                GemmTile tile = {0, 0, 0, 0};
                // groups that overlap may have any number of tiles: those past a.most are cut off
                const bool some = walk.find(a, min(t, a.most), lane, &tile);
                if (t >= a.most) tile.rows = 0;
                mbar_wait_warp<true>(tr.bar(tile_empty), tr.phase() ^ 1, kGemmWaitNs, abort);
                if (__any_sync(0xffffffffu, *abort)) break;
                if (lane == 0) {
                    sh.tile[tr.slot()] = tile;
                    mbar_arrive(tr.bar(tile_full));
                }
                ++tr.n;
                if (!some || t >= a.most) {
                    walk.cut |= some;
                    break;
                }
                const int mine = min(tile.rows - rank * kBM, kBM);
                // lanes 0-7 and 8-15: the weight blocks' scales of a chunk
                const int b0 = kSwiglu ? tile.n : tile.n * 2;
                const int b1 = kSwiglu ? a.N / 256 + tile.n : min(b0 + 1, (a.N - 1) / 128);
                const float* ws = a.w_scales + tile.g * a.w_sgroup + (int64_t)(lane < 8 ? b0 : b1) * a.KB + (lane & 7);
                const float* xs = a.x_scales + (int64_t)(tile.row0 + rank * kBM) * a.x_sstride;
#pragma unroll 1
                for (int kb = k0; kb < k1; kb += kScaleChunk) {
                    mbar_wait_warp<true>(sr.bar(scale_empty), sr.phase() ^ 1, kGemmWaitNs, abort);
                    const float w = lane < 16 && kb + (lane & 7) < k1 ? ws[kb] : 0.0f;
                    float* dst = &sh.scale[sr.slot()][0][0][0];
#pragma unroll 1
                    for (int i = 0; i < kScaleChunk && kb + i < k1; i += 4) {
                        const float w00 = __shfl_sync(0xffffffffu, w, i), w01 = __shfl_sync(0xffffffffu, w, 8 + i);
                        const float w10 = __shfl_sync(0xffffffffu, w, i + 1), w11 = __shfl_sync(0xffffffffu, w, 9 + i);
                        const float w20 = __shfl_sync(0xffffffffu, w, i + 2), w21 = __shfl_sync(0xffffffffu, w, 10 + i);
                        const float w30 = __shfl_sync(0xffffffffu, w, i + 3), w31 = __shfl_sync(0xffffffffu, w, 11 + i);
#pragma unroll 1
                        for (int r = lane; r < mine; r += 32) {
                            const float* p = xs + r * a.x_sstride + kb + i;
                            float4 v;
                            if (a.x_vec && (!kSplit || (k0 & 3) == 0) && kb + i + 4 <= k1) {
                                v = *reinterpret_cast<const float4*>(p);
                            } else {
                                v.x = *p;
                                v.y = kb + i + 1 < k1 ? p[1] : 0.0f;
                                v.z = kb + i + 2 < k1 ? p[2] : 0.0f;
                                v.w = kb + i + 3 < k1 ? p[3] : 0.0f;
                            }
                            float* d = dst + i * 2 * kBM + r;
                            d[0] = v.x * w00;
                            d[kBM] = v.x * w01;
                            d[2 * kBM] = v.y * w10;
                            d[3 * kBM] = v.y * w11;
                            d[4 * kBM] = v.z * w20;
                            d[5 * kBM] = v.z * w21;
                            d[6 * kBM] = v.w * w30;
                            d[7 * kBM] = v.w * w31;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sr.bar(scale_full));
                    ++sr.n;
                }
            }
            if (walk.cut && a.status && blockIdx.x == 0) flag(a.status, FLAG_CAPACITY);
        } else if (warp == 0 && lane == 0) {
            // ---- copies: kStages blocks of K ahead of the products.  Each block fills its
            // own half of a stage; block 0's barrier counts the bytes of both.
            RingPos<kTileRing> tr;
            uint32_t free_phase = (1u << kStages) - 1;  // a fresh barrier counts as passed
            bool ok = true;
            while (ok) {
                if (!mbar_wait_or_abort<true>(tr.bar(tile_full), tr.phase(), kGemmWaitNs, abort)) break;
                const GemmTile tile = sh.tile[tr.slot()];
                mbar_arrive(tr.bar(tile_empty));
                ++tr.n;
                if (tile.rows == 0) break;
                const int boxes0 = (min(tile.rows, kBM) + kBoxRows - 1) / kBoxRows;
                const int boxes1 = (max(tile.rows - kBM, 0) + kBoxRows - 1) / kBoxRows;
                const uint32_t bytes = (boxes0 + boxes1) * kBoxRows * kBK + kBN * kBK;
                const int boxes = rank ? boxes1 : boxes0;
                const int row = tile.row0 + rank * kBM;
                const int w0 = kSwiglu ? tile.n * 128 : tile.n * kBN, w1 = kSwiglu ? a.N / 2 + w0 : w0 + 128;
                const uint32_t full0 = kCtas == 2 ? smem_of(full, 0) : full;
                for (int kb = k0; kb < k1; ++kb) {
                    const int u = (kb - k0) & (kStages - 1);
                    if (!mbar_wait_or_abort<true>(done + u * 8, free_phase >> u & 1, kGemmWaitNs, abort)) {
                        ok = false;
                        break;
                    }
                    free_phase ^= 1u << u;
                    uint8_t* sa = tiles + u * kStage;
                    if (rank == 0) mbar_arrive_expect_tx(&sh.full[u], bytes);
                    tma_load_3d<kCtas>(sa + kStageA, &map_w, kb * kBK, rank ? w1 : w0, tile.g, full0 + u * 8);
                    if (kCtas == 1) tma_load_3d<kCtas>(sa + kStageA + 128 * kBK, &map_w, kb * kBK, w1, tile.g, full0 + u * 8);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d<kCtas>(sa + b * kBoxRows * kBK, &map_x, kb * kBK, row + b * kBoxRows, full0 + u * 8);
                }
            }
            // no copy may be in flight when the blocks end, also after a wait that ran out: the last
            // phase that this stage's copies complete is the one before its next
            if (rank == 0)
                for (int u = 0; u < kStages; ++u)
                    mbar_wait_bounded(&sh.full[u], free_phase >> u & 1, kGemmWaitNs);
        } else if (warp == 1 && rank == 0) {
            // ---- products: one block of K per accumulator, two accumulators.  The whole warp runs the
            // loop, so that descriptors stay in uniform registers; one lane issues (a loop of one lane
            // alone issued a block in about 900 cycles, measured, against 517 that it takes)
            const uint32_t idesc = idesc_e4m3(kTileM, kBN);
            const uint64_t da0 = smem_desc_sw128(tiles), db0 = smem_desc_sw128(tiles + kStageA);
            RingPos<kTileRing> tr;
            uint32_t full_phase = 0, empty_phase = 3;
            while (true) {
                mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), kGemmWaitNs, abort);
                const int rows = sh.tile[tr.slot()].rows;
                __syncwarp();
                if (lane == 0) mbar_arrive(tr.bar(tile_empty));
                ++tr.n;
                if (rows == 0 || __any_sync(0xffffffffu, *abort)) break;
#pragma unroll 1
                for (int kb = 0; kb < k1 - k0; ++kb) {
                    const int u = kb & (kStages - 1), c = kb & 1;
                    mbar_wait_warp<true>(full + u * 8, full_phase >> u & 1, kGemmWaitNs, abort);
                    mbar_wait_warp<true>(acc_empty + c * 8, empty_phase >> c & 1, kGemmWaitNs, abort);
                    full_phase ^= 1u << u;
                    empty_phase ^= 1u << c;
                    tc_fence_after();
                    const uint32_t at = u * (kStage >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBK / 32; ++k)
                            mma_e4m3<kCtas>(tmem + c * kBN, da0 + at + k * 2, db0 + at + k * 2, idesc, k > 0);
                        mma_commit<kCtas>(done + u * 8);
                    }
                    __syncwarp();
                }
            }
            // every product has finished before either block frees its tensor memory or ends: the second block waits
            // for this one below, and nothing arrives on its own barrier, which would have to outlive the arrival
            if (elect_one()) mma_commit_here<kCtas>(smem_u32(&sh.drain));
            __syncwarp();
            mbar_wait_bounded(&sh.drain, 0, kGemmWaitNs);
        }
        if constexpr (kSplit) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else {
        // 512 x 112 + 128 x 32 registers are the launch's 640 x 96
        asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        // ---- sums: each warpgroup adds its columns of every block of K -----------
        const int quarter = (warp - 4) >> 2, r = ((warp & 3) << 5) + lane;
        // swiglu: 32 gate columns and the 32 up columns of the same channels
        const uint32_t c0 = kSwiglu ? quarter * 32 : quarter * 64, c1 = kSwiglu ? 128 + quarter * 32 : quarter * 64 + 32;
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t free_bar = kCtas == 2 ? smem_of(acc_empty, 0) : acc_empty;
        const uint32_t sc0 = smem_u32(&sh.scale[0][0][kSwiglu ? 0 : quarter >> 1][r]);
        RingPos<kTileRing> tr;
        RingPos<kScaleRing> sr;
        uint32_t done_phase = 0;
        while (true) {
            mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), kGemmWaitNs, abort);
            // the slot is held until the tile is written, so that its fields need no registers
            const GemmTile* tile = &sh.tile[tr.slot()];
            if (tile->rows == 0 || __any_sync(0xffffffffu, *abort)) break;
            const bool rows_here = rank * kBM + (warp & 3) * 32 < tile->rows;
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            uint32_t sc = 0;
#pragma unroll 1
            for (int kb = 0; kb < k1 - k0; kb += kStages) {
                if ((kb & (kScaleChunk - 1)) == 0) {
                    mbar_wait_warp<true>(sr.bar(scale_full), sr.phase(), kGemmWaitNs, abort);
                    sc = sc0 + sr.slot() * (kScaleChunk * 2 * kBM * 4);
                }
#pragma unroll
                for (int u = 0; u < kStages; ++u) {
                    if (kb + u >= k1 - k0) break;
                    const float f0 = ld_shared_f32(sc + u * (2 * kBM * 4));
                    const float f1 = kSwiglu ? ld_shared_f32(sc + u * (2 * kBM * 4) + kBM * 4) : f0;
                    mbar_wait_warp<true>(done + u * 8, done_phase >> u & 1, kGemmWaitNs, abort);
                    done_phase ^= 1u << u;
                    if (rows_here) {
                        tc_fence_after();
                        const uint32_t ad = lane_base + (u & 1) * kBN;
                        float v[32];
                        tmem_ld(ad + c0, v);
                        tmem_wait_ld(v);
                        fma_by(acc, v, f0);
                        tmem_ld(ad + c1, v);
                        tmem_wait_ld(v);
                        tc_fence_before();
                        __syncwarp();  // all loads are in registers: the accumulator is free
                        if (lane == 0) mbar_hand_back(free_bar + (u & 1) * 8);
                        fma_by(acc + 32, v, f1);
                    } else if (lane == 0) {
                        mbar_hand_back(free_bar + (u & 1) * 8);
                    }
                }
                sc += kStages * 2 * kBM * 4;
                if ((kb & (kScaleChunk - 1)) == kScaleChunk - kStages || kb + kStages >= k1 - k0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sr.bar(scale_empty));
                    ++sr.n;
                }
            }
            const int mine = tile->rows - rank * kBM;  // rows of this block, also none or more than kBM
            const int row0 = tile->row0 + rank * kBM, tn = tile->n;
            if constexpr (kSplit) {
                // the ring is idle now: the block's sums wait there for the cluster's
                if (r < mine) {
                    float* d = reinterpret_cast<float*>(tiles) + r * kSplitStride;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        *reinterpret_cast<float4*>(d + c0 + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                        *reinterpret_cast<float4*>(d + c1 + i) = make_float4(acc[32 + i], acc[33 + i], acc[34 + i], acc[35 + i]);
                    }
                }
            } else if constexpr (kSwiglu) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    acc[i] = silu_mul(acc[i], acc[32 + i]);
                    m = max_or_nan(m, fabsf(acc[i]));
                }
                // the block's maximum over all warpgroups' channels; two buffers: a
                // warp writes one again only after every warp has passed the other
                const int mx = tr.n & 1;
                sh.amax[mx][quarter][r] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.amax_full[mx]));
                mbar_wait_warp<true>(smem_u32(&sh.amax_full[mx]), tr.n >> 1 & 1, kGemmWaitNs, abort);
#pragma unroll
                for (int i = 0; i < kSumGroups; ++i) m = max_or_nan(m, sh.amax[mx][i][r]);
                const float scale = __fdiv_rn(m, 448.0f);
                const int64_t row = row0 + r;
                if (quarter == 0 && r < mine) a.out_scales[row * a.out_sstride + tn] = scale;
                if (kCtas == 2 && mine - (warp & 3) * 32 >= 32) {
                    // a full set of rows goes out as one copy (32 lanes' rows cost the stores a cycle each)
                    uint8_t* stage = out_stage + (warp - 4) * Shape::kOut;
                    bulk_wait_read<0>();  // lane 0's copy of the last tile has read the buffer
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        *reinterpret_cast<int4*>(stage + lane * 32 + q * 16) = quantize16_by(&acc[q * 16], scale);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&map_out, stage, tn * 128 + quarter * 32, row0 + (warp & 3) * 32);
                        bulk_commit();
                    }
                } else if (r < mine) {
                    uint8_t* o = reinterpret_cast<uint8_t*>(a.out) + row * a.out_stride + tn * 128 + quarter * 32;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        *reinterpret_cast<int4*>(o + q * 16) = quantize16_by(&acc[q * 16], scale);
                }
            } else if (rows_here) {
                const int n0 = tn * kBN + quarter * 64;
                uint8_t* stage = out_stage + (warp - 4) * Shape::kOut;
                const int rows = min(32, mine - (warp & 3) * 32);
                __nv_bfloat16* o =
                    reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(row0 + (warp & 3) * 32) * a.out_stride + n0;
                if constexpr (kCtas == 1) {
                    // 16 columns at a time: each lane its row's 32 bytes, a whole sector (128 rows a group: 222 us, by 16
                    // bytes 236), or twice 16 bytes, or, where rows are not so aligned, 8 columns through shared
                    // memory, so that 8 lanes store neighbours
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        __nv_bfloat162 p[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) p[i] = __floats2bfloat162_rn(acc[q * 16 + 2 * i], acc[q * 16 + 2 * i + 1]);
                        if (a.out_wide && n0 + 64 <= a.N) {
                            if (lane < rows) st_global_32(o + lane * a.out_stride + q * 16, reinterpret_cast<const uint32_t*>(p));
                            continue;
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = q * 16 + h * 8, n = n0 + at;
                            const int4 v = *reinterpret_cast<const int4*>(p + h * 4);
                            if (a.out_vec && n + 8 <= a.N) {
                                if (lane < rows) *reinterpret_cast<int4*>(o + lane * a.out_stride + at) = v;
                            } else if (n < a.N) {
                                *reinterpret_cast<int4*>(stage + lane * 16) = v;
                                __syncwarp();
                                const int c = lane & 7;
                                if (n + c < a.N)
                                    for (int i = lane >> 3; i < rows; i += 4)
                                        o[i * a.out_stride + at + c] = *reinterpret_cast<const __nv_bfloat16*>(stage + i * 16 + c * 2);
                                __syncwarp();
                            }
                        }
                    }
                } else {
                    // The warp's 32 rows x 64 columns through shared memory in the 128-byte swizzle.  A full
                    // set of rows goes out as one copy, which the next tile's products hide; the rows of
                    // a group's last tile, and unaligned rows, are stored by the lanes.  So are the last columns
                    // where N is no multiple of 8: a copy writes whole 16 bytes, also past the row's end.
                    bulk_wait_read<0>();  // lane 0's copy of the last tile has read the buffer
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        __nv_bfloat162 p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(acc[q * 8 + 2 * i], acc[q * 8 + 2 * i + 1]);
                        *reinterpret_cast<int4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = *reinterpret_cast<const int4*>(p);
                    }
                    if (a.out_vec && rows == 32 && (a.out_clip || n0 + 64 <= a.N)) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (n0 < a.N) tma_store_2d(&map_out, stage, n0 * 2, row0 + (warp & 3) * 32);
                            bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        auto at = [&](int i, int c) { return stage + i * 128 + (((c >> 3) ^ (i & 7)) << 4) + (c & 7) * 2; };
                        if (a.out_vec) {
                            const int c = (lane & 7) * 8;
                            for (int i = lane >> 3; i < rows; i += 4) {
                                const int4 v = *reinterpret_cast<const int4*>(at(i, c));
                                __nv_bfloat16* d = o + i * a.out_stride + c;
                                if (n0 + c + 8 <= a.N) {
                                    *reinterpret_cast<int4*>(d) = v;
                                } else {
                                    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&v);
                                    for (int j = 0; j < 8; ++j)
                                        if (n0 + c + j < a.N) d[j] = e[j];
                                }
                            }
                        } else {
                            for (int c = lane; c < 64 && n0 + c < a.N; c += 32)
                                for (int i = 0; i < rows; ++i)
                                    o[i * a.out_stride + c] = *reinterpret_cast<const __nv_bfloat16*>(at(i, c));
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(tr.bar(tile_empty));
            ++tr.n;
        }
        bulk_wait_all();
        if constexpr (kSplit) {
            __syncwarp();
            cluster_sync();
            // rows part, part + parts, ... of the tile, a warp each: the blocks' sums in block order.  Only
            // these warps have the registers for it; the others pass both barriers below
            const GemmTile tile = sh.tile[0];
            for (int r = part + parts * (warp - 4); r < tile.rows && !*abort; r += parts * kSumWarps) {
                const uint32_t at = smem_u32(tiles) + r * kSplitStride * 4;
                float v[8] = {};
                // four blocks' at a time
#pragma unroll 1
                for (int b0 = 0; b0 < parts; b0 += 4) {
                    if (kSwiglu || a.out_vec) {
                        // gate and up of 4 channels, or 8 neighbours
                        const int ca = kSwiglu ? lane * 4 : lane * 8, cb = kSwiglu ? 128 + lane * 4 : lane * 8 + 4;
                        float4 x[4], y[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < parts) {
                                x[b] = ld_cluster_f32x4(smem_of(at + ca * 4, b0 + b));
                                y[b] = ld_cluster_f32x4(smem_of(at + cb * 4, b0 + b));
                            }
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < parts) {
                                v[0] += x[b].x, v[1] += x[b].y, v[2] += x[b].z, v[3] += x[b].w;
                                v[4] += y[b].x, v[5] += y[b].y, v[6] += y[b].z, v[7] += y[b].w;
                            }
                    } else {  // column lane + 32 i: unaligned rows are stored 2 bytes a lane, neighbours by neighbours
                        float x[4][8];
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < parts)
#pragma unroll
                                for (int i = 0; i < 8; ++i) x[b][i] = ld_cluster_f32(smem_of(at + (lane + 32 * i) * 4, b0 + b));
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < parts)
#pragma unroll
                                for (int i = 0; i < 8; ++i) v[i] += x[b][i];
                    }
                }
                const int64_t row = tile.row0 + r;
                if constexpr (kSwiglu) {
                    float h[16] = {}, m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[i] = silu_mul(v[i], v[4 + i]);
                        m = max_or_nan(m, fabsf(h[i]));
                    }
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float scale = __fdiv_rn(m, 448.0f);
                    uint8_t* o = reinterpret_cast<uint8_t*>(a.out) + row * a.out_stride + tile.n * 128 + lane * 4;
                    *reinterpret_cast<int*>(o) = quantize16_by(h, scale).x;
                    if (lane == 0) a.out_scales[row * a.out_sstride + tile.n] = scale;
                } else {
                    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.out_stride;
                    const int n0 = tile.n * kBN + lane * 8;
                    if (a.out_vec && n0 + 8 <= a.N) {
                        __nv_bfloat162 p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                        *reinterpret_cast<int4*>(o + n0) = *reinterpret_cast<const int4*>(p);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int n = a.out_vec ? n0 + i : tile.n * kBN + lane + 32 * i;
                            if (n < a.N) o[n] = __float2bfloat16_rn(v[i]);
                        }
                    }
                }
            }
            __syncwarp();
            cluster_sync();  // no block ends while another reads its sums
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free<kCtas>(tmem, 512);
    if (tid == 0 && *abort && a.status) flag(a.status, FLAG_TIMEOUT);
    __syncwarp();
    if (kCtas == 2) cluster_sync();  // neither block ends while the other still frees
}

// ---- host -------------------------------------------------------------------------
static ep_status check_products(const char* fn, const ep_fp8_rows* x, const ep_row_groups* g, const ep_fp8_weight* w,
                                const uint32_t* status_out) {
    if (!x || !g || !w) return set_error(EP_ERR_INVALID_ARG, "%s: null descriptor", fn);
    if (w->groups < 1 || w->groups > kMaxGroups)
        return set_error(EP_ERR_INVALID_ARG, "%s: groups %d outside 1..%d", fn, w->groups, kMaxGroups);
    if (w->n < 1 || w->n > 0x7fffffff - kBN || w->k < 128 || w->k % 128)
        return set_error(EP_ERR_INVALID_ARG, "%s: weight rows %d, channels %d (a multiple of 128)", fn, w->n, w->k);
    if (!w->codes || !w->scales || !aligned16(w->codes))
        return set_error(EP_ERR_INVALID_ARG, "%s: weight codes (16-byte aligned) and scales are required", fn);
    if (x->rows < 0 || x->rows > 0x7fffffff - 2 * kBM)
        return set_error(EP_ERR_INVALID_ARG, "%s: %lld rows", fn, (long long)x->rows);
    if (x->rows > 0) {
        if (!x->codes || !x->scales || !aligned16(x->codes))
            return set_error(EP_ERR_INVALID_ARG, "%s: row codes (16-byte aligned) and scales are required", fn);
        if (x->code_stride < w->k || x->code_stride % 16 || x->scale_stride < w->k / 128)
            return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld, %lld for %d channels", fn, (long long)x->code_stride,
                             (long long)x->scale_stride, w->k);
    }
    if (!aligned_to(w->scales, 4) || !aligned_to(x->scales, 4) || !aligned_to(g->counts, 4) || !aligned_to(g->offsets, 4) ||
        !aligned_to(g->bases, 4) || !aligned_to(status_out, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: a pointer is not aligned to its elements", fn);
    if (g->bases && g->per_base < 1) return set_error(EP_ERR_INVALID_ARG, "%s: groups per base %d", fn, g->per_base);
    if (g->stride < 0 || g->expected < 0)
        return set_error(EP_ERR_INVALID_ARG, "%s: group stride %lld, expected rows %lld", fn, (long long)g->stride, (long long)g->expected);
    return EP_OK;
}

template <bool kSwiglu, int kCtas, bool kSplit>
static ep_status launch_shape(const char* fn, const CUtensorMap& map_x, const CUtensorMap& map_w,
                              const CUtensorMap& map_out, GemmArgs a, int sms,
                              int cluster, void* stream) {
    using Shape = GemmShape<kCtas>;
    const int64_t most = most_tiles(a, Shape::kTileM);
    if (most > kMaxTiles) return set_error(EP_ERR_INVALID_ARG, "%s: %lld tiles", fn, (long long)most);
    a.most = (int)most;
    int dev = 0;
    EP_CUDA(cudaGetDevice(&dev));
    static std::atomic<bool> known[kMaxDevicesTracked];  // devices whose launch attribute is set
    if (dev >= kMaxDevicesTracked || !known[dev].load(std::memory_order_relaxed)) {
        EP_CUDA(cudaFuncSetAttribute(gemm_kernel<kSwiglu, kCtas, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem));
        if (dev < kMaxDevicesTracked) known[dev].store(true, std::memory_order_relaxed);
    }
    const int units = (int)(most < sms / cluster ? most : sms / cluster);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = Shape::kSmem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    EP_CUDA(cudaLaunchKernelEx(&cfg, gemm_kernel<kSwiglu, kCtas, kSplit>, map_x, map_w, map_out, a));
    return EP_OK;
}

// Blocks that share a tile's K where the tiles are few: by 4 or 2 if that needs no more than the SMs and leaves
// each two blocks of K.  Clusters of other sizes leave some SMs of a group of SMs without one, and a second wave
// doubles the time, so that they may take only a part of the SMs; beyond 4 a block keeps more blocks of K.
// One row, us by 4 or 2 / by this: K 7168, N 256 10.2 / 7.8 (8), 2048 10.4 / 8.8 (8), 4096 10.7 / 10.4 (6; by 8
// 16.8), 5120 11.8 / 11.1 (5), 10240 18.6 / 14.5 (3); K 16384, N 256 16.7 / 11.1 (8), 4096 17.4 / 14.9 (6).
static int split_of(int64_t tiles, int kb, int sms) {
    struct Rule { int split, blocks, percent; };  // blocks of K for each, share of the SMs
    for (const Rule r : {Rule{8, 4, 66}, {6, 8, 66}, {5, 8, 66}, {4, 2, 100}, {3, 2, 80}, {2, 2, 100}})
        if (kb >= r.split * r.blocks && tiles * r.split * 100 <= (int64_t)sms * r.percent) return r.split;
    return 1;
}

// Whether pairs of blocks make the tiles: where they need fewer tiles, 1.75 times or better (one of theirs costs 1.6
// to 1.75).  40 groups, us by one block / by pairs, K 2048, N 7168: 64 rows a group 103 / 128, 128 120 / 141, 256
// 169 / 148, 320 215 / 262, 384 235 / 258, 448 308 / 260, 512 304 / 266, 576 358 / 375, 640 384 / 389, 704 454 / 391,
// 896 521 / 502, 1024 587 / 497; first product, K 7168, 2I 4096: 64 200 / 248, 256 300 / 286, 320 381 / 482, 448
// 548 / 475, 576 646 / 674, 640 643 / 666, 704 774 / 663, 896 880 / 880, 1024 1058 / 902.
static bool by_pairs(int64_t rows) {
    if (rows > 0x7fffffff) return true;
    const int64_t one = (rows + kBM - 1) / kBM, two = (rows + 2 * kBM - 1) / (2 * kBM);
    return one * 4 >= two * 7;
}

template <bool kSwiglu>
static ep_status launch_gemm(const char* fn, const ep_fp8_rows* x, const ep_row_groups* g, const ep_fp8_weight* w,
                             GemmArgs a, void* stream) {
    a.x_scales = x->scales;
    a.x_sstride = x->scale_stride;
    a.x_vec = aligned16(x->scales) && x->scale_stride % 4 == 0;
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
    CUtensorMap map_x, map_w, map_out;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)w->k, (cuuint64_t)x->rows};
        const cuuint64_t strides[1] = {(cuuint64_t)x->code_stride};
        const cuuint32_t box[2] = {kBK, kBoxRows};
        const ep_status st = encode_rows(&map_x, x->codes, 2, dims, strides, box, fn);
        if (st != EP_OK) return st;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)w->k, (cuuint64_t)w->n, (cuuint64_t)w->groups};
        const cuuint64_t strides[2] = {(cuuint64_t)w->k, (cuuint64_t)w->k * (cuuint64_t)w->n};
        const cuuint32_t box[3] = {kBK, 128, 1};
        const ep_status st = encode_rows(&map_w, w->codes, 3, dims, strides, box, fn);
        if (st != EP_OK) return st;
    }
    map_out = map_x;  // used by pairs of blocks only
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const int split = split_of(most_tiles(a, kBM), a.KB, sms);
    if (split > 1) return launch_shape<kSwiglu, 1, true>(fn, map_x, map_w, map_out, a, sms, split, stream);
    // Rows of a group: as the caller expects, or what the arrays hold, shared out.  Regions with counts, as the
    // packed layout has, are sized for the worst case: a low-latency step fills a few percent of them.
    const int64_t per_group =
        g->expected > 0 ? g->expected : x->rows / w->groups / (w->groups > 1 && !g->offsets && g->counts ? 16 : 1);
    if (by_pairs(per_group)) {
        if (kSwiglu || a.out_vec) {
            constexpr int kBytes = kSwiglu ? 1 : 2;
            const cuuint64_t dims[2] = {(cuuint64_t)(kSwiglu ? w->n / 2 : w->n) * kBytes, (cuuint64_t)x->rows};
            const cuuint64_t strides[1] = {(cuuint64_t)a.out_stride * kBytes};
            const cuuint32_t box[2] = {kSwiglu ? 32 : 128, 32};
            const ep_status st = encode_rows(&map_out, a.out, 2, dims, strides, box, fn,
                                             kSwiglu ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
            if (st != EP_OK) return st;
        }
        return launch_shape<kSwiglu, 2, false>(fn, map_x, map_w, map_out, a, sms, 2, stream);
    }
    return launch_shape<kSwiglu, 1, false>(fn, map_x, map_w, map_out, a, sms, 1, stream);
}

}  // namespace ep

using namespace ep;

extern "C" ep_status ep_expert_gemm(const ep_fp8_rows* x, const ep_row_groups* groups, const ep_fp8_weight* w, void* out,
                                    int64_t out_stride, uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_gemm";
    const ep_status st = check_products(fn, x, groups, w, status_out);
    if (st != EP_OK) return st;
    if (x->rows == 0) return EP_OK;
    if (!out || out_stride < w->n) return set_error(EP_ERR_INVALID_ARG, "%s: output stride %lld for %d channels", fn, (long long)out_stride, w->n);
    if (reinterpret_cast<uintptr_t>(out) & 1) return set_error(EP_ERR_INVALID_ARG, "%s: output is not 2-byte aligned", fn);
    GemmArgs a{};
    a.out = out;
    a.out_stride = out_stride;
    a.out_vec = aligned16(out) && out_stride % 8 == 0;
    a.out_wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && out_stride % 16 == 0;
    a.out_clip = w->n % 8 == 0;
    a.status = status_out;
    return launch_gemm<false>(fn, x, groups, w, a, stream);
}

extern "C" ep_status ep_expert_swiglu(const ep_fp8_rows* x, const ep_row_groups* groups, const ep_fp8_weight* w13, uint8_t* out,
                                      int64_t out_stride, float* out_scales, int64_t out_scale_stride,
                                      uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_swiglu";
    const ep_status st = check_products(fn, x, groups, w13, status_out);
    if (st != EP_OK) return st;
    if (w13->n % 256) return set_error(EP_ERR_INVALID_ARG, "%s: %d weight rows (gate and up, each a multiple of 128)", fn, w13->n);
    if (x->rows == 0) return EP_OK;
    const int inter = w13->n / 2;
    if (!out || !out_scales || !aligned16(out) || !aligned_to(out_scales, 4) || out_stride < inter || out_stride % 16 || out_scale_stride < inter / 128)
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
