// ep_fp4.cu -- MXFP4 rows and the experts' products on them: quantisation, y = x w^T per group of
// rows, and the first product with its activation and requantisation fused.
//
// Mathematics.  Row r, output channel n, blocks b of 32 along K, codes x, w (e2m1) and E8M0 bytes:
//   y[r][n] = sum_b 2^(sx[r][b] - 127) 2^(sw[n][b] - 127) sum_{k in b} x[r][k] w[n][k]
// which tcgen05.mma computes whole (kind::mxf4, block scales from tensor memory, fp32 sums), so that the
// accumulator leaves tensor memory once a tile, not once a block of K.
//
// Shape.  128 rows x 192 or 224 weight rows a tile (64 or 128 where that fills the SMs better: fp4_choice): tensor memory
// then holds two accumulators and the scales beside them, so that a tile is written while the next is multiplied.  One warp
// copies codes (a stage is 256 of K, 128 bytes a row), four stage scales: each thread loads its rows' bytes and
// writes them where tcgen05.cp reads them (32 rows of 16 bytes: row r's four bytes at (r % 32) * 16 + r / 32 * 4),
// one issues copies of scales and products, four write the results.
//
// Bound.  Up to 128 rows a group the weights' bytes: 256 groups of about 64 rows, K 7168, 2I 4096 594 us, K 2048, N 7168
// 324 us, 6.7 TB/s.  With long groups shared memory: a stage's codes are written to it and read from it once, 82 KB at
// 128 bytes a cycle = 640 cycles for 192 weight rows, and a stage takes 650 (the products some 370).  Pairs of blocks share
// the weight's rows, 56 KB a stage and SM: first product, 40 groups of 2048 rows, 914 us by one block, 737 by pairs (6.5
// PFLOP/s); the second 541 us by 192 weight rows a tile, 500 by 224, 406 by pairs (5.9 PFLOP/s, results included).  A long run
// of such products meets the board's power limit (65536 rows to 256 groups, first product: 976 us at first, 1060 to 1100 later).
// A fifth stage changes nothing, weights fetched ahead into the second-level cache cost time.  With few tiles, what one
// SM brings in from memory: one row, K 7168, N 4096 11.2 us by 64 blocks, 8.3 by 128 in clusters of two.
#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "ep_fp4.cuh"
#include "ep_groups.cuh"

namespace ep {

constexpr int k4BM = 128;         // rows of a tile
constexpr int k4BK = 256;         // codes of K a stage: 128 bytes a row
constexpr int k4BoxRows = 32;     // rows of one copy of x
constexpr int k4ScaleWarps = 4, k4OutWarps = 4;
constexpr int k4Threads = 128 + 32 * (k4ScaleWarps + k4OutWarps);
constexpr int kSplitRow = 64 + 4;  // floats of a row of sums: rows fall into other banks
constexpr int k4TileRing = 4;
constexpr int k4Group = 2;        // stages whose scales are staged together
constexpr int64_t k4WaitNs = 2000000000ll;

// kCtas = 2: a pair of blocks makes a tile of 256 rows, each with its own rows and half of the weight's, and with the
// scales of all of the weight's.  The first issues the products of both, which read both blocks' memory: the second's
// copies count on the first's barriers, and one of its warps tells the first of scales in place, by a release at cluster
// scope that covers shared memory (us, 40 groups of 2048 rows, first / second product: 739 / 406; by the scales' warps
// themselves 758 / 408; by two warps with a release of all memory 910 / 447; stage by stage for codes and scales, with
// a release at block scope, which does not reach the other block, 736 / 461).
template <bool kSwiglu, int kBN, int kCtas>
struct Fp4Shape {
    static constexpr int kTileM = kCtas * k4BM;
    static constexpr int kChunks = (kBN + 127) / 128;               // of 128 weight rows' scales
    static constexpr int kCodesA = k4BM * 128, kCodesB = kBN / kCtas * 128, kCodes = kCodesA + kCodesB;
    static constexpr int kScalesA = 2 * 512, kScalesB = 2 * kChunks * 512, kScales = kScalesA + kScalesB;  // [128 of K][chunk][32][16]
    static constexpr int kSlot = k4Group * kScales;                 // the scales that are staged together
    static constexpr int kSlots = kSwiglu || kCtas == 2 ? 4 : 2;    // no stage less for the four of a pair
    static constexpr int kOut = kSwiglu ? 0 : 32 * 64;              // of a warp's output on its way: 32 rows of 32 columns
    static constexpr int kRest = kSlots * kSlot + k4OutWarps * kOut;
    static constexpr int kStages = (225 * 1024 - kRest) / kCodes < 8 ? (225 * 1024 - kRest) / kCodes : 8;
    static constexpr size_t kSmem = 1024 + kStages * kCodes + kRest;
    // columns of tensor memory: two accumulators, then two sets of scales in turn
    static constexpr int kScaleCols = 8 + 2 * kChunks * 4, kScaleAt = 2 * kBN;
    static constexpr int kCols = 2 * kBN + 2 * kScaleCols > 256 ? 512 : 256;
};

struct Fp4Args : TileArgs {
    const uint8_t* x_scales;
    int64_t x_sstride;
    const uint8_t* w_scales;
    int N, K, KT;       // KT: stages of K
    void* out;          // bf16 rows, or codes
    int64_t out_stride; // elements; codes: bytes
    uint8_t* out_scales;
    int64_t out_sstride;
    bool out_vec;             // 16-byte stores
    bool out_clip;            // rows end at a multiple of 16 bytes, so that a copy that crosses their end is cut there
    int x_vec, w_vec;         // bytes of scales that a load may take: 32, 16 or 4
    uint32_t* status;
};

template <int kStages, int kSlots>
struct Fp4Shared {
    uint64_t full[kStages], done[kStages], scale_full[kSlots], scale_empty[kSlots], acc_full[2], acc_empty[2];
    uint64_t tile_full[k4TileRing], tile_empty[k4TileRing], drain;
    uint32_t tmem;
    int abort;
    GemmTile tile[k4TileRing];
};

// A ring of kSize slots, kSize any number.
template <int kSize>
struct Turn {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == kSize) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// 32 bytes of scales, four stages', from byte `at` of a row with `bytes` of them (a multiple of 4); 0 past its end.  Plain
// loads, since the kernel before may still write them when this one is launched; by the first-level cache (past it: 256
// groups of about 64 rows, first product 603 us for 599).
struct Scales32 {
    uint32_t v[8];
};
__device__ __forceinline__ Scales32 load_scales(const uint8_t* row, int at, int bytes, int vec) {
    Scales32 s;
    if (vec == 32 && at % 32 == 0 && at + 32 <= bytes) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(s.v[0]), "=r"(s.v[1]), "=r"(s.v[2]), "=r"(s.v[3]), "=r"(s.v[4]), "=r"(s.v[5]), "=r"(s.v[6]), "=r"(s.v[7])
                     : "l"(row + at));
        return s;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        if (vec >= 16 && at + i * 4 + 16 <= bytes) {
            const uint4 q = *reinterpret_cast<const uint4*>(row + at + i * 4);
            s.v[i] = q.x, s.v[i + 1] = q.y, s.v[i + 2] = q.z, s.v[i + 3] = q.w;
        } else {
#pragma unroll
            for (int j = i; j < i + 4; ++j) s.v[j] = at + j * 4 < bytes ? *reinterpret_cast<const uint32_t*>(row + at + j * 4) : 0;
        }
    }
    return s;
}

// kSwiglu: half of the tile's weight rows are gate rows, half the up rows of the same channels.
// kSplit (kBN = 64, one block): the blocks of a cluster make one tile, each from its share of the stages, two by two.  For
// launches with fewer tiles than SMs: a block alone brings in some 45 GB/s from memory, whatever it has under way.  Every
// cluster has at most one tile.
template <bool kSwiglu, int kBN, int kCtas, bool kSplit>
__global__ void __launch_bounds__(k4Threads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_box,
                const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_out, const Fp4Args a) {
    using Shape = Fp4Shape<kSwiglu, kBN, kCtas>;
    constexpr int kStages = Shape::kStages, kSlots = Shape::kSlots, kCodes = Shape::kCodes, kScales = Shape::kScales, kHalf = kBN / 2, kTileM = Shape::kTileM;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Fp4Shared<kStages, kSlots> sh;
    // codes of all stages first, each on 1024 bytes; then the scales, then the rows on their way out
    uint8_t* codes = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    uint8_t* scales = codes + kStages * kCodes;
    uint8_t* out_stage = scales + kSlots * Shape::kSlot;  // on 1024 bytes too
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
    const int part = kSplit ? (int)cluster_rank() : 0, parts = kSplit ? cluster_size() : 1;
    const int unit = blockIdx.x / (kCtas * parts), units = gridDim.x / (kCtas * parts);
    const int pairs = (a.KT + k4Group - 1) / k4Group;
    const int kt0 = kSplit ? part * pairs / parts * k4Group : 0, kt1 = kSplit ? min((part + 1) * pairs / parts * k4Group, a.KT) : a.KT;
    volatile int* abort = &sh.abort;
    const uint32_t full = smem_u32(sh.full), done = smem_u32(sh.done);
    const uint32_t scale_full = smem_u32(sh.scale_full), scale_empty = smem_u32(sh.scale_empty);
    const uint32_t acc_full = smem_u32(sh.acc_full), acc_empty = smem_u32(sh.acc_empty);
    const uint32_t tile_full = smem_u32(sh.tile_full), tile_empty = smem_u32(sh.tile_empty);

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.done[s], 1);
        }
        for (int b = 0; b < kSlots; ++b) {
            mbar_init(&sh.scale_full[b], k4ScaleWarps + (kCtas == 2 && rank == 0 ? 1 : 0));  // its own, and what the other block of a pair tells
            mbar_init(&sh.scale_empty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], kCtas * k4OutWarps);
        }
        for (int b = 0; b < k4TileRing; ++b) {
            mbar_init(&sh.tile_full[b], 1);
            mbar_init(&sh.tile_empty[b], 2 + k4ScaleWarps + k4OutWarps);
            sh.tile[b].rows = 0;
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_box);
        tma_prefetch_desc(&map_w);
    }
    if (warp == 2) tmem_alloc<kCtas>(&sh.tmem, Shape::kCols);
    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();  // both blocks' barriers are ready
    tc_fence_after();
    // All above may run beside the end of the kernel before; the kernel after may do the same.
    grid_wait();
    grid_launch_next();
    const uint32_t tmem = sh.tmem;

    if (warp == 3) {
        // ---- tiles
        TileWalk<kTileM> walk;
        RingPos<k4TileRing> tr;
        for (int t = unit;; t += units) {
            GemmTile tile = {0, 0, 0, 0};
            const bool some = walk.find(a, min(t, a.most), lane, &tile);
            if (t >= a.most) tile.rows = 0;  // groups that overlap may have any number of tiles
            mbar_wait_warp<true>(tr.bar(tile_empty), tr.phase() ^ 1, k4WaitNs, abort);
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
        }
        if (walk.cut && a.status && blockIdx.x == 0) flag(a.status, FLAG_CAPACITY);
    } else if (warp == 0) {
        if (lane == 0) {
            // ---- copies of codes; a whole tile's rows come as one copy (as four of 32: 1024 rows a group, first product 513 us
            // for 464)
            RingPos<k4TileRing> tr;
            Turn<kStages> st;
            bool ok = true;
            while (ok) {
                if (!mbar_wait_or_abort<true>(tr.bar(tile_full), tr.phase(), k4WaitNs, abort)) break;
                const GemmTile tile = sh.tile[tr.slot()];
                mbar_arrive(tr.bar(tile_empty));
                ++tr.n;
                if (tile.rows == 0) break;
                const int rows = min(tile.rows - rank * k4BM, k4BM), row = tile.row0 + rank * k4BM;
                const int boxes = (max(rows, 0) + k4BoxRows - 1) / k4BoxRows;
                uint32_t bytes = boxes * k4BoxRows * 128 + Shape::kCodesB;
                if (kCtas == 2)  // a pair's bytes all count on the first block's barriers
                    bytes += (max(tile.rows - k4BM, 0) + k4BoxRows - 1) / k4BoxRows * k4BoxRows * 128 + Shape::kCodesB;
                const uint32_t full0 = kCtas == 2 ? smem_of(full, 0) : full;
                // the first block of a pair has the gate rows, or the first half, the second the others
                const int first = kSwiglu ? tile.n * kHalf : tile.n * kBN, second = kSwiglu ? a.N / 2 + first : first + kHalf;
                const int w0 = rank ? second : first;
                for (int kt = kt0; kt < kt1; ++kt) {
                    if (!mbar_wait_or_abort<true>(done + st.slot * 8, st.phase ^ 1, k4WaitNs, abort)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = codes + st.slot * kCodes;
                    const uint32_t bar = full0 + st.slot * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&sh.full[st.slot], bytes);
                    tma_load_3d<kCtas>(sa + Shape::kCodesA, &map_w, kt * 128, w0, tile.g, bar);
                    if (kSwiglu && kCtas == 1) tma_load_3d<1>(sa + Shape::kCodesA + kHalf * 128, &map_w, kt * 128, second, tile.g, bar);
                    if (boxes == k4BM / k4BoxRows) tma_load_2d<kCtas>(sa, &map_x, kt * 128, row, bar);
                    else
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d<kCtas>(sa + b * k4BoxRows * 128, &map_box, kt * 128, row + b * k4BoxRows, bar);
                    st.next();
                }
            }
            // no copy may be in flight when the blocks end, also after a wait that ran out: the last phase that
            // a stage's copies complete is the one before its next
            for (int u = 0; u < kStages && rank == 0; ++u) {
                mbar_wait_bounded(&sh.full[st.slot], st.phase ^ 1, k4WaitNs);
                st.next();
            }
            // The first block may have given up before it counted the second's last ones, which land in microseconds.
            if (rank != 0 && *abort)
                for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {
                }
        }
    } else if (warp == 1 && rank != 0) {
        // ---- the second block's scales are in place: told to the first block
        const uint32_t told = smem_of(scale_full, 0);
        RingPos<k4TileRing> tr;
        Turn<kSlots> sl;
        while (true) {
            mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), k4WaitNs, abort);
            const int rows = sh.tile[tr.slot()].rows;
            __syncwarp();
            if (lane == 0) mbar_arrive(tr.bar(tile_empty));
            ++tr.n;
            if (rows == 0 || __any_sync(0xffffffffu, *abort)) break;
#pragma unroll 1
            for (int kt = 0; kt < a.KT; kt += k4Group) {
                mbar_wait_warp<true>(scale_full + sl.slot * 8, sl.phase, k4WaitNs, abort);
                if (lane == 0) mbar_arrive_mate(told + sl.slot * 8);
                sl.next();
            }
        }
    } else if (warp == 1) {
        // ---- copies of scales into tensor memory, products: for both blocks of a pair by the first
        constexpr uint32_t idesc0 = idesc_mxf4(kTileM, kBN, 0), idesc2 = idesc_mxf4(kTileM, kBN, 2);
        const uint64_t da0 = smem_desc_sw128(codes), db0 = smem_desc_sw128(codes + Shape::kCodesA), ds0 = smem_desc_rows16(scales);
        RingPos<k4TileRing> tr;
        Turn<kStages> st;
        Turn<kSlots> sl;
        while (true) {
            mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), k4WaitNs, abort);
            const int rows = sh.tile[tr.slot()].rows;
            __syncwarp();
            if (lane == 0) mbar_arrive(tr.bar(tile_empty));
            const uint32_t c = tr.n & 1, turn = tr.n >> 1 & 1;
            ++tr.n;
            if (rows == 0 || __any_sync(0xffffffffu, *abort)) break;
            mbar_wait_warp<true>(acc_empty + c * 8, turn ^ 1, k4WaitNs, abort);
            // two stages, one group of scales, at a time (one: pairs, 2048 rows a group 755 us for 737)
#pragma unroll 1
            for (int kt = kt0; kt < kt1; kt += k4Group) {
                const bool two = kt + 1 < kt1;
                const Turn<kStages> st0 = st;
                st.next();
                mbar_wait_warp<true, kCtas == 2>(scale_full + sl.slot * 8, sl.phase, k4WaitNs, abort);
                mbar_wait_warp<true, kCtas == 2>(full + st0.slot * 8, st0.phase, k4WaitNs, abort);
                if (two) mbar_wait_warp<true, kCtas == 2>(full + st.slot * 8, st.phase, k4WaitNs, abort);
                if (kCtas == 2) fence_acquire_mate();
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ds = ds0 + sl.slot * (Shape::kSlot >> 4);
#pragma unroll
                    for (int g = 0; g < k4Group; ++g) {
                        const uint32_t sa = tmem + Shape::kScaleAt + g * Shape::kScaleCols;
#pragma unroll
                        for (int h = 0; h < 2 + 2 * Shape::kChunks; ++h)  // the rows' two, then the weights', as they lie
                            tmem_copy_scales<kCtas>(sa + h * 4, ds + g * (kScales >> 4) + h * 32);
                    }
#pragma unroll
                    for (int g = 0; g < k4Group; ++g) {
                        if (g == 1 && !two) break;
                        const uint32_t sa = tmem + Shape::kScaleAt + g * Shape::kScaleCols, sb = sa + 8;
                        const int slot = g ? st.slot : st0.slot;
                        const uint32_t at = slot * (kCodes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_mxf4<kCtas>(tmem + c * kBN, da0 + at + k * 2, db0 + at + k * 2, k & 1 ? idesc2 : idesc0, sa + (k >> 1) * 4,
                                            sb + (k >> 1) * 4 * Shape::kChunks, kt > kt0 || g > 0 || k > 0);
                        mma_commit<kCtas>(done + slot * 8);
                    }
                    mma_commit<kCtas>(scale_empty + sl.slot * 8);
                    if (kt + k4Group >= kt1) mma_commit<kCtas>(acc_full + c * 8);
                }
                __syncwarp();
                if (two) st.next();
                sl.next();
            }
        }
        // every product has finished before either block frees its tensor memory: the second waits for this one below
        if (elect_one()) mma_commit_here<kCtas>(smem_u32(&sh.drain));
        __syncwarp();
        mbar_wait_bounded(&sh.drain, 0, k4WaitNs);
    } else if (warp >= 4 && warp < 4 + k4ScaleWarps) {
        // ---- scales: thread r those of row r, and of weight rows r and 128 + r.  A load takes four stages' (a whole sector)
        // and the next is on its way; two stages' are shown to the tensor cores with one fence
        constexpr int kAhead = 2;
        const int r = tid - 128, bytes = a.K / 32;
        RingPos<k4TileRing> tr;
        Turn<kSlots> sl;
        const uint32_t to = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
        while (true) {
            mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), k4WaitNs, abort);
            const GemmTile tile = sh.tile[tr.slot()];
            __syncwarp();
            if (lane == 0) mbar_arrive(tr.bar(tile_empty));
            ++tr.n;
            if (tile.rows == 0 || __any_sync(0xffffffffu, *abort)) break;
            auto weight_row = [&](int i) {  // of the group, or -1
                if (i >= kBN) return -1;
                const int n = !kSwiglu ? tile.n * kBN + i : i < kHalf ? tile.n * kHalf + i : a.N / 2 + tile.n * kHalf + i - kHalf;
                return n < a.N ? n : -1;
            };
            const int n0 = weight_row(r), n1 = weight_row(128 + r);
            const int row = rank * k4BM + r;
            const uint8_t* px = row < tile.rows ? a.x_scales + (int64_t)(tile.row0 + row) * a.x_sstride : nullptr;
            const uint8_t* p0 = n0 >= 0 ? a.w_scales + ((int64_t)tile.g * a.N + n0) * bytes : nullptr;
            const uint8_t* p1 = n1 >= 0 ? a.w_scales + ((int64_t)tile.g * a.N + n1) * bytes : nullptr;
            Scales32 vx[kAhead], v0[kAhead], v1[kAhead];
            auto fetch = [&](int i, int at) {
#pragma unroll
                for (int j = 0; j < 8; ++j) vx[i].v[j] = v0[i].v[j] = v1[i].v[j] = 0;
                if (at >= bytes) return;
                if (px) vx[i] = load_scales(px, at, bytes, a.x_vec);
                if (p0) v0[i] = load_scales(p0, at, bytes, a.w_vec);
                if (Shape::kChunks > 1 && p1) v1[i] = load_scales(p1, at, bytes, a.w_vec);
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, kt0 * 8 + i * 32);
#pragma unroll 1
            for (int kt = kt0; kt < kt1; kt += 4 * kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; j += k4Group) {
                        if (kt + 4 * i + j >= kt1) break;
                        mbar_wait_warp<true>(scale_empty + sl.slot * 8, sl.phase ^ 1, k4WaitNs, abort);
                        uint8_t* d = scales + sl.slot * Shape::kSlot + to;
#pragma unroll
                        for (int h = j; h < j + k4Group; ++h, d += kScales) {
                            *reinterpret_cast<uint32_t*>(d) = vx[i].v[2 * h];
                            *reinterpret_cast<uint32_t*>(d + 512) = vx[i].v[2 * h + 1];
                            uint8_t* db = d + Shape::kScalesA;
                            *reinterpret_cast<uint32_t*>(db) = v0[i].v[2 * h];
                            *reinterpret_cast<uint32_t*>(db + 512 * Shape::kChunks) = v0[i].v[2 * h + 1];
                            if (Shape::kChunks > 1) {
                                *reinterpret_cast<uint32_t*>(db + 512) = v1[i].v[2 * h];
                                *reinterpret_cast<uint32_t*>(db + 512 * 3) = v1[i].v[2 * h + 1];
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(scale_full + sl.slot * 8);
                        sl.next();
                    }
                    fetch(i, kt * 8 + (kAhead + i) * 32);
                }
            }
        }
    } else if (warp >= 4 + k4ScaleWarps) {
        // ---- results: a lane a row
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), free_bar = kCtas == 2 ? smem_of(acc_empty, 0) : acc_empty;
        uint8_t* stage = out_stage + (warp & 3) * Shape::kOut;
        RingPos<k4TileRing> tr;
        while (true) {
            mbar_wait_warp<true>(tr.bar(tile_full), tr.phase(), k4WaitNs, abort);
            const GemmTile tile = sh.tile[tr.slot()];
            __syncwarp();
            if (lane == 0) mbar_arrive(tr.bar(tile_empty));
            const uint32_t c = tr.n & 1, turn = tr.n >> 1 & 1;
            ++tr.n;
            if (tile.rows == 0 || __any_sync(0xffffffffu, *abort)) break;
            mbar_wait_warp<true>(acc_full + c * 8, turn, k4WaitNs, abort);
            tc_fence_after();
            const int first = rank * k4BM + (warp & 3) * 32, rows = min(32, tile.rows - first);  // of this warp
            if (rows > 0) {
                const int64_t row0 = tile.row0 + first;
                if constexpr (kSplit) {
                    // the ring is idle now: the block's sums wait there for the cluster's
                    float* d = reinterpret_cast<float*>(codes) + (first + lane) * kSplitRow;
#pragma unroll
                    for (int q = 0; q < kBN / 32; ++q) {
                        float v[32];
                        tmem_ld(lanes + c * kBN + q * 32, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(d + q * 32 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                } else if constexpr (kSwiglu) {
                    for (int q = 0; q < kHalf / 32; ++q) {
                        const int ch = tile.n * kHalf + q * 32;
                        if (ch >= a.N / 2) break;
                        float g[32], u[32];
                        tmem_ld(lanes + c * kBN + q * 32, g);
                        tmem_ld(lanes + c * kBN + kHalf + q * 32, u);
                        tmem_wait_ld(g);
                        tmem_wait_ld(u);
                        float m = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            g[i] = silu_mul(g[i], u[i]);
                            m = max_or_nan(m, fabsf(g[i]));
                        }
                        const uint32_t b = e8m0_of(m);
                        const float by = e8m0_inverse(b);
                        if (lane < rows) {
                            const int4 v = make_int4((int)e2m1x8(g, by), (int)e2m1x8(g + 8, by), (int)e2m1x8(g + 16, by), (int)e2m1x8(g + 24, by));
                            *reinterpret_cast<int4*>(static_cast<uint8_t*>(a.out) + (row0 + lane) * a.out_stride + ch / 2) = v;
                            a.out_scales[(row0 + lane) * a.out_sstride + ch / 32] = (uint8_t)b;
                        }
                    }
                } else {
                    // 32 columns at a time through shared memory in the 64-byte swizzle.  A full set of rows goes out as one
                    // copy, which the next columns hide; the rows of a group's last tile, and unaligned rows, by the lanes,
                    // neighbours by neighbours.  So are the last columns where N is no multiple of 8: a copy writes whole 16
                    // bytes, also past the row's end.
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + row0 * a.out_stride;
                    for (int q = 0; q < kBN / 32; ++q) {
                        const int n0 = tile.n * kBN + q * 32;
                        if (n0 >= a.N) break;
                        float v[32];
                        tmem_ld(lanes + c * kBN + q * 32, v);
                        bulk_wait_read<0>();  // lane 0's copy of the columns before has read the buffer
                        tmem_wait_ld(v);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            __nv_bfloat162 p[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) p[j] = __floats2bfloat162_rn(v[i * 8 + 2 * j], v[i * 8 + 2 * j + 1]);
                            *reinterpret_cast<int4*>(stage + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = *reinterpret_cast<const int4*>(p);
                        }
                        if (a.out_vec && rows == 32 && (a.out_clip || n0 + 32 <= a.N)) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_2d(&map_out, stage, n0 * 2, (int)row0);
                                bulk_commit();
                            }
                            continue;
                        }
                        __syncwarp();
                        auto at = [&](int i, int k) { return stage + i * 64 + (((k >> 3) ^ (i >> 1 & 3)) << 4) + (k & 7) * 2; };
                        if (a.out_vec) {
                            const int k = (lane & 3) * 8;
                            for (int i = lane >> 2; i < rows; i += 8) {
                                const int4 w = *reinterpret_cast<const int4*>(at(i, k));
                                __nv_bfloat16* d = o + i * a.out_stride + n0 + k;
                                if (n0 + k + 8 <= a.N) {
                                    *reinterpret_cast<int4*>(d) = w;
                                } else {
                                    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&w);
                                    for (int j = 0; j < 8; ++j)
                                        if (n0 + k + j < a.N) d[j] = e[j];
                                }
                            }
                        } else {
                            if (n0 + lane < a.N)
                                for (int i = 0; i < rows; ++i)
                                    o[i * a.out_stride + n0 + lane] = *reinterpret_cast<const __nv_bfloat16*>(at(i, lane));
                        }
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_hand_back(free_bar + c * 8);
        }
        bulk_wait_all();
        if constexpr (kSplit) {
            // rows part, part + parts, ..., a warp each: the blocks' sums in block order
            __syncwarp();
            cluster_sync();
            const GemmTile tile = sh.tile[0];
            const bool some = tr.n > 0 && tile.rows > 0 && !*abort;
            for (int r = part + parts * (warp & 3); some && r < tile.rows; r += parts * k4OutWarps) {
                const uint32_t at = smem_u32(codes) + r * kSplitRow * 4;
                const int64_t row = tile.row0 + r;
                float2 v = make_float2(0.0f, 0.0f);
                if constexpr (kSwiglu) {  // gate and up of one channel a lane: a block of 32 a row
                    for (int b = 0; b < parts; ++b) {
                        v.x += ld_cluster_f32(smem_of(at + lane * 4, b));
                        v.y += ld_cluster_f32(smem_of(at + (kHalf + lane) * 4, b));
                    }
                    const float h = silu_mul(v.x, v.y);
                    float m = fabsf(h);
#pragma unroll
                    for (int o = 16; o; o >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const uint32_t b = e8m0_of(m);
                    const float mate = __shfl_down_sync(0xffffffffu, h, 1), by = e8m0_inverse(b);
                    if (lane % 2 == 0)
                        static_cast<uint8_t*>(a.out)[row * a.out_stride + tile.n * (kHalf / 2) + lane / 2] =
                            (uint8_t)__nv_cvt_float2_to_fp4x2(make_float2(h * by, mate * by), __NV_E2M1, cudaRoundNearest);
                    if (lane == 0) a.out_scales[row * a.out_sstride + tile.n] = (uint8_t)b;
                } else {
                    for (int b = 0; b < parts; ++b) {
                        const float2 w = ld_cluster_f32x2(smem_of(at + lane * 8, b));
                        v.x += w.x;
                        v.y += w.y;
                    }
                    const int n = tile.n * kBN + lane * 2;
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + row * a.out_stride + n;
                    if (a.out_vec && n + 2 <= a.N) {
                        *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(v.x, v.y);
                    } else {
                        if (n < a.N) o[0] = __float2bfloat16_rn(v.x);
                        if (n + 1 < a.N) o[1] = __float2bfloat16_rn(v.y);
                    }
                }
            }
        }
    }
    if constexpr (kSplit) {
        __syncwarp();
        if (warp < 4 + k4ScaleWarps) cluster_sync();
        cluster_sync();  // no block ends while another reads its sums
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free<kCtas>(tmem, Shape::kCols);
    if (tid == 0 && *abort && a.status) flag(a.status, FLAG_TIMEOUT);
    __syncwarp();
    if (kCtas == 2) cluster_sync();  // neither block ends while the other still frees
}

// ---- quantisation ---------------------------------------------------------------------
// 8 channels a thread, four neighbours a block of 32: bound by memory, loads of 512 bytes a warp.
__global__ void __launch_bounds__(256) quantize_fp4_kernel(const __nv_bfloat16* x, int64_t x_stride, int64_t rows, int K, uint8_t* codes,
                                                           int64_t code_stride, uint8_t* scales, int64_t scale_stride) {
    grid_wait();
    grid_launch_next();
    const int per_row = K / 8;
    const int64_t total = rows * per_row;  // a multiple of 16: groups of four lanes are whole
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (total + 31) / 32 * 32; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row;
        const int at = (int)(i - row * per_row);
        float v[8] = {}, m = 0.0f;
        if (i < total) {
            const int4 p = ld_na_v4(x + row * x_stride + at * 8);
            const uint32_t u[4] = {(uint32_t)p.x, (uint32_t)p.y, (uint32_t)p.z, (uint32_t)p.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(u[j] << 16);
                v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_or_nan(m, fabsf(v[j]));
        m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t b = e8m0_of(m);
        if (i < total) {
            *reinterpret_cast<uint32_t*>(codes + row * code_stride + at * 4) = e2m1x8(v, e8m0_inverse(b));
            if ((at & 3) == 0) scales[row * scale_stride + at / 4] = (uint8_t)b;
        }
    }
}

// ---- host -------------------------------------------------------------------------
static ep_status check_fp4(const char* fn, const ep_fp4_rows* x, const ep_row_groups* g, const ep_fp4_weight* w, const uint32_t* status_out) {
    if (!x || !g || !w) return set_error(EP_ERR_INVALID_ARG, "%s: null descriptor", fn);
    if (w->groups < 1 || w->groups > kMaxGroups)
        return set_error(EP_ERR_INVALID_ARG, "%s: groups %d outside 1..%d", fn, w->groups, kMaxGroups);
    if (w->n < 1 || w->n > 0x7fffffff - 512 || w->k < 128 || w->k % 128)
        return set_error(EP_ERR_INVALID_ARG, "%s: weight rows %d, channels %d (a multiple of 128)", fn, w->n, w->k);
    if (!w->codes || !w->scales || !aligned16(w->codes) || !aligned_to(w->scales, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: weight codes (16-byte aligned) and scales (4-byte aligned) are required", fn);
    if (x->rows < 0 || x->rows > 0x7fffffff - 2 * k4BM) return set_error(EP_ERR_INVALID_ARG, "%s: %lld rows", fn, (long long)x->rows);
    if (x->rows > 0) {
        if (!x->codes || !x->scales || !aligned16(x->codes) || !aligned_to(x->scales, 4))
            return set_error(EP_ERR_INVALID_ARG, "%s: row codes (16-byte aligned) and scales (4-byte aligned) are required", fn);
        if (x->code_stride < w->k / 2 || x->code_stride % 16 || x->scale_stride < w->k / 32 || x->scale_stride % 4)
            return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld, %lld for %d channels", fn, (long long)x->code_stride,
                             (long long)x->scale_stride, w->k);
    }
    if (!aligned_to(g->counts, 4) || !aligned_to(g->offsets, 4) || !aligned_to(g->bases, 4) || !aligned_to(status_out, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: a pointer is not aligned to its elements", fn);
    if (g->bases && g->per_base < 1) return set_error(EP_ERR_INVALID_ARG, "%s: groups per base %d", fn, g->per_base);
    if (g->stride < 0 || g->expected < 0)
        return set_error(EP_ERR_INVALID_ARG, "%s: group stride %lld, expected rows %lld", fn, (long long)g->stride, (long long)g->expected);
    return EP_OK;
}

template <bool kSwiglu, int kBN, int kCtas, bool kSplit>
static ep_status launch_fp4_shape(const char* fn, const ep_fp4_rows* x, const ep_fp4_weight* w, Fp4Args a, int sms, int cluster, int dev, void* stream) {
    using Shape = Fp4Shape<kSwiglu, kBN, kCtas>;
    constexpr int kTileN = kSwiglu ? kBN / 2 : kBN;
    a.n_tiles = ((kSwiglu ? w->n / 2 : w->n) + kTileN - 1) / kTileN;
    const int64_t most = most_tiles(a, Shape::kTileM);
    if (most > kMaxTiles) return set_error(EP_ERR_INVALID_ARG, "%s: %lld tiles", fn, (long long)most);
    a.most = (int)most;
    CUtensorMap map_x, map_box, map_w, map_out;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)w->k / 2, (cuuint64_t)x->rows};
        const cuuint64_t strides[1] = {(cuuint64_t)x->code_stride};
        const cuuint32_t box[2] = {128, k4BM}, part[2] = {128, k4BoxRows};
        EP_TRY(encode_rows(&map_x, x->codes, 2, dims, strides, box, fn));
        EP_TRY(encode_rows(&map_box, x->codes, 2, dims, strides, part, fn));
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)w->k / 2, (cuuint64_t)w->n, (cuuint64_t)w->groups};
        const cuuint64_t strides[2] = {(cuuint64_t)w->k / 2, (cuuint64_t)w->k / 2 * (cuuint64_t)w->n};
        const cuuint32_t box[3] = {128, kSwiglu || kCtas == 2 ? kBN / 2 : kBN, 1};
        EP_TRY(encode_rows(&map_w, w->codes, 3, dims, strides, box, fn));
    }
    map_out = map_x;  // used for aligned bf16 rows only
    if (!kSwiglu && a.out_vec) {
        const cuuint64_t dims[2] = {(cuuint64_t)w->n * 2, (cuuint64_t)x->rows};
        const cuuint64_t strides[1] = {(cuuint64_t)a.out_stride * 2};
        const cuuint32_t box[2] = {64, 32};
        EP_TRY(encode_rows(&map_out, a.out, 2, dims, strides, box, fn, CU_TENSOR_MAP_SWIZZLE_64B));
    }
    static std::atomic<bool> known[kMaxDevicesTracked];  // devices whose launch attribute is set
    if (dev >= kMaxDevicesTracked || !known[dev].load(std::memory_order_relaxed)) {
        EP_CUDA(cudaFuncSetAttribute(fp4_gemm_kernel<kSwiglu, kBN, kCtas, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem));
        if (dev < kMaxDevicesTracked) known[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t units = most < sms / cluster ? most : sms / cluster;
    return launch_next(fp4_gemm_kernel<kSwiglu, kBN, kCtas, kSplit>, units * cluster, k4Threads, stream, Shared{Shape::kSmem, cluster}, map_x, map_box, map_w, map_out, a);
}

// Blocks that share a tile's K where the tiles are few: each four stages or more, and no more blocks than SMs (clusters of
// 8 leave some SMs of a group of SMs without one).
static int fp4_split(int64_t tiles, int stages, int sms) {
    struct Rule { int split, percent; };  // share of the SMs
    for (const Rule r : {Rule{8, 66}, {4, 100}, {2, 100}})
        if (stages >= r.split * 2 * k4Group && tiles * r.split * 100 <= (int64_t)sms * r.percent) return r.split;
    return 1;
}

// The shape of a launch's tiles: the one with the least rounds over the SMs * cost of a round, the widest of equal ones.  A
// round's cost is what bounds it, the rows of codes that a stage brings into an SM, 128 + columns.  us by 192 columns / by what
// is chosen: second product, K 2048, N 7168, 40 groups of 2048 rows 541 / 500 (224: 6 % fewer bytes a column, and N is 32 of
// them); one group, K 7168, 1000 rows: N 4096 26.4 / 18.0 (224), N 7168 27.8 / 23.2 (by 224 30.0; pairs), N 2048 15.5 / 13.6 (128);
// K 4096, N 4096, 777 rows 16.4 / 12.6 (128); first product, 300 rows, 2I 4096, by 64 20.7, by 128 13.8.
// Pairs of blocks have twice the rows, at 0.825 of a round's cost by one block.  40 groups, us by one block / by pairs: K 7168,
// 2I 4096, 256 rows a group 137 / 129, 448 242 / 206, 640 297 / 284, 768 371 / 296, 1024 460 / 390, 2048 900 / 739; K 2048, N
// 7168, 448 134 / 116, 640 165 / 160, 1024 258 / 214, 2048 500 / 411.  Half a tile of each group is empty on average where their
// lengths vary: second product, 64 groups of 512 rows on average 236 / 214, of 1024 423 / 375, of 1536 615 / 532 (K 512, N
// 4096, 512 rows 85 / 87); first product, 64 of 512 423 / 380, but 256 of 256 1020 / 1075, so that they need more than 384.
// And a launch of one round gains nothing: 777 rows, 4096 -> 4096 12.6 / 13.3.
struct Fp4Choice {
    int columns, ctas;
};
static Fp4Choice fp4_choice(bool swiglu, int64_t rows, int groups, int64_t n, int sms) {
    auto rounds = [&](int columns, int ctas) {
        const int64_t tiles = std::max<int64_t>((rows + ctas * k4BM - 1) / (ctas * k4BM), 1) * groups * ((n + columns - 1) / columns), units = sms / ctas;
        return (tiles + units - 1) / units;
    };
    Fp4Choice best = {64, 1};
    int64_t least = rounds(64, 1) * (k4BM + 64);
    auto consider = [&](int columns, int ctas, int cost) {
        const int64_t c = rounds(columns, ctas) * cost;
        if (c <= least) {
            least = c;
            best = {columns, ctas};
        }
    };
    consider(128, 1, k4BM + 128);
    consider(192, 1, k4BM + 192);
    if (!swiglu) consider(224, 1, k4BM + 224);
    if (rows > 3 * k4BM && least > k4BM + 224) consider(swiglu ? 192 : 224, 2, swiglu ? 264 : 290);
    return best;
}

template <bool kSwiglu>
static ep_status launch_fp4(const char* fn, const ep_fp4_rows* x, const ep_row_groups* g, const ep_fp4_weight* w, Fp4Args a, void* stream) {
    a.x_scales = x->scales;
    a.x_sstride = x->scale_stride;
    auto vec = [](const void* p, int64_t stride) { return aligned_to(p, 32) && stride % 32 == 0 ? 32 : aligned16(p) && stride % 16 == 0 ? 16 : 4; };
    a.x_vec = vec(x->scales, x->scale_stride);
    a.w_scales = w->scales;
    a.w_vec = vec(w->scales, w->k / 32);
    a.G = w->groups;
    a.N = w->n;
    a.K = w->k;
    a.KT = (w->k + k4BK - 1) / k4BK;
    a.counts = g->counts;
    a.offsets = g->offsets;
    a.bases = g->bases;
    a.per_base = g->per_base;
    a.group_stride = g->stride;
    a.rows = x->rows;
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    a.n_tiles = (w->n + 63) / 64;
    const int split = fp4_split(most_tiles(a, k4BM), a.KT, sms);
    if (split > 1) return launch_fp4_shape<kSwiglu, 64, 1, true>(fn, x, w, a, sms, split, dev, stream);
    // Rows of a group: as the caller expects, or what the arrays hold, shared out; regions with counts are sized for the
    // worst case, and a low-latency step fills a few percent of them.
    const int64_t rows = g->expected > 0 ? std::min<int64_t>(g->expected, 0x7fffffff) : x->rows / w->groups / (w->groups > 1 && !g->offsets && g->counts ? 16 : 1);
    const Fp4Choice c = fp4_choice(kSwiglu, rows, w->groups, w->n, sms);
    if (c.columns == 64) return launch_fp4_shape<kSwiglu, 64, 1, false>(fn, x, w, a, sms, 1, dev, stream);
    if (c.columns == 128) return launch_fp4_shape<kSwiglu, 128, 1, false>(fn, x, w, a, sms, 1, dev, stream);
    if constexpr (kSwiglu) {
        if (c.ctas == 2) return launch_fp4_shape<kSwiglu, 192, 2, false>(fn, x, w, a, sms, 2, dev, stream);
    } else {
        if (c.ctas == 2) return launch_fp4_shape<kSwiglu, 224, 2, false>(fn, x, w, a, sms, 2, dev, stream);
        if (c.columns == 224) return launch_fp4_shape<kSwiglu, 224, 1, false>(fn, x, w, a, sms, 1, dev, stream);
    }
    return launch_fp4_shape<kSwiglu, 192, 1, false>(fn, x, w, a, sms, 1, dev, stream);
}

}  // namespace ep

using namespace ep;

extern "C" int64_t ep_fp4_row_bytes(int hidden) { return hidden > 0 ? fp4_row_bytes(hidden) : 0; }

extern "C" ep_status ep_quantize_fp4(const void* x, int64_t x_stride, int64_t rows, int32_t channels, uint8_t* codes, int64_t code_stride,
                                     uint8_t* scales, int64_t scale_stride, void* stream) {
    const char* fn = "ep_quantize_fp4";
    if (rows < 0 || rows > 0x7fffffff || channels < 128 || channels % 128)
        return set_error(EP_ERR_INVALID_ARG, "%s: %lld rows of %d channels (a multiple of 128)", fn, (long long)rows, channels);
    if (rows == 0) return EP_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned_to(scales, 4))
        return set_error(EP_ERR_INVALID_ARG, "%s: x and codes (16-byte aligned) and scales (4-byte aligned) are required", fn);
    if (x_stride % 8 || code_stride % 16 || scale_stride % 4 ||
        (rows > 1 && (x_stride < channels || code_stride < channels / 2 || scale_stride < channels / 32)))
        return set_error(EP_ERR_INVALID_ARG, "%s: row strides %lld, %lld, %lld for %d channels", fn, (long long)x_stride, (long long)code_stride,
                         (long long)scale_stride, channels);
    int dev = 0, sms = 0;
    EP_CUDA(cudaGetDevice(&dev));
    EP_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const int64_t need = (rows * (channels / 8) + 255) / 256, most = (int64_t)sms * 8;
    return launch_next(quantize_fp4_kernel, need < most ? need : most, 256, stream, static_cast<const __nv_bfloat16*>(x), x_stride, rows, channels,
                       codes, code_stride, scales, scale_stride);
}

extern "C" ep_status ep_dispatch_permuted_fp4(ep_ctx* c, const uint8_t* xq, const int64_t* topk_idx, const float* topk_weights,
                                              const ep_dispatch_handle* h, uint8_t* permuted_xq, int32_t* perm_src_token, float* perm_weight,
                                              int64_t perm_capacity_rows, void* stream) {
    if (!c) return set_error(EP_ERR_INVALID_ARG, "ctx is NULL");
    if (c->cfg.hidden % 128) return set_error(EP_ERR_INVALID_ARG, "FP4 rows need hidden %% 128 == 0");
    return dispatch_permuted_rows(c, xq, fp4_row_bytes(c->cfg.hidden), topk_idx, topk_weights, h, permuted_xq, perm_src_token, perm_weight,
                                  perm_capacity_rows, stream);
}

extern "C" ep_status ep_expert_gemm_fp4(const ep_fp4_rows* x, const ep_row_groups* groups, const ep_fp4_weight* w, void* out, int64_t out_stride,
                                        uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_gemm_fp4";
    EP_TRY(check_fp4(fn, x, groups, w, status_out));
    if (x->rows == 0) return EP_OK;
    if (!out || out_stride < w->n || !aligned_to(out, 2))
        return set_error(EP_ERR_INVALID_ARG, "%s: output (2-byte aligned), stride %lld for %d channels", fn, (long long)out_stride, w->n);
    Fp4Args a{};
    a.out = out;
    a.out_stride = out_stride;
    a.out_vec = aligned16(out) && out_stride % 8 == 0;
    a.out_clip = w->n % 8 == 0;
    a.status = status_out;
    return launch_fp4<false>(fn, x, groups, w, a, stream);
}

extern "C" ep_status ep_expert_swiglu_fp4(const ep_fp4_rows* x, const ep_row_groups* groups, const ep_fp4_weight* w13, uint8_t* out,
                                          int64_t out_stride, uint8_t* out_scales, int64_t out_scale_stride, uint32_t* status_out, void* stream) {
    const char* fn = "ep_expert_swiglu_fp4";
    EP_TRY(check_fp4(fn, x, groups, w13, status_out));
    if (w13->n % 256) return set_error(EP_ERR_INVALID_ARG, "%s: %d weight rows (gate and up, each a multiple of 128)", fn, w13->n);
    if (x->rows == 0) return EP_OK;
    const int inter = w13->n / 2;
    if (!out || !out_scales || !aligned16(out) || !aligned_to(out_scales, 4) || out_stride < inter / 2 || out_stride % 16 ||
        out_scale_stride < inter / 32 || out_scale_stride % 4)
        return set_error(EP_ERR_INVALID_ARG, "%s: output rows (16-byte aligned, strides %lld, %lld) for %d channels", fn, (long long)out_stride,
                         (long long)out_scale_stride, inter);
    Fp4Args a{};
    a.out = out;
    a.out_stride = out_stride;
    a.out_scales = out_scales;
    a.out_sstride = out_scale_stride;
    a.status = status_out;
    return launch_fp4<true>(fn, x, groups, w13, a, stream);
}
