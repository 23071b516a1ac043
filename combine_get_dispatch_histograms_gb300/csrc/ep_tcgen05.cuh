// ep_tcgen05.cuh -- inline-PTX primitives of the tensor-core kernels: tensor
// memory, tcgen05.mma on 8-bit operands, tiled bulk copies, bounded barriers.
#pragma once
#include <cuda.h>

#include "ep_internal.cuh"

namespace ep {

// ---- bounded mbarrier waits, on shared addresses -----------------------------------
// kLong: a thread that has to wait is suspended for up to 20 us instead of the
// system's own limit, so that waiting warps do not take issue slots from those
// that share their scheduler.
template <bool kLong>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (kLong)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The clock is read only once in 256 failed tries (each suspends the thread for
// a while), so that a wait in a hot loop costs no timer access.  Returns false
// after `limit_ns`, or as soon as another role gave up (*abort).
template <bool kLong = false>
__device__ __forceinline__ bool mbar_wait_or_abort(uint32_t bar, uint32_t parity, int64_t limit_ns, volatile int* abort) {
    if (mbar_try<kLong>(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try<kLong>(bar, parity)) return true;
        if ((i & 255u) == 0) {
            if (*abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if ((int64_t)(t - t0) > limit_ns) {
                *abort = 1;
                return false;
            }
        }
    }
}
// The same for a whole warp, which stays together; after a give-up it returns
// as after success, and the caller looks at *abort where it can leave.
template <bool kLong = false>
__device__ __forceinline__ void mbar_wait_warp(uint32_t bar, uint32_t parity, int64_t limit_ns, volatile int* abort) {
    if (__all_sync(0xffffffffu, mbar_try<kLong>(bar, parity))) return;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try<kLong>(bar, parity))) return;
        if ((i & 255u) == 0) {
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            const bool over = (int64_t)(t - t0) > limit_ns;
            if (over) *abort = 1;
            if (__any_sync(0xffffffffu, over || *abort)) return;
        }
    }
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Programmatic launches.  grid_wait: until the kernel before has ended and its writes are visible.  It ends
// after its own wait, so that everything before it has ended too.  grid_launch_next: once every block has said
// so, the next kernel may start, if it was launched for that; whoever calls it after grid_wait promises the
// next kernel that all before this one is complete.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- the two blocks of a cluster ---------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Cluster address of the same shared variable in block `rank`.
__device__ __forceinline__ uint32_t smem_of(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// Arrives on a barrier of either block, without ordering memory: what it hands
// over is tensor memory, read through tcgen05.wait::ld, and the fences of
// tcgen05 order that.  A release here costs the warp 200 (block scope) to 1000
// cycles (cluster scope) a call, measured.
__device__ __forceinline__ void mbar_hand_back(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---- tiled bulk copies (the innermost coordinate is a multiple of 16 bytes) ------
// Into this block's shared memory; `bar` (a cluster address) counts the bytes,
// with kCtas = 2 also where it lies in the other block of the pair.
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
            "[%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(x), "r"(y)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                smem_u32(dst)),
            "l"(m), "r"(bar), "r"(x), "r"(y)
            : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
            "%5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
            "[%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
}

// From this block's shared memory, 128-byte rows in the 128-byte swizzle; part of
// the thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m), "r"(smem_u32(src)),
                 "r"(x), "r"(y)
                 : "memory");
}

// ---- tensor memory and tcgen05.mma, by one block or by pairs of blocks ---------------
// Every tcgen05 instruction of a kernel names the same number of blocks.
template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {  // a whole warp (of both blocks)
    if constexpr (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {  // the same warps
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[kCtas * 128 x N] (+)= A[kCtas * 128 x 32] B[N x 32]^T, e4m3 operands in
// shared memory.  With two blocks each holds half of A's rows, half of B's rows
// and the accumulator rows of its half of A; one thread of block 0 issues.
template <int kCtas>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
// The same for one block and bf16 operands: D[128 x N] (+)= A[128 x 16] B[N x 16]^T.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrives on `bar` (of both blocks) when every tcgen05.mma this thread issued has finished.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same on the barrier of the issuing block alone.
template <int kCtas>
__device__ __forceinline__ void mma_commit_here(uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Consecutive columns of this warp's 32 lanes: thread i gets lane i's row.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for this warp's tensor-memory loads.  `v` passes through the statement
// so that no use of the loaded values moves above the wait.
__device__ __forceinline__ void tmem_wait_ld(float (&v)[32]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
          "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
          "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
          "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
        :
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld(float (&v)[16]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
          "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
        :
        : "memory");
}

// Shared-memory descriptor of a K-major tile with 128-byte rows in the 128-byte
// swizzle (8-row atoms of 1024 bytes).
__device__ __forceinline__ uint64_t smem_desc_sw128(const void* p) {
    return (uint64_t)((smem_u32(p) & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, e4m3 x e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// The same with bf16 x bf16.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) { return idesc_e4m3(m, n) | (1u << 7) | (1u << 10); }

// silu(g) * u with the approximate power and reciprocal.  Off by at most 8 * 2^-23 of itself for g >= 0; for g < 0 by
// |g| * 2^-23 more, since rounding the power's argument g * log2(e) moves the power by up to 2^-24 |g| of itself, and so
// does log2(e)'s own.  For g below about -87 the reciprocal or the power leaves the range, and the result is a zero
// of -u's sign where it should be smaller than 88 * 2^-126 |u|.  With expf and a division right to 2 ulp as many codes
// of expert_swiglu (3.2e-6 of them) round other than a plain form's as with this, and another order of the plain form's
// sums moves 2e-6 to 2e-5; but 4096 -> 1408 takes 4658 us for 4505, 128 -> 768 119 for 94, a layer of one token 80 for 75.
__device__ __forceinline__ float silu_mul(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

// The larger of both, or NaN if either is one: a block's maximum, and with it its scale and codes, keeps a NaN.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// d[i] += v[i] * f, two at a time: half the instructions, and fewer register-bank
// conflicts (1.2 cycles a value and warp against 1.5, measured).
template <int kN>
__device__ __forceinline__ void fma_by(float* d, float (&v)[kN], float f) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
        const float2 s = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(f, f), make_float2(d[i], d[i + 1]));
        d[i] = s.x;
        d[i + 1] = s.y;
    }
}

// ---- host: tensor maps ------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
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

// A map of bytes [..][rows][row bytes] in boxes of 128 bytes x rows, 128-byte swizzle.
inline ep_status encode_rows(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                             const cuuint32_t* box, const char* what,
                             CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(EP_ERR_INVALID_ARG, "%s: the tensor map was refused (%d)", what, (int)r);
    return EP_OK;
}

}  // namespace ep
