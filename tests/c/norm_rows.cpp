// Runs the row loop of norm_backward_block on the host, a thread a GPU thread, one block after the other: what its blocks
// write when a copy does not come, which no GPU is made to show.  argv: hidden, rows, blocks, stages, the row whose copy of
// dy is lost (-1: none).  Prints a line a row, "ok" (dx is right), "nan" (all NaN) or "stale", and one for dweight.
#include <atomic>
#include <barrier>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <thread>
#include <type_traits>
#include <vector>

#include <cuda_bf16.h>
#include <vector_types.h>

// ---- the device's side of the source below ----
namespace host {
thread_local dim3 thread, block;
dim3 block_size, grid_size;
std::unique_ptr<std::barrier<>> all;
struct Warp {
    std::barrier<> in{32};
    float v[32];
};
std::vector<std::unique_ptr<Warp>> warps;
const void* lost = nullptr;
uint32_t pending[8];
}  // namespace host
#define threadIdx host::thread
#define blockIdx host::block
#define blockDim host::block_size
#define gridDim host::grid_size
#undef __global__
#undef __device__
#undef __shared__
#undef __launch_bounds__
#undef __forceinline__
#undef __align__
#define __global__ static
#define __device__
#define __shared__ static
#define __launch_bounds__(...)
#define __forceinline__ inline
#define __align__(n)
static void __syncthreads() { host::all->arrive_and_wait(); }
static float __shfl_xor_sync(unsigned, float v, int o) {
    host::Warp& w = *host::warps[host::thread.x >> 5];
    const int lane = host::thread.x & 31;
    w.v[lane] = v;
    w.in.arrive_and_wait();
    const float r = w.v[lane ^ o];
    w.in.arrive_and_wait();
    return r;
}
static float __uint_as_float(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static float __int_as_float(int u) { return __uint_as_float((uint32_t)u); }
static float rsqrtf(float x) { return 1.0f / std::sqrt(x); }
static float __fdiv_rn(float a, float b) { return a / b; }

namespace ep {
alignas(128) uint8_t ring[256 * 1024];
static int4 ld_na_v4(const void* p) { int4 v; memcpy(&v, p, 16); return v; }
static void st_na_v4(void* p, int4 v) { memcpy(p, &v, 16); }
static void ld_global_32(const void* p, uint32_t* v) { memcpy(v, p, 32); }
static void st_global_32(void* p, const uint32_t* v) { memcpy(p, v, 32); }
static float max_or_nan(float a, float b) { return a != a || b != b ? NAN : a > b ? a : b; }
static int4 quantize16_by(const float*, float) { return {}; }
static void grid_wait() {}
static void grid_launch_next() {}
static void fence_mbar_init() {}
// A barrier counts the phases that have ended; one thread issues all copies.
static void mbar_init(uint64_t* b, int) { *b = 0; }
static void mbar_arrive_expect_tx(uint64_t* b, uint32_t bytes) { host::pending[(uintptr_t)b / 8 % 8] = bytes; }
static void bulk_g2s(void* d, const void* s, uint32_t bytes, uint64_t* b) {
    if (s == host::lost) return;
    memcpy(d, s, bytes);
    if ((host::pending[(uintptr_t)b / 8 % 8] -= bytes) == 0) std::atomic_ref<uint64_t>(*b).fetch_add(1);
}
static bool mbar_wait_bounded(uint64_t* b, uint32_t parity, int64_t) {
    const auto end = std::chrono::steady_clock::now() + std::chrono::milliseconds(host::lost ? 300 : 60000);
    while ((std::atomic_ref<uint64_t>(*b).load() & 1) == parity) {
        if (std::chrono::steady_clock::now() > end) return false;
        std::this_thread::yield();
    }
    return true;
}
}  // namespace ep

#include NORM_SOURCE

using T = float;

int main(int argc, char** argv) {
    if (argc != 6) return 2;
    const int H = atoi(argv[1]), rows = atoi(argv[2]), blocks = atoi(argv[3]), stages = atoi(argv[4]), lost = atoi(argv[5]);
    const int threads = ((H / 8 + 1) / 2 + 31) / 32 * 32;
    if (H % 8 || stages < 1 || stages > 4 || stages * H * 10 > (int)sizeof(ep::ring) || threads > 1024) return 2;
    std::vector<__nv_bfloat16> dy((size_t)rows * H);
    std::vector<float> h((size_t)rows * H), d((size_t)rows * H), w(H), dx((size_t)rows * H, 12345.0f), part((size_t)blocks * H);
    uint32_t seed = 1;
    auto next = [&] { return (float)((seed = seed * 1664525u + 1013904223u) >> 8) / (1 << 24) - 0.5f; };
    for (size_t i = 0; i < h.size(); ++i) dy[i] = __float2bfloat16(next()), h[i] = next(), d[i] = next();
    for (float& v : w) v = 1.0f + next();
    const float eps = 1e-5f;
    const ep::NormBackArgs a = {dy.data(), h.data(), d.data(), w.data(), dx.data(), part.data(), H, H, H, H, rows, H, eps, true};
    if (lost >= 0) host::lost = &dy[(size_t)lost * H];
    host::block_size = dim3(threads);
    host::grid_size = dim3(blocks);
    for (int i = 0; i < threads / 32; ++i) host::warps.push_back(std::make_unique<host::Warp>());
    for (int b = 0; b < blocks; ++b) {
        host::all = std::make_unique<std::barrier<>>(threads);
        std::vector<std::thread> team;
        for (int t = 0; t < threads; ++t)
            team.emplace_back([&, t] {
                host::thread = dim3(t);
                host::block = dim3(b);
                ep::norm_backward_block<2>(a, stages);
                host::all->arrive_and_drop();
            });
        for (std::thread& t : team) t.join();
    }
    for (int r = 0; r < rows; ++r) {
        const float* hr = &h[(size_t)r * H];
        double ss = 0, gh = 0;
        for (int c = 0; c < H; ++c) {
            ss += (double)hr[c] * hr[c];
            gh += (double)__bfloat162float(dy[(size_t)r * H + c]) * w[c] * hr[c];
        }
        const double s = 1 / std::sqrt(ss / H + eps);
        int right = 0, nan = 0;
        for (int c = 0; c < H; ++c) {
            const double g = (double)__bfloat162float(dy[(size_t)r * H + c]) * w[c];
            const float v = dx[(size_t)r * H + c];
            right += std::fabs(v - (d[(size_t)r * H + c] + s * (g - hr[c] * s * s * (gh / H)))) < 1e-4;
            nan += v != v;
        }
        puts(right == H ? "ok" : nan == H ? "nan" : "stale");
    }
    bool bad = false;
    for (float v : part) bad |= v != v;
    puts(bad ? "dweight nan" : "dweight ok");
}
