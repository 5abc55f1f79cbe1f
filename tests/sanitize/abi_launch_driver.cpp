// The grids that the calls of include/bitlinear.h launch for the rotation, the cache and attention over it, at the largest
// shapes that they accept (built and run by tests/test_launches_host.py): this program has hipLaunchKernel itself, which
// writes the grid down and launches nothing. A grid has fewer than 2^32 threads in x, at most 2^16 - 1 workgroups
// in y and in z, and the launches of a kernel have as many workgroups together as there is work.
#include <cstdint>
#include <cstdio>
#include <vector>

#include <hip/hip_runtime_api.h>

#include "../../include/bitlinear.h"

struct Launch {
    dim3 grid, block;
};
static std::vector<Launch> launches;
// what a launch goes through on the host: the configuration is put down, and taken up again by the kernel's stub
static Launch next;
extern "C" hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t)
{
    next = {grid, block};
    return hipSuccess;
}
extern "C" hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream)
{
    *grid = next.grid;
    *block = next.block;
    *lds = 0;
    *stream = nullptr;
    return hipSuccess;
}
extern "C" hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **, size_t, hipStream_t)
{
    launches.push_back({grid, block});
    return hipSuccess;
}
extern "C" hipError_t hipGetLastError() { return hipSuccess; }

static int failures = 0;
static void check(const char *what, bl_status st, int64_t a, int64_t b, int64_t c, int64_t d)
{
    bool ok = st == BL_OK && !launches.empty();
    for (const Launch &l : launches)
        ok = ok && l.grid.x && l.grid.y && l.grid.z && (uint64_t)l.grid.x * l.block.x < (uint64_t)1 << 32 && l.grid.y < 1u << 16 &&
             l.grid.z < 1u << 16 && l.block.x * l.block.y * l.block.z <= 1024;
    if (!ok) {
        ++failures;
        std::fprintf(stderr, "%s m %lld heads %lld/%lld of %lld: status %d\n", what, (long long)a, (long long)b, (long long)c, (long long)d, (int)st);
        for (const Launch &l : launches)
            if ((uint64_t)l.grid.x * l.block.x >= (uint64_t)1 << 32 || l.grid.y >= 1u << 16 || l.grid.z >= 1u << 16)
                std::fprintf(stderr, "    %u x %u x %u of %u\n", l.grid.x, l.grid.y, l.grid.z, l.block.x);
    }
}
// threads in x of all launches whose workgroups have `block` of them
static int64_t threads(unsigned block)
{
    int64_t n = 0;
    for (const Launch &l : launches)
        if (l.block.x == block) n += (int64_t)l.grid.x * block;
    return n;
}

int main()
{
    void *A = reinterpret_cast<void *>(0x10000);
    const int32_t *I = static_cast<const int32_t *>(A);
    const int8_t *C = static_cast<const int8_t *>(A);
    const float *F = static_cast<const float *>(A);
    const size_t room = (size_t)1 << 62;
    const int64_t kTok = BL_MAX_TOKENS, kHeads = BL_MAX_HEADS, kBig = BL_MAX_DIM;
    struct Shape {
        int64_t m, hq, hkv;
    };
    const Shape shapes[] = {{1, 1, 1}, {1 << 20, 32, 8}, {1 << 21, 64, 32}, {kTok, 32, 8}, {kTok, 128, 64}, {kTok, kHeads, kHeads},
                            {kTok / 8, kHeads, 1}, {70, kHeads, 1}, {1 << 18, 256, 2}};
    for (const Shape &s : shapes)
        for (int64_t d : {(int64_t)64, (int64_t)128})
            for (bl_dtype t : {BL_F32, BL_BF16})
                for (int64_t seqs : {s.m, (int64_t)1, (int64_t)300})
                    for (int64_t wide : {(int64_t)1, (int64_t)300, kBig}) {
                        const int64_t stride = s.hq * d;
                        const int32_t *cu = seqs == s.m ? nullptr : I;
                        const int64_t rows = s.m * s.hq;
                        if (s.m * (s.hq / s.hkv) > INT32_MAX - 1024) continue;
                        auto run = [&](const char *what, auto call) {
                            launches.clear();
                            const bl_status st = call();
                            check(what, st, s.m, s.hq, s.hkv, d);
                        };
                        run("rotate", [&] { return bitlinear_rotate(A, stride, A, s.hkv * d, t, s.m, s.hq, s.hkv, d, cu, I, seqs, F, 32, 0, 1.0f, F, F, 1e-5f, A, stride, A, s.hkv * d, nullptr); });
                        run("cache_append", [&] { return bitlinear_cache_append(A, s.hkv * d, A, s.hkv * d, t, s.m, s.hkv, d, cu, I, seqs, I, wide, (int8_t *)A, (int8_t *)A, (float *)A, (float *)A, 99, nullptr); });
                        run("cache_bounds", [&] { return bitlinear_cache_bounds(C, 99, s.hkv, d, s.m, cu, I, seqs, I, wide, (int8_t *)A, nullptr); });
                        run("attention_cached", [&] { return bitlinear_attention_cached(A, stride, t, s.m, s.hq, s.hkv, d, cu, I, seqs, I, wide, C, C, F, F, 99, 0.1f, A, nullptr, A, room, nullptr); });
                        run("attention_cached with weights", [&] { return bitlinear_attention_cached(A, stride, t, s.m, s.hq, s.hkv, d, cu, I, seqs, I, wide, C, C, F, F, 99, 0.1f, A, (float *)A, A, room, nullptr); });
                        run("attention_selected", [&] { return bitlinear_attention_selected(A, stride, t, s.m, s.hq, s.hkv, d, cu, I, seqs, I, 300, I, wide, C, C, F, F, 99, 0.1f, A, A, room, nullptr); });
                        for (int64_t prefix : {(int64_t)1, kBig}) {
                            run("attention_shared", [&] { return bitlinear_attention_shared(A, stride, t, s.m, s.hq, s.hkv, d, I, prefix, I, cu, I, seqs, I, wide, C, C, F, F, 99, 0.1f, A, A, room, nullptr); });
                            // the joining workgroups: a thread per element, or a workgroup per row
                            if (threads(512) < rows * d) {
                                ++failures;
                                std::fprintf(stderr, "attention_shared m %lld heads %lld: rows are not joined\n", (long long)s.m, (long long)s.hq);
                            }
                        }
                        if (s.hq / s.hkv <= 128)
                            run("block_select", [&] { return bitlinear_block_select(A, stride, t, s.m, s.hq, s.hkv, d, cu, I, seqs, I, wide, C, F, 99, 40, 1, 2, (int32_t *)A, A, room, nullptr); });
                    }
    if (failures) {
        std::fprintf(stderr, "%d launches are wrong\n", failures);
        return 1;
    }
    std::printf("abi launch driver: ok\n");
    return 0;
}
