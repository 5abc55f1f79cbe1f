// Drives the host side of the rotation, the shared prefix and the chosen blocks
// (include/bitlinear.h) under AddressSanitizer and UndefinedBehaviorSanitizer, host
// code only (built and run by tests/test_sanitizers_serving.py): the argument checks,
// the size queries at the largest shapes, and, where there is no GPU, the launch
// arithmetic too -- calls that are valid but for their fake addresses then end in BL_ERR_HIP.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include <hip/hip_runtime_api.h>

#include "../../include/bitlinear.h"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); ++failures; } } while (0)

static void *A = reinterpret_cast<void *>(0x10000);
static const int64_t kBig = BL_MAX_DIM, kTok = BL_MAX_TOKENS, kHeads = BL_MAX_HEADS;
static const size_t kRoom = std::numeric_limits<size_t>::max() / 2;
static const int32_t *I = static_cast<const int32_t *>(A);
static const int8_t *C = static_cast<const int8_t *>(A);
static const float *F = static_cast<const float *>(A);

static bl_status rotate(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t rot, int interleaved = 0,
                        float eps = 1e-5f)
{
    return bitlinear_rotate(A, hq * d, A, hkv * d, t, m, hq, hkv, d, packed ? I : nullptr, I, seqs, F, rot, interleaved, 1.0f, F, nullptr, eps, A,
                            hq * d, A, hkv * d, nullptr);
}
static bl_status shared(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t prefix,
                        void *ws = A, size_t room = kRoom)
{
    return bitlinear_attention_shared(A, hq * d, t, m, hq, hkv, d, I, prefix, I, packed ? I : nullptr, I, seqs, I, wide, C, C, F, F, 99, 0.1f, A,
                                      ws, room, nullptr);
}
static bl_status bounds(int64_t m, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t pages)
{
    return bitlinear_cache_bounds(C, pages, hkv, d, m, packed ? I : nullptr, I, seqs, I, wide, (int8_t *)A, nullptr);
}
static bl_status choose(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t keep,
                        int64_t first, int64_t recent, void *ws = A, size_t room = kRoom)
{
    return bitlinear_block_select(A, hq * d, t, m, hq, hkv, d, packed ? I : nullptr, I, seqs, I, wide, C, F, 99, keep, first, recent,
                                  (int32_t *)A, ws, room, nullptr);
}
static bl_status selected(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t keep,
                          void *ws = A, size_t room = kRoom)
{
    return bitlinear_attention_selected(A, hq * d, t, m, hq, hkv, d, packed ? I : nullptr, I, seqs, I, wide, I, keep, C, C, F, F, 99, 0.1f, A, ws,
                                        room, nullptr);
}

int main()
{
    const int64_t most = std::numeric_limits<int64_t>::max(), least = std::numeric_limits<int64_t>::min();
    // size queries: the widest accepted, and everything beyond
    for (int64_t m : {(int64_t)1, (int64_t)70, kTok, kTok + 1, (int64_t)0, least, most})
        for (int64_t hq : {(int64_t)1, (int64_t)20, kHeads, kHeads + 1, (int64_t)-3, most})
            for (int64_t hkv : {(int64_t)1, (int64_t)5, kHeads, (int64_t)0, least, most})
                for (int64_t wide : {(int64_t)1, (int64_t)63, kBig, kBig + 1, least, most}) {
                    (void)bitlinear_block_select_workspace_size(m, hkv, wide);
                    for (int64_t d : {(int64_t)64, (int64_t)128, (int64_t)96, least}) {
                        (void)bitlinear_attention_selected_workspace_size(m, hq, hkv, d, wide);
                        for (int64_t seqs : {(int64_t)1, (int64_t)300, kTok, (int64_t)0, most})
                            for (int64_t prefix : {(int64_t)1, kBig, least})
                                (void)bitlinear_attention_shared_workspace_size(m, hq, hkv, d, seqs, wide, prefix);
                    }
                }
    CHECK(bitlinear_attention_shared_workspace_size(1, 32, 8, 128, 1, 1, 1) > 0);
    CHECK(bitlinear_attention_shared_workspace_size(kTok, kHeads, 1, 128, kTok, 1, 1) == 0);  // rows past 31 bits
    CHECK(bitlinear_block_select_workspace_size(kTok, kHeads, kBig) == (size_t)4 << 54);
    CHECK(bitlinear_attention_selected_workspace_size(1, 32, 8, 128, 64) > 0);

    // refusals
    CHECK(rotate(BL_F32, 4, 8, 2, 128, true, 1, 100) == BL_ERR_SHAPE && rotate(BL_F32, 4, 8, 2, 64, true, 1, 128) == BL_ERR_SHAPE);
    CHECK(rotate(BL_F32, 4, 8, 2, 128, false, 3, 64) == BL_ERR_SHAPE && rotate(BL_F32, 4, 8, 2, 128, true, 1, least) == BL_ERR_SHAPE);
    CHECK(rotate(BL_F32, 4, 8, 2, 128, true, 1, 64, 7) == BL_ERR_VALUE && rotate(BL_F32, 4, 8, 2, 128, true, 1, 64, 0, std::nanf("")) == BL_ERR_VALUE);
    CHECK(rotate((bl_dtype)4, 4, 8, 2, 128, true, 1, 64) == BL_ERR_DTYPE);
    CHECK(shared(BL_F32, 4, 8, 2, 64, false, 3, 4, 9) == BL_ERR_SHAPE && shared(BL_F32, 4, 8, 2, 64, true, 3, 4, most) == BL_ERR_SHAPE);
    CHECK(shared(BL_F32, 4, 8, 2, 64, true, 3, 4, 9, A, 8) == BL_ERR_WORKSPACE && shared(BL_F32, 4, 8, 2, 64, true, 3, 4, 9, nullptr, 0) == BL_ERR_NULL);
    CHECK(bounds(4, 2, 64, false, 3, 4, 9) == BL_ERR_SHAPE && bounds(4, 2, 64, true, 3, 4, most) == BL_ERR_SHAPE);
    CHECK(choose(BL_F32, 4, 258, 2, 64, true, 3, 4, 4, 0, 1) == BL_ERR_SHAPE && choose(BL_F32, 4, 8, 2, 64, true, 3, 4, most, 0, 1) == BL_ERR_VALUE);
    CHECK(choose(BL_F32, 4, 8, 2, 64, true, 3, 4, 4, least, 1) == BL_ERR_VALUE && choose(BL_F32, 4, 8, 2, 64, true, 3, 4, 4, 0, most) == BL_ERR_VALUE);
    CHECK(choose(BL_F32, 1, 8, 2, 64, true, 1, kBig, 4, 0, 1, nullptr, 0) == BL_ERR_NULL);
    CHECK(selected(BL_F32, 4, 8, 2, 64, true, 3, 4, 0) == BL_ERR_SHAPE && selected(BL_F32, 4, 8, 2, 64, true, 3, 4, most) == BL_ERR_SHAPE);
    CHECK(selected(BL_F32, 1, 8, 2, 128, true, 1, 2048, 300, A, 8) == BL_ERR_WORKSPACE);

    // launches: every type, width and rule, small and at the widest sizes that a launch is made for
    int devices = 0;
    if (hipGetDeviceCount(&devices) != hipSuccess) devices = 0;
    if (devices == 0) {
        for (bl_dtype t : {BL_F32, BL_BF16})
            for (int64_t d : {(int64_t)64, (int64_t)128})
                for (bool packed : {false, true}) {
                    for (int inter : {0, 1})
                        CHECK(rotate(t, 1, 20, 5, d, packed, 1, 16, inter) == BL_ERR_HIP && rotate(t, kTok, 128, 64, d, packed, kTok, d, inter) == BL_ERR_HIP);
                    CHECK(bounds(33, 5, d, packed, 33, 40, 2000) == BL_ERR_HIP && bounds(kTok, kHeads, d, packed, kTok, kBig, INT32_MAX) == BL_ERR_HIP);
                    for (int64_t wide : {(int64_t)1, (int64_t)300, (int64_t)5000, kBig}) {
                        CHECK(shared(t, 1, 20, 5, d, packed, 1, wide, 1) == BL_ERR_HIP && shared(t, 1, 20, 5, d, packed, 1, 1, wide) == BL_ERR_HIP);
                        CHECK(shared(t, 600, 8, 8, d, packed, 600, wide, wide) == BL_ERR_HIP && shared(t, 40, 32, 2, d, packed, 40, wide, 40) == BL_ERR_HIP);
                        CHECK(shared(t, 1 << 16, 64, 4, d, packed, 1 << 16, wide, wide) == BL_ERR_HIP);
                        CHECK(choose(t, 1, 20, 5, d, packed, 1, wide, 4, 1, 1) == BL_ERR_HIP && choose(t, 600, 8, 8, d, packed, 600, wide, kBig, 0, 1) == BL_ERR_HIP);
                        CHECK(choose(t, 1 << 16, 128, 1, d, packed, 1 << 16, wide, 4, 1, 1) == BL_ERR_HIP);
                        CHECK(selected(t, 1, 20, 5, d, packed, 1, wide, wide) == BL_ERR_HIP && selected(t, 600, 8, 8, d, packed, 600, wide, 7) == BL_ERR_HIP);
                        CHECK(selected(t, 1 << 16, 64, 4, d, packed, 1 << 16, wide, wide) == BL_ERR_HIP);
                    }
                }
    }
    if (failures) {
        std::fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    std::printf("abi serving driver: ok (%s)\n", devices ? "without launches" : "with launches");
    return 0;
}
