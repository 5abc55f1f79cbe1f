// Drives the host side of the attention and cache calls (include/bitlinear.h)
// under AddressSanitizer and UndefinedBehaviorSanitizer, host code only (built and
// run by tests/test_sanitizers_attention.py): the argument checks, the size queries
// at the largest shapes, and, where there is no GPU, the launch arithmetic too --
// calls that are valid but for their fake addresses then end in BL_ERR_HIP.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include <hip/hip_runtime_api.h>

#include "../../include/bitlinear.h"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); ++failures; } } while (0)

static void *A = reinterpret_cast<void *>(0x10000), *MIS = reinterpret_cast<void *>(0x10004);
static const int64_t kBig = BL_MAX_DIM, kTok = BL_MAX_TOKENS, kHeads = BL_MAX_HEADS;
static const size_t kRoom = std::numeric_limits<size_t>::max() / 2;

static bl_status attention(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, int64_t seqs, float scale = 0.1f, void *q = A)
{
    return bitlinear_attention(q, hq * d, A, hkv * d, A, hkv * d, t, m, hq, hkv, d, (const int32_t *)A, seqs, scale, A, A, kRoom, nullptr);
}
static bl_status append(bl_dtype t, int64_t m, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t pages)
{
    return bitlinear_cache_append(A, hkv * d, A, hkv * d, t, m, hkv, d, packed ? (const int32_t *)A : nullptr, (const int32_t *)A, seqs,
                                  (const int32_t *)A, wide, (int8_t *)A, (int8_t *)A, (float *)A, (float *)A, pages, nullptr);
}
static bl_status read(bl_dtype t, int64_t m, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, int64_t pages)
{
    return bitlinear_cache_read((const int8_t *)A, (const int8_t *)A, (const float *)A, (const float *)A, pages, (const int32_t *)A, wide,
                                packed ? (const int32_t *)A : nullptr, (const int32_t *)A, seqs, t, m, hkv, d, A, A, nullptr);
}
static bl_status cached(bl_dtype t, int64_t m, int64_t hq, int64_t hkv, int64_t d, bool packed, int64_t seqs, int64_t wide, bool weights,
                        void *ws = A, size_t room = kRoom)
{
    return bitlinear_attention_cached(A, hq * d, t, m, hq, hkv, d, packed ? (const int32_t *)A : nullptr, (const int32_t *)A, seqs,
                                      (const int32_t *)A, wide, (const int8_t *)A, (const int8_t *)A, (const float *)A, (const float *)A,
                                      99, 0.1f, A, weights ? (float *)A : nullptr, ws, room, nullptr);
}
static bl_status evict(int64_t seqs, int64_t wide, int64_t keep, int64_t first, int64_t recent)
{
    return bitlinear_cache_evict((const int32_t *)A, (const int32_t *)A, (const float *)A, seqs, wide, keep, first, recent, (int32_t *)A,
                                 (int32_t *)A, (float *)A, (int32_t *)A, (int32_t *)A, nullptr);
}

int main()
{
    const int64_t most = std::numeric_limits<int64_t>::max(), least = std::numeric_limits<int64_t>::min();
    // size queries: the widest accepted, and everything beyond
    for (int64_t m : {(int64_t)1, (int64_t)70, kTok, kTok + 1, (int64_t)0, least, most})
        for (int64_t hq : {(int64_t)1, (int64_t)20, kHeads, kHeads + 1, (int64_t)-3, most})
            for (int64_t hkv : {(int64_t)1, (int64_t)5, kHeads, (int64_t)0, least, most})
                for (int64_t seqs : {(int64_t)1, (int64_t)300, kTok, (int64_t)0, most})
                    for (int64_t d : {(int64_t)64, (int64_t)128, (int64_t)96, least}) {
                        (void)bitlinear_attention_workspace_size(BL_F32, m, hq, hkv, d, seqs);
                        for (int64_t wide : {(int64_t)1, (int64_t)63, kBig, kBig + 1, least})
                            (void)bitlinear_attention_cached_workspace_size(m, hq, hkv, d, seqs, wide, 1);
                    }
    CHECK(bitlinear_attention_workspace_size(BL_F32, 100, 8, 2, 128, 3) > 0);
    CHECK(bitlinear_attention_workspace_size(BL_BF16, 100, 8, 2, 128, 3) == 0);
    CHECK(bitlinear_attention_workspace_size(BL_F32, kTok, kHeads, 1, 128, 3) == 0);  // rows past 31 bits
    CHECK(bitlinear_attention_cached_workspace_size(1, 32, 8, 128, 1, 2048, 0) > 0);

    // refusals
    CHECK(attention(BL_BF16, 4, 8, 2, 128, 1, 0.1f, nullptr) == BL_ERR_NULL);
    CHECK(attention(BL_BF16, 4, 8, 2, 128, 1, 0.1f, MIS) == BL_ERR_ALIGN);
    CHECK(attention((bl_dtype)5, 4, 8, 2, 128, 1) == BL_ERR_DTYPE);
    CHECK(attention(BL_BF16, 4, 8, 2, 128, 1, std::nanf("")) == BL_ERR_VALUE);
    CHECK(attention(BL_BF16, kTok + 1, 8, 2, 128, 1) == BL_ERR_SHAPE && attention(BL_BF16, 4, 8, 3, 128, 1) == BL_ERR_SHAPE);
    CHECK(attention(BL_F32, kTok, kHeads, 1, 128, 1) == BL_ERR_SHAPE && attention(BL_F32, 4, 8, 2, 80, 1) == BL_ERR_SHAPE);
    CHECK(append(BL_F32, 4, 2, 64, false, 3, 4, 9) == BL_ERR_SHAPE && append(BL_F32, 4, 2, 64, true, 3, 0, 9) == BL_ERR_SHAPE);
    CHECK(append(BL_F32, 4, 2, 64, true, 3, 4, (int64_t)1 << 31) == BL_ERR_SHAPE && append((bl_dtype)-1, 4, 2, 64, true, 3, 4, 9) == BL_ERR_DTYPE);
    CHECK(read(BL_F32, 4, 2, 64, false, 3, 4, 9) == BL_ERR_SHAPE && read(BL_F32, 4, kHeads + 1, 64, true, 3, 4, 9) == BL_ERR_SHAPE);
    CHECK(cached(BL_F32, 4, 8, 2, 64, false, 3, 4, false) == BL_ERR_SHAPE && cached(BL_F32, 1, 8, 2, 128, true, 1, 2048, true, A, 8) == BL_ERR_WORKSPACE);
    CHECK(cached(BL_F32, 1, 8, 2, 128, true, 1, 2048, true, nullptr, 0) == BL_ERR_NULL);
    CHECK(evict(2, 64, 1, 1, 1) == BL_ERR_VALUE && evict(2, 64, most, 1, most) == BL_ERR_VALUE && evict(2, 64, 4, least, 1) == BL_ERR_VALUE);
    CHECK(evict(0, 64, 4, 1, 1) == BL_ERR_SHAPE && evict(2, kBig + 1, 4, 1, 1) == BL_ERR_SHAPE);

    // launches: every type, width and rule, small and at the widest sizes that a launch is made for
    int devices = 0;
    if (hipGetDeviceCount(&devices) != hipSuccess) devices = 0;
    if (devices == 0) {
        for (bl_dtype t : {BL_F32, BL_BF16})
            for (int64_t d : {(int64_t)64, (int64_t)128}) {
                CHECK(attention(t, 1, 1, 1, d, 1) == BL_ERR_HIP && attention(t, 5000, 32, 8, d, 3) == BL_ERR_HIP);
                CHECK(attention(t, kTok, 256, 64, d, kTok) == BL_ERR_HIP);
                for (bool packed : {false, true}) {
                    CHECK(append(t, 33, 5, d, packed, 33, 40, 2000) == BL_ERR_HIP && append(t, kTok, kHeads, d, packed, kTok, kBig, INT32_MAX) == BL_ERR_HIP);
                    CHECK(read(t, 33, 5, d, packed, 33, 40, 2000) == BL_ERR_HIP && read(t, kTok, kHeads, d, packed, kTok, kBig, INT32_MAX) == BL_ERR_HIP);
                    for (bool weights : {false, true})
                        for (int64_t wide : {(int64_t)1, (int64_t)300, (int64_t)5000, kBig}) {
                            CHECK(cached(t, 1, 20, 5, d, packed, 1, wide, weights) == BL_ERR_HIP);
                            CHECK(cached(t, 40, 32, 2, d, packed, 40, wide, weights) == BL_ERR_HIP);
                            CHECK(cached(t, 600, 8, 8, d, packed, 600, wide, weights) == BL_ERR_HIP);
                            CHECK(cached(t, kTok, 64, 4, d, packed, kTok, wide, weights) == BL_ERR_HIP);
                        }
                }
            }
        CHECK(evict(1, 1, 1, 0, 1) == BL_ERR_HIP && evict(kTok, kBig, most, kBig, kBig) == BL_ERR_HIP);
    }
    if (failures) {
        std::fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    std::printf("abi attention driver: ok (%s)\n", devices ? "without launches" : "with launches");
    return 0;
}
