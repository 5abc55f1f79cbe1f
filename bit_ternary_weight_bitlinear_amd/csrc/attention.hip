// attention.hip -- causal attention over packed prompts.
//
//   out_i = sum_{j <= i} p_ij v_j,   p_i = softmax_j(scale * q_i . k_j)
//
// One pass over the keys with the running maximum and sum of the softmax.
#include "attention.hpp"

namespace bl {

__device__ inline float wave_sum_f32(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// One wave per row and query head, D / 64 dims per lane.
template <typename T, int D>
__global__ __launch_bounds__(64) void attention_kernel(AttentionProblem a)
{
    constexpr int E = D / 64;
    const int lane = threadIdx.x, head = blockIdx.y;
    const int first = a.cu[0] < 0 ? 0 : a.cu[0];
    SeqTile t;
    if (!find_tile(a.cu, (int)a.seqs, a.m, blockIdx.x - first, [](int, int n) { return n; }, t)) return;
    const int64_t row = t.begin + t.tile;
    const int64_t kv = head / (a.q_heads / a.kv_heads);
    float q[E], o[E] = {}, mx = kNegInf, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = to_f32(static_cast<const T *>(a.q)[row * a.q_stride + head * D + e * 64 + lane]);
    for (int64_t j = t.begin; j <= row; ++j) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s = __builtin_fmaf(q[e], to_f32(static_cast<const T *>(a.k)[j * a.k_stride + kv * D + e * 64 + lane]), s);
        s = wave_sum_f32(s) * (a.scale * kLog2e);
        const float now = fmaxf(mx, s), keep = __builtin_amdgcn_exp2f(mx - now), p = __builtin_amdgcn_exp2f(s - now);
        mx = now;
        l = __builtin_fmaf(l, keep, p);
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = __builtin_fmaf(o[e], keep, p * to_f32(static_cast<const T *>(a.v)[j * a.v_stride + kv * D + e * 64 + lane]));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) store_out(static_cast<T *>(a.out) + (row * a.q_heads + head) * D + e * 64 + lane, o[e] / l);
}

// ---------------------------------------------------------------- bf16 on the matrix cores
//
// A workgroup of 4 waves takes 128 query rows of one kv head (64 with KS = 2): row
// r of a sequence is token r / group, query head r % group, so the heads that
// share K and V share their tiles and short prompts fill a tile. A wave has 32
// rows, and everything of a row in one lane pair:
//   S^T = K Q^T      (v_mfma_f32_32x32x16_bf16, A = 32 keys, B = 32 query rows)
//   O^T = V^T P^T    (A = 32 dims of V read transposed from LDS, B = P)
// The result's column is lane % 32, so maximum, sum and rescaling are per lane,
// joined with lane ^ 32 alone; and S^T's registers are P^T's operand as they lie
// when V's keys are taken in the order 4h .. 4h+3, 8+4h .. 8+4h+3 (h = lane / 32)
// of every 16: P never leaves the registers.
// K and V tiles of 64 keys come by direct loads into two LDS buffers, one barrier
// per tile. 16-byte chunks are permuted within a row by the global address, so
// that the operand reads touch every bank once (conflicts: 1 % of the LDS time).
// P is rounded to bf16 for its product with V, as the inputs are; sums and
// statistics stay in fp32.
// Bound by the matrix cores and the softmax's VALU work in about equal parts (55 %
// and 50 % of the cycles at 8192 tokens), which two waves per SIMD overlap poorly.
// Measured and not kept: eight waves per workgroup (536 against 543 us at 8192
// tokens, 57.9 against 46.4 at 2048), raised wave priority around the products
// (545 to 551), the row sum by dot products of pairs (551), 64 rows per wave with
// the next tile's logits formed beside the softmax (registers spill: 1757 us).
constexpr int kKeys = 64;

template <int D>
__device__ inline int k_swizzle(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D>
__device__ inline int v_swizzle(int row) { return D == 128 ? (row & 3) << 2 : (row & 2) << 1; }

// value of both halves of the wave: (lower, upper)
__device__ inline void both_halves(float v, float &lower, float &upper)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    lower = __uint_as_float(r[0]);
    upper = __uint_as_float(r[1]);
}

// Rescaling is put off until a maximum has grown by 2^kSlack: p stays below that,
// which neither bf16 nor the fp32 sums notice.
constexpr float kSlack = 8.0f;

constexpr int kSchedMatrix = 0x8, kSchedLdsRead = 0x100;

// Where a tile's mask leaves out keys, 0 * v must not bring a NaN or infinity of
// theirs into the sum. The workgroup looks through such a tile of V (the last one
// or two) when it has arrived; what is not finite becomes 0 there, and a second
// tile holds what it was: +inf as 1, -inf as 2^7, NaN as 2^14. A product of that
// tile with the mask counts per dim and row what the row sees (at most 64 of each,
// so fp32 holds all three counts).
__device__ inline bool not_finite_pair(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u || (w & 0x7F80u) == 0x7F80u; }
__device__ inline uint32_t finite_pair(uint32_t w)
{
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    if ((w & 0x00007F80u) == 0x00007F80u) w &= 0xFFFF0000u;
    return w;
}
__device__ inline uint32_t counted(uint32_t b)  // of bf16 bits, as bf16 bits
{
    return (b & 0x7F80u) != 0x7F80u ? 0u : b & 0x7Fu ? 0x4680u : b & 0x8000u ? 0x4300u : 0x3F80u;
}
__device__ inline uint32_t counted_pair(uint32_t w) { return counted(w & 0xFFFFu) | counted(w >> 16) << 16; }
__device__ inline float counted_value(float n)
{
    const int c = (int)n, plus = c & 127, minus = (c >> 7) & 127;
    return c >= 1 << 14 || (plus && minus) ? __builtin_nanf("") : plus ? __builtin_inff() : minus ? kNegInf : 0.0f;
}

template <int D, int KS>
__global__ __launch_bounds__(256, 2) void attention_bf16_kernel(AttentionProblem a, int group)
{
    constexpr int ROWS = 128 / KS, C = D / 16, DT = D / 32, NB = 2 / KS;
    constexpr int kTile = kKeys * D * 2;                  // bytes of a K or V tile
    constexpr int kLoads = kTile / (1024 * 4);            // direct loads per wave and tile
    constexpr int kChunks = D / 8;                        // 16-byte chunks per row
    constexpr int kLoadRows = kKeys / kLoads;             // rows that one load of the four waves brings
    // K, K, V, V, counts of what is not finite
    __shared__ __align__(1024) char lds[5 * kTile];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, col = lane & 31;
    const int head = blockIdx.x % (int)a.kv_heads;
    SeqTile t;
    if (!find_tile(a.cu, (int)a.seqs, a.m, blockIdx.x / (int)a.kv_heads,
                   [=](int, int n) { return (int)(((int64_t)n * group + ROWS - 1) / ROWS); }, t))
        return;
    const int rows = t.n * group;
    t.tile = (rows + ROWS - 1) / ROWS - 1 - t.tile;       // the longest rows first
    const int r_wave = t.tile * ROWS + wave / KS * 32;
    const int b0 = KS == 1 ? 0 : wave % KS;               // the wave's 32-key blocks of a tile: b0 .. b0+NB-1

    // query rows (rows past the last one repeat it and are not stored)
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    int tok;
    v8bf qf[C];
    {
        int r = r_wave + col;
        r = r < rows ? r : rows - 1;
        tok = r / group;
        const bf16_t *src = static_cast<const bf16_t *>(a.q) + (t.begin + tok) * a.q_stride +
                            (int64_t)(head * group + r % group) * D + 8 * h;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            uint4 w = *reinterpret_cast<const uint4 *>(src + 16 * i);
            w = make_uint4(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip);
            qf[i] = __builtin_bit_cast(v8bf, w);
        }
    }
    const int last_row = t.tile * ROWS + ROWS < rows ? t.tile * ROWS + ROWS - 1 : rows - 1;
    const int tiles = last_row / group / kKeys + 1;
    // first tile that some row of the workgroup, of the wave, does not see whole
    const int group_masked = (t.tile * ROWS / group + 1) / kKeys;
    const int wave_masked = ((r_wave < rows ? r_wave : rows - 1) / group + 1) / kKeys;

    // direct loads: load i of the four waves brings rows kLoadRows*i .. kLoadRows*(i+1)-1 of a tile
    const uint32_t base = lds_addr(lds);
    const int load_row = wave * (kLoadRows / 4) + lane / kChunks;
    const int k_chunk = ((lane % kChunks) ^ k_swizzle<D>(load_row)) * 16, v_chunk = ((lane % kChunks) ^ v_swizzle<D>(load_row)) * 16;
    const uint32_t k_off = (uint32_t)load_row * (uint32_t)(a.k_stride * 2) + k_chunk;
    const uint32_t v_off = (uint32_t)load_row * (uint32_t)(a.v_stride * 2) + v_chunk;
    auto bring = [&](const void *x, int64_t stride, uint32_t off, int chunk, int tile, uint32_t to) {
        const int64_t first = t.begin + (int64_t)tile * kKeys;
        const int left = t.n - 1 - tile * kKeys;
        const bf16_t *from = static_cast<const bf16_t *>(x) + first * stride + (int64_t)head * D;
        if (left >= kKeys - 1) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) dma16(from + i * kLoadRows * stride, off, to + (4 * i + wave) * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = i * kLoadRows + load_row;
                dma16(from, (uint32_t)(row < left ? row : left) * (uint32_t)(stride * 2) + chunk, to + (4 * i + wave) * 1024);
            }
        }
    };
    auto request = [&](int tile) {
        bring(a.k, a.k_stride, k_off, k_chunk, tile, base + (tile & 1) * kTile);
        bring(a.v, a.v_stride, v_off, v_chunk, tile, base + (2 + (tile & 1)) * kTile);
    };

    // operand addresses inside a tile; rows 32 keys further on, and 8 keys for V, are constant offsets
    int k_at[C], v_at[DT];
#pragma unroll
    for (int i = 0; i < C; ++i) k_at[i] = (32 * b0 + col) * (D * 2) + (((2 * i + h) ^ k_swizzle<D>(col)) << 4);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
        const int key = 4 * h + ((lane & 15) >> 2), chunk = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        v_at[d] = (32 * b0 + key) * (D * 2) + ((chunk ^ v_swizzle<D>(key)) << 4) + (lane & 1) * 8;
    }
    auto k_fragment = [&](int tile, int b, int i) {
        return *reinterpret_cast<const v8bf *>(lds + (tile & 1) * kTile + k_at[i] + b * 32 * D * 2);
    };
    // 16 lanes read 4 keys x 16 dims and get 4 keys of one dim each
    auto v_fragment = [&](int place, int kc, int d) {
        v4s part[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(uintptr_t)(
                base + place * kTile + v_at[d] + (16 * kc + 8 * e) * D * 2));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };

    v16f o[DT];
    float mx = kNegInf, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = v16f{};

    // V of a masked tile, once it is there: keeps what is not finite from rows that do not see it
    auto clean = [&](int tile) {
        char *vt = lds + (2 + (tile & 1)) * kTile + wave * (kTile / 4) + lane * 16, *ct = lds + 4 * kTile + wave * (kTile / 4) + lane * 16;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kTile / 4096; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(vt + i * 1024);
            bad = bad || not_finite_pair(w.x) || not_finite_pair(w.y) || not_finite_pair(w.z) || not_finite_pair(w.w);
        }
        int *flags = reinterpret_cast<int *>(lds + 4 * kTile);
        bad = __any(bad);
        if (lane == 0) flags[wave] = bad;
        __syncthreads();
        if (!(flags[0] | flags[1] | flags[2] | flags[3])) return;
        __syncthreads();
        for (int i = 0; i < kTile / 4096; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(vt + i * 1024);
            *reinterpret_cast<uint4 *>(vt + i * 1024) = make_uint4(finite_pair(w.x), finite_pair(w.y), finite_pair(w.z), finite_pair(w.w));
            *reinterpret_cast<uint4 *>(ct + i * 1024) = make_uint4(counted_pair(w.x), counted_pair(w.y), counted_pair(w.z), counted_pair(w.w));
        }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            v16f count = {};
#pragma unroll
            for (int n = 0; n < 2 * NB; ++n) {
                const int kc = 2 * b0 + n;
                v8bf seen;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    seen[i] = (__bf16)(tile * kKeys + 16 * kc + 8 * (i >> 2) + 4 * h + (i & 3) <= tok ? 1.0f : 0.0f);
                count = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_fragment(4, n, d), seen, count, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] += counted_value(count[i]);
        }
    };

    request(0);
    for (int tile = 0; tile < tiles; ++tile) {
        ring_barrier<0>();
        if (tile + 1 < tiles) request(tile + 1);
        if (tile >= group_masked) clean(tile);

        v16f s[NB];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_fragment(tile, b, i), qf[i], i ? s[b] : v16f{}, 0, 0, 0);
        // the operand reads run kAhead fragments ahead of the products
        constexpr int kAhead = 6;
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, kAhead, 0);
#pragma unroll
        for (int i = 0; i < NB * C - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, kAhead, 0);
        if (tile >= wave_masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = tile * kKeys + 32 * (b0 + b) + 8 * (i >> 2) + 4 * h + (i & 3);
                    s[b][i] = key <= tok ? s[b][i] : kNegInf;
                }
        }
        float big = kNegInf, lo, up;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) big = fmaxf(big, s[b][i]);
        both_halves(big, lo, up);
        big = fmaxf(lo, up) * c;
        if (__any(big > mx + kSlack)) {
            // only where it has grown: a row's result does not depend on its neighbours
            const float now = big > mx + kSlack ? big : mx;
            const float keep = now == mx ? 1.0f : __builtin_amdgcn_exp2f(mx - now);
            mx = now;
            sum *= keep;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= keep;
        }
        const float ref = KS > 1 && mx == kNegInf ? 0.0f : mx;  // -inf: none of the wave's keys is seen yet
        v8bf p[2 * NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ref));
                sum += e;
                p[2 * b + (i >> 3)][i & 7] = (__bf16)e;
            }
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_fragment(2 + (tile & 1), n, d), p[n], o[d], 0, 0, 0);
    }

    if constexpr (KS > 1) {
        // the wave with the tiles' upper keys hands its part over, 4 lanes' values of 16 bytes at a time
        __syncthreads();
        float *part = reinterpret_cast<float *>(lds + wave / KS * (DT * 4096 + 512));
        if (b0) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<v4f *>(part + ((d * 4 + g) * 64 + lane) * 4) =
                        v4f{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
            part[DT * 1024 + lane] = mx;
            part[DT * 1024 + 64 + lane] = sum;
        }
        __syncthreads();
        if (b0) return;
        const float other = part[DT * 1024 + lane], top = fmaxf(mx, other);
        const float f0 = __builtin_amdgcn_exp2f(mx - top), f1 = __builtin_amdgcn_exp2f(other - top);
        sum = __builtin_fmaf(sum, f0, part[DT * 1024 + 64 + lane] * f1);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const v4f w = *reinterpret_cast<const v4f *>(part + ((d * 4 + g) * 64 + lane) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][4 * g + i] = __builtin_fmaf(o[d][4 * g + i], f0, w[i] * f1);
            }
    }
    float lo, up;
    both_halves(sum, lo, up);
    const float inv = 1.0f / (lo + up);
    const int r = r_wave + col;
    if (r >= rows) return;
    bf16_t *dst = static_cast<bf16_t *>(a.out) + ((t.begin + tok) * a.q_heads + head * group + r % group) * D + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            bf16_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) store_out(&w[i], o[d][4 * g + i] * inv);
            *reinterpret_cast<uint2 *>(dst + 32 * d + 8 * g) = *reinterpret_cast<const uint2 *>(w);
        }
}

// Few workgroups: a tile's keys are split over two waves (KS = 2), so that there
// are twice as many and the longest takes half as long. It pays up to one and a
// half workgroups per CU, three for 64-wide heads, whose LDS lets more of them
// share a CU (20/5 heads of 128, one prompt, KS = 1 / 2: 1024 tokens 24.3 / 21.1
// us, 2048 44.2 / 39.2, 3000 68.2 / 72.7, 4096 103 / 119; 16/4 heads of 64, 4096
// tokens: 62.6 / 53.4).
constexpr int64_t kFewGroups128 = 384, kFewGroups64 = 768;

int64_t attention_workspace(const AttentionProblem &) { return 0; }

hipError_t launch_attention(const AttentionProblem &p, void *, hipStream_t st)
{
    const int group = (int)(p.q_heads / p.kv_heads);
    if (p.bf16) {
        auto go = [&](auto width, auto splits) {
            constexpr int D = decltype(width)::value, KS = decltype(splits)::value;
            const int64_t n = p.m * group * KS / 128 + p.seqs;
            hipLaunchKernelGGL((attention_bf16_kernel<D, KS>), dim3((unsigned)(n * p.kv_heads)), dim3(256), 0, st, p, group);
        };
        const int64_t groups = (p.m * group / 128 + p.seqs) * p.kv_heads;
        if (p.head_dim == 128) groups > kFewGroups128 ? go(Width<128>{}, Width<1>{}) : go(Width<128>{}, Width<2>{});
        else groups > kFewGroups64 ? go(Width<64>{}, Width<1>{}) : go(Width<64>{}, Width<2>{});
        return hipGetLastError();
    }
    const dim3 grid((unsigned)p.m, (unsigned)p.q_heads);
    if (p.head_dim == 128) hipLaunchKernelGGL((attention_kernel<float, 128>), grid, dim3(64), 0, st, p);
    else hipLaunchKernelGGL((attention_kernel<float, 64>), grid, dim3(64), 0, st, p);
    return hipGetLastError();
}

}  // namespace bl
