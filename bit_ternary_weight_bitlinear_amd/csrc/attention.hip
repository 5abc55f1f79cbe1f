// attention.hip -- causal attention over packed prompts.
//
//   out_i = sum_{j <= i} p_ij v_j,   p_i = softmax_j(scale * q_i . k_j)
//
// One pass over the keys with the running maximum and sum of the softmax.
#include "attention.hpp"

namespace bl {

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
// and 50 % of the cycles at 8192 tokens), which two waves per SIMD overlap poorly:
// 510 to 545 us there (box to box), 1.01 to 1.08 PFLOP/s, where a plain bf16
// product of 16384^3 reaches 1.39. The clock falls to 1.6 GHz meanwhile (2.4 in
// shorter calls), so power bounds it too.
// With KS = 2 a SIMD mostly has one wave, whose products, softmax and LDS reads would
// follow one another: there K runs a tile ahead, the next tile's logits are formed
// beside this one's softmax, and all operands are read ahead of both (2048 tokens,
// 20/5 heads: 33.5 us beside 36.5; 2500 tokens of 6/2 heads 32.3 beside 36.5). Two
// waves per SIMD gain nothing from it (343 beside 337 at 8192 tokens, 20/5 heads).
// Measured and not kept, at 8192 tokens beside 520 to 543 us: eight waves per
// workgroup (536; 57.9 against 46.4 at 2048 tokens), those in two groups of four,
// half a step apart, so that one's products meet the other's softmax (577), raised
// wave priority around the products (545 to 551), the row sum by dot products of
// pairs (551), V's operands read before the softmax (533 beside 509), 64 rows per
// wave, one's products beside the other's softmax (580 beside 518: the 512 registers
// that it needs are half accumulation registers, reached by copies).
// With KS = 2, at 2500 tokens of 6/2 heads beside 32.5 us: four buffers instead of
// two (35.2), products and softmax interleaved by hand (33.8 to 39).

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

// |scale| log2 e; neither 0 nor infinite, so that it leaves masked logits, and ones of 0, as they are
__device__ inline float logit_factor(float scale) { return fminf(fmaxf(fabsf(scale) * kLog2e, 1e-45f), 3.402823466e38f); }

constexpr int kSchedMatrix = 0x8, kSchedLdsRead = 0x100;

// Elements of V that are not finite: 0 * v must not bring them into rows that do not see
// them, and a rescale by 2^-inf must not make a NaN of an infinity. Where a tile's mask
// leaves out keys, the workgroup looks through such a tile of V (the last one or two) when
// it has arrived and sets them to 0. What they make of a row is settled when it is stored.
__device__ inline bool not_finite_pair(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w >> 16 & 0x7F80u) == 0x7F80u; }
__device__ inline uint32_t finite_pair(uint32_t w)
{
    if ((w >> 16 & 0x7F80u) == 0x7F80u) w &= 0x0000FFFFu;
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    return w;
}

// by the workgroup: whether the tile held any
template <int BYTES, int WAVES>
__device__ inline bool set_aside(char *tile, int *flags)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    char *vt = tile + wave * (BYTES / WAVES) + lane * 16;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < BYTES / (1024 * WAVES); ++i) {
        const uint4 w = *reinterpret_cast<const uint4 *>(vt + i * 1024);
        bad = bad || not_finite_pair(w.x) || not_finite_pair(w.y) || not_finite_pair(w.z) || not_finite_pair(w.w);
    }
    int any = 0;
    bad = __any(bad);
    if (lane == 0) flags[wave] = bad;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) any |= flags[i];
    if (!any) return false;
    for (int i = 0; i < BYTES / (1024 * WAVES); ++i) {
        const uint4 w = *reinterpret_cast<const uint4 *>(vt + i * 1024);
        *reinterpret_cast<uint4 *>(vt + i * 1024) = make_uint4(finite_pair(w.x), finite_pair(w.y), finite_pair(w.z), finite_pair(w.w));
    }
    __syncthreads();
    return true;
}

// four adjacent elements
template <typename T>
struct Adjacent {
    typedef v4f type;
};
template <>
struct Adjacent<bf16_t> {
    typedef uint2 type;
};

// bit e (+inf or NaN) and 4 + e (-inf or NaN) of what four adjacent elements are
template <typename T>
__device__ inline int odd_kinds(typename Adjacent<T>::type four)
{
    T w[4];
    __builtin_memcpy(w, &four, sizeof(w));
    int kinds = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float f = to_f32(w[e]);
        const bool finite = fabsf(f) <= 3.402823466e38f;
        kinds |= (!finite && f != kNegInf ? 1 << e : 0) | (!finite && f != -kNegInf ? 16 << e : 0);
    }
    return kinds;
}

// By the wave: groups first .. first+n-1 of its stored rows (dims 32 * (i / 4) + 8 * (i % 4)
// + 4h .. +3; `wanted` where a lane has a row), once more where they are not finite or V
// was set aside: an element becomes NaN where the row sees a NaN, or infinities of both
// signs, among its `keys` elements of V, and the infinity where it sees one. The keys that
// all rows see are looked through by 32 lanes together. Only inputs that hold such values
// come here (8192 tokens, 32/8 heads of 128 in bf16: 0.69 ms with an infinity in the
// first row, 2.7 with one in every row, 0.54 without).
template <typename T>
__device__ inline void settle(T *dst, const T *v, int64_t stride, int keys, int first, int n, bool aside, bool wanted)
{
    const int col = threadIdx.x & 31, common = __builtin_amdgcn_readfirstlane(keys);  // rows ascend
    for (int i = first; i < first + n; ++i) {
        const int at = 32 * (i >> 2) + 8 * (i & 3);
        // read and written as the type that it was stored as
        using Four = typename Adjacent<T>::type;
        Four *four = reinterpret_cast<Four *>(dst + at), was = {};
        if (wanted) was = *four;
        const bool odd = wanted && (aside || odd_kinds<T>(was));
        if (!__any(odd)) continue;
        auto at_key = [&](int j) { return *reinterpret_cast<const Four *>(v + j * stride + at); };
        int kinds = 0;
#pragma unroll 4
        for (int j = col; j < common && kinds != 0xFF; j += 32) kinds |= odd_kinds<T>(at_key(j));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) kinds |= __shfl_xor(kinds, d);
        for (int j = common; j < keys; ++j) kinds |= odd_kinds<T>(at_key(j));
        if (!odd) continue;
        T now[4];
        __builtin_memcpy(now, &was, sizeof(now));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool plus = kinds >> e & 1, minus = kinds >> (4 + e) & 1;
            if (plus || minus) store_out(&now[e], plus && minus ? __builtin_nanf("") : plus ? -kNegInf : kNegInf);
        }
        __builtin_memcpy(&was, now, sizeof(now));
        *four = was;
    }
}

// registers 4 * (i % 4) .. +3 of accumulator i / 4
template <int DT>
__device__ inline v4f o_group(const v16f (&o)[DT], int i)
{
    const int d = i >> 2, g = 4 * (i & 3);
    return v4f{o[d][g], o[d][g + 1], o[d][g + 2], o[d][g + 3]};
}

template <int DT>
constexpr int kJoinPart = DT * 4096 + 3 * 256;  // bytes of a wave's results

// KS neighbouring waves hold the same rows over different keys: each writes its
// accumulators, maximum, sum and the scale of its accumulators (relative to 2^mx) and
// joins a KS-th of the dims, which it gives to store with 1 / sum and the scale.
template <int DT, int KS, typename F>
__device__ inline void join_waves(char *lds, const v16f (&o)[DT], float mx, float sum, float scale, F store)
{
    constexpr int kPart = kJoinPart<DT>, N = 4 * DT / KS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), mine = wave % KS;
    char *parts = lds + wave / KS * KS * kPart;
    __syncthreads();
    {
        float *to = reinterpret_cast<float *>(parts + mine * kPart);
        float lo, up;
        both_halves(sum, lo, up);
#pragma unroll
        for (int i = 0; i < 4 * DT; ++i) *reinterpret_cast<v4f *>(to + (i * 64 + lane) * 4) = o_group(o, i);
        to[DT * 1024 + lane] = mx;
        to[DT * 1024 + 64 + lane] = lo + up;
        to[DT * 1024 + 128 + lane] = scale;
    }
    __syncthreads();
    float top = kNegInf, most = 0.0f, all = 0.0f, f[KS];
    const float *from = reinterpret_cast<const float *>(parts);
    constexpr int kStep = kPart / 4;
#pragma unroll
    for (int p = 0; p < KS; ++p) top = fmaxf(top, from[p * kStep + DT * 1024 + lane]);
#pragma unroll
    for (int p = 0; p < KS; ++p) {
        const float e = __builtin_amdgcn_exp2f(from[p * kStep + DT * 1024 + lane] - top);
        all = __builtin_fmaf(from[p * kStep + DT * 1024 + 64 + lane], e, all);
        f[p] = from[p * kStep + DT * 1024 + 128 + lane] * e;
        most = fmaxf(most, f[p]);
    }
#pragma unroll
    for (int p = 0; p < KS; ++p) f[p] /= most;
    const float inv = 1.0f / all;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = mine * N + n;
        v4f v = {};
#pragma unroll
        for (int p = 0; p < KS; ++p) {
            const v4f w = *reinterpret_cast<const v4f *>(from + p * kStep + (i * 64 + lane) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(w[e], f[p], v[e]);
        }
        store(i, v, inv, most);
    }
}

template <int D, int KS>
__global__ __launch_bounds__(256, 2) void attention_bf16_kernel(AttentionProblem a, int group, int first_group)
{
    constexpr bool AHEAD = KS > 1;
    constexpr int WAVES = 4, ROWS = 32 * WAVES / KS, KEYS = 64;
    constexpr int C = D / 16, DT = D / 32, NB = KEYS / 32 / KS;
    constexpr int kTile = KEYS * D * 2;                   // bytes of a K or V tile
    constexpr int kLoads = kTile / (1024 * WAVES);        // direct loads per wave and tile
    constexpr int kChunks = D / 8;                        // 16-byte chunks per row
    constexpr int kLoadRows = KEYS / kLoads;              // rows that one load of all waves brings
    constexpr int kTiles = 4 * kTile, kJoin = KS > 1 ? WAVES * kJoinPart<DT> : 0;
    __shared__ __align__(1024) char lds[kTiles > kJoin ? kTiles : kJoin];  // K, K, V, V; the waves' results
    __shared__ int flags[WAVES];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, col = lane & 31;
    const int index = first_group + (int)blockIdx.x, head = index % (int)a.kv_heads;
    SeqTile t;
    if (!find_tile(a.cu, (int)a.seqs, a.m, index / (int)a.kv_heads,
                   [=](int, int n) { return (int)(((int64_t)n * group + ROWS - 1) / ROWS); }, t))
        return;
    const int rows = t.n * group;
    t.tile = (rows + ROWS - 1) / ROWS - 1 - t.tile;       // the longest rows first
    const int r_wave = t.tile * ROWS + wave / KS * 32;
    const int b0 = KS == 1 ? 0 : wave % KS;               // the wave's 32-key blocks of a tile: b0 .. b0+NB-1

    // query rows (rows past the last one repeat it and are not stored)
    const float c = logit_factor(a.scale);
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
    const int tiles = last_row / group / KEYS + 1;
    // first tile that some row of the workgroup, of the wave, does not see whole
    const int group_masked = (t.tile * ROWS / group + 1) / KEYS;
    const int wave_masked = ((r_wave < rows ? r_wave : rows - 1) / group + 1) / KEYS;

    // direct loads: load i of the waves brings rows kLoadRows*i .. kLoadRows*(i+1)-1 of a tile
    const uint32_t base = lds_addr(lds);
    const int load_row = wave * (kLoadRows / WAVES) + lane / kChunks;
    const int k_chunk = ((lane % kChunks) ^ k_swizzle<D>(load_row)) * 16, v_chunk = ((lane % kChunks) ^ v_swizzle<D>(load_row)) * 16;
    const uint32_t k_off = (uint32_t)load_row * (uint32_t)(a.k_stride * 2) + k_chunk;
    const uint32_t v_off = (uint32_t)load_row * (uint32_t)(a.v_stride * 2) + v_chunk;
    auto bring = [&](const void *x, int64_t stride, uint32_t off, int chunk, int tile, uint32_t to) {
        const int64_t first = t.begin + (int64_t)tile * KEYS;
        const int left = t.n - 1 - tile * KEYS;
        const bf16_t *from = static_cast<const bf16_t *>(x) + first * stride + (int64_t)head * D;
        if (left >= KEYS - 1) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) dma16(from + i * kLoadRows * stride, off, to + (WAVES * i + wave) * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = i * kLoadRows + load_row;
                dma16(from, (uint32_t)(row < left ? row : left) * (uint32_t)(stride * 2) + chunk, to + (WAVES * i + wave) * 1024);
            }
        }
    };
    auto request_k = [&](int tile) { bring(a.k, a.k_stride, k_off, k_chunk, tile, base + (tile & 1) * kTile); };
    auto request_v = [&](int tile) { bring(a.v, a.v_stride, v_off, v_chunk, tile, base + (2 + (tile & 1)) * kTile); };

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

    bool aside = false;  // a masked tile of V held values that are not finite
    v16f s[NB];
    // the fragments in the order of their use: n / NB is the 16 dims, n % NB the block of keys
    auto k_nth = [&](int tile, int n) { return k_fragment(tile, n % NB, n / NB); };
    auto logits = [&](v16f (&to)[NB], auto fragment) {
#pragma unroll
        for (int n = 0; n < NB * C; ++n)
            to[n % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fragment(n), qf[n / NB], n / NB ? to[n % NB] : v16f{}, 0, 0, 0);
    };
    v8bf kf[AHEAD ? NB * C : 1];
    auto read_k = [&](int tile) {
#pragma unroll
        for (int n = 0; n < NB * C; ++n) kf[n] = k_nth(tile, n);
    };
    auto k_read = [&](int n) { return kf[n]; };

    request_k(0);
    // every logit 0, also where q . k overflows (behind the request: q's rows are waited for here)
    if (a.scale == 0.0f)
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) qf[i][e] = (__bf16)((float)qf[i][e] * 0.0f);
    if constexpr (AHEAD) {
        ring_barrier<0>();
        request_v(0);
        if (tiles > 1) request_k(1);
        read_k(0);
        logits(s, k_read);
    } else {
        request_v(0);
    }
    for (int tile = 0; tile < tiles; ++tile) {
        ring_barrier<0>();
        if (!AHEAD && tile + 1 < tiles) request_k(tile + 1);
        if (tile + 1 < tiles) request_v(tile + 1);
        if (AHEAD && tile + 2 < tiles) request_k(tile + 2);
        if (tile >= group_masked) aside |= set_aside<kTile, WAVES>(lds + (2 + (tile & 1)) * kTile, flags);

        if constexpr (AHEAD) {
            read_k(tile + 1);  // old bytes of the buffer, and of no use, behind the last tile
        } else {
            logits(s, [&](int n) { return k_nth(tile, n); });
            // the operand reads run kAhead fragments ahead of the products
            constexpr int kAhead = 6;
            __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, kAhead, 0);
#pragma unroll
            for (int i = 0; i < NB * C - kAhead; ++i) {
                __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 1, 0);
                __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(kSchedMatrix, kAhead, 0);
        }
        if (tile >= wave_masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = tile * KEYS + 32 * (b0 + b) + 8 * (i >> 2) + 4 * h + (i & 3);
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
        const float ref = mx == kNegInf ? 0.0f : mx;  // -inf: no key with a weight yet
        v8bf vf[AHEAD ? 2 * NB : 1][DT];
        v16f next[NB];
        if constexpr (AHEAD) {
#pragma unroll
            for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
                for (int d = 0; d < DT; ++d) vf[n][d] = v_fragment(2 + (tile & 1), n, d);
            logits(next, k_read);
        }
        auto v_nth = [&](int n, int d) {
            if constexpr (AHEAD) return vf[n][d];
            else return v_fragment(2 + (tile & 1), n, d);
        };
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
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_nth(n, d), p[n], o[d], 0, 0, 0);
        if constexpr (AHEAD) {
            __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 4 * NB * DT, 0);
#pragma unroll
            for (int b = 0; b < NB; ++b) s[b] = next[b];
        }
    }

    const int r = r_wave + col;
    bf16_t *dst = static_cast<bf16_t *>(a.out) + ((t.begin + tok) * a.q_heads + head * group + r % group) * D + 4 * h;
    float all = 0.0f, norm = 0.0f;
    auto store = [&](int i, const v4f &v, float inv, float) {  // dims 32 * (i / 4) + 8 * (i % 4) + 4 * h .. +3
        bf16_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) store_out(&w[e], v[e] * inv);
        *reinterpret_cast<uint2 *>(dst + 32 * (i >> 2) + 8 * (i & 3)) = *reinterpret_cast<const uint2 *>(w);
        all += (v[0] + v[1]) + (v[2] + v[3]);
        norm = inv;
    };
    if constexpr (KS == 1) {
        float lo, up;
        both_halves(sum, lo, up);
        const float inv = 1.0f / (lo + up);
        if (r < rows)
#pragma unroll
            for (int i = 0; i < 4 * DT; ++i) store(i, o_group(o, i), inv, 1.0f);
    } else {
        join_waves<DT, KS>(lds, o, mx, sum, 1.0f, [&](int i, const v4f &v, float inv, float one) { if (r < rows) store(i, v, inv, one); });
    }
    // not where the weights have no sum: such a row is NaN whatever V holds
    const bool wanted = (aside || all - all != 0.0f) && norm - norm == 0.0f && r < rows;
    if (__any(wanted))
        settle(dst, static_cast<const bf16_t *>(a.v) + t.begin * a.v_stride + head * D + 4 * h, a.v_stride, tok + 1, wave % KS * (4 * DT / KS), 4 * DT / KS, aside, wanted);
}

// ---------------------------------------------------------------- fp32 on the matrix cores
//
// fp32 products from fp16 ones: x = 2^a (hi + lo) with hi the nearest fp16 of
// x / 2^a and lo that of the rest (22 bits and a sign), a such that the row's
// largest magnitude lies in 2^14 .. 2^15; then xy ~ hi hi' + hi lo' + lo hi', off
// by 3 * 2^-22 of |x||y| at most, with fp32 sums. Rows' elements below 2^-17 of the
// largest keep 2^-39 of it (fp16's smallest step is 2^-24), and with a >= -112 none is
// held closer than 2^-137. Three matrix products instead of one on the fp32 matrix
// cores, whose rate is a sixteenth.
// A first kernel writes K and V in this form, once per row (the rows that read
// them split nothing): [head][token][hi, lo][D], and 2^a per row (of K 2^(a - 23): the
// sums are below 2^38, and large rows of K must not overflow where those of q are small).
// The scale of K's rows multiplies the logits. That of V's rows goes into the
// weights: w_j = p_j 2^a_j / ref with ref the running maximum of p_j 2^a_j, so that
// hi and lo of w keep 22 bits of the largest products (and a row of V counts for as
// much as its weight lets it, however large it is).
// An infinity times a second part, which may be 0 or of the other sign, is not what the
// definition has. K's elements that are not finite are lo, with a hi of 0: lo meets q's
// first part only, and the product has q's sign (q's own make their rows NaN either way).
// V's are 0 in both parts, and their row's scale is negative: rows that see one are
// settled when they are stored.
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
constexpr float kSlackF32 = 3.0f;      // as kSlack
constexpr float kMostWeight = 8.0f;    // the same for w ...
constexpr float kWeightOne = 2048.0f;  // ... so that w times this stays below 2^14
constexpr int kKeyShift = 23, kMostQuery = 100;  // a row of q's a above this is made up for apart

// a of a row whose largest finite magnitude is big; 2^a and 2^-a are normal, and so are
// the smallest weights that count relative to it
__device__ inline int row_exponent(float big)
{
    const int a = (int)(__float_as_uint(big) >> 23) - 127 - 14;
    return a < -112 ? -112 : a;
}
__device__ inline float power_of_two(int a) { return __uint_as_float((uint32_t)(a + 127) << 23); }
__device__ inline float finite_abs(float v) { return fabsf(v) <= 3.402823466e38f ? fabsf(v) : 0.0f; }
__device__ inline void split_f16(float v, _Float16 &hi, _Float16 &lo)
{
    hi = (_Float16)v;
    const float rest = v - (float)hi;
    lo = (_Float16)(rest - rest == 0.0f ? rest : 0.0f);
}

// A product as the fp32 number it rounds to. Without this the compiler may round it
// to fp16 in one step where hi is used and in two where the rest is formed; near a
// tie these differ by a unit of hi.
__device__ inline float rounded(float v)
{
    asm("" : "+v"(v));
    return v;
}

// D / 4 lanes per row of K or V (blockIdx.y: 0, 1)
template <int D>
__global__ __launch_bounds__(256) void attention_split_kernel(AttentionProblem a, char *__restrict__ planes,
                                                              float *__restrict__ scales, int first_group)
{
    constexpr int L = D / 4;
    const int64_t rows = a.m * a.kv_heads, n = ((int64_t)first_group + blockIdx.x) * (256 / L) + threadIdx.x / L;
    if (n >= rows) return;
    const int64_t tok = n / a.kv_heads, head = n % a.kv_heads, at = head * a.m + tok;
    const int is_v = blockIdx.y, lane = threadIdx.x % L;
    const float *src = static_cast<const float *>(is_v ? a.v : a.k) + tok * (is_v ? a.v_stride : a.k_stride) + head * D + 4 * lane;
    const float4 x = *reinterpret_cast<const float4 *>(src);
    float big = fmaxf(fmaxf(finite_abs(x.x), finite_abs(x.y)), fmaxf(finite_abs(x.z), finite_abs(x.w)));
#pragma unroll
    for (int d = 1; d < L; d <<= 1) big = fmaxf(big, __shfl_xor(big, d));
    const int exponent = row_exponent(big);
    const float inv = power_of_two(-exponent);
    _Float16 hi[4], lo[4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = (&x.x)[i];
        const bool odd = !(fabsf(f) <= 3.402823466e38f);
        split_f16(odd ? 0.0f : f * inv, hi[i], lo[i]);
        if (odd && !is_v) lo[i] = (_Float16)f;
        bad |= odd && is_v;
    }
    const uint64_t any = __ballot(bad) >> (threadIdx.x & 63 & ~(L - 1)) & ((1ull << L) - 1);
    char *dst = planes + (is_v * rows + at) * (D * 4) + lane * 8;
    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(hi);
    *reinterpret_cast<uint2 *>(dst + D * 2) = *reinterpret_cast<const uint2 *>(lo);
    const float scale = power_of_two(exponent);
    if (lane == 0) scales[is_v * rows + at] = !is_v ? scale * power_of_two(-kKeyShift) : any ? -scale : scale;
}

// The loop of attention_bf16_kernel (as it is there with KS = 1) with the four 16-bit
// planes of a tile of 32 * KS keys, 32 keys per wave. Bound by the matrix cores: 8192
// tokens, 32/8 heads of 128: 1.49 ms, 369 TFLOP/s of fp32 (three times that in
// fp16 products; the fp32 matrix cores reach 153 in a plain product). With KS = 2, 2500
// tokens of 6/2 heads: 82.7 us; 97.5 with matrix results in accumulation registers
// (build.py), 84.2 with V's operands read as they are used, 88.2 with the next tile's
// logits formed beside the softmax (too many registers). Two accumulators for the
// logits' main and cross terms instead of one measured the same.
template <int D, int KS>
__global__ __launch_bounds__(256, KS == 1 ? 2 : 1) void attention_f32_kernel(AttentionProblem a, int group, int first_group,
                                                                            const char *__restrict__ planes,
                                                                            const float *__restrict__ scales)
{
    constexpr int ROWS = 128 / KS, C = D / 16, DT = D / 32, KEYS = 32 * KS;
    constexpr int kPlane = KEYS * D * 2;
    constexpr int kLoads = kPlane / (1024 * 4);           // direct loads per wave and plane
    constexpr int kChunks = D / 8, kLoadRows = KEYS / kLoads;
    constexpr int kStage = 4 * kPlane + 512;              // K hi, lo, V hi, lo, scales of K and V
    static_assert(KS == 1 || 2 * kStage >= 4 * kJoinPart<DT>, "the waves' results fit");
    __shared__ __align__(1024) char lds[2 * kStage];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, col = lane & 31;
    const int index = first_group + (int)blockIdx.x, head = index % (int)a.kv_heads;
    SeqTile t;
    if (!find_tile(a.cu, (int)a.seqs, a.m, index / (int)a.kv_heads,
                   [=](int, int n) { return (int)(((int64_t)n * group + ROWS - 1) / ROWS); }, t))
        return;
    const int rows = t.n * group;
    t.tile = (rows + ROWS - 1) / ROWS - 1 - t.tile;
    const int r_wave = t.tile * ROWS + wave / KS * 32;
    const int b0 = KS == 1 ? 0 : wave % KS;               // the wave's 32 keys of a tile

    const int last_row = t.tile * ROWS + ROWS < rows ? t.tile * ROWS + ROWS - 1 : rows - 1;
    const int tiles = last_row / group / KEYS + 1;
    const int wave_masked = ((r_wave < rows ? r_wave : rows - 1) / group + 1) / KEYS;

    const uint32_t base = lds_addr(lds);
    const int load_row = wave * (kLoadRows / 4) + lane / kChunks;
    const int k_chunk = ((lane % kChunks) ^ k_swizzle<D>(load_row)) * 16, v_chunk = ((lane % kChunks) ^ v_swizzle<D>(load_row)) * 16;
    const int64_t plane_rows = a.m * a.kv_heads, first_row = (int64_t)head * a.m + t.begin;
    auto request = [&](int tile) {
        const uint32_t to = base + (tile & 1) * kStage;
        const int left = t.n - 1 - tile * KEYS;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
            const char *from = planes + (is_v * plane_rows + first_row + (int64_t)tile * KEYS) * (D * 4);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = i * kLoadRows + load_row;
                const uint32_t off = (uint32_t)(row < left ? row : left) * (D * 4) + (is_v ? v_chunk : k_chunk);
#pragma unroll
                for (int lo = 0; lo < 2; ++lo) dma16(from + lo * D * 2, off, to + (2 * is_v + lo) * kPlane + (4 * i + wave) * 1024);
            }
        }
        if (wave < 2) {  // scales of K, V: 64 keys (32 of them twice where a tile has no more)
            const int key = lane % KEYS;
            dma4(scales + wave * plane_rows + first_row + (int64_t)tile * KEYS, (uint32_t)(key < left ? key : left) * 4,
                 to + 4 * kPlane + wave * 256);
        }
    };

    request(0);

    int tok;
    float c, large_q;  // what c is not made up of
    v8h qh[C], ql[C];
    {
        int r = r_wave + col;
        r = r < rows ? r : rows - 1;
        tok = r / group;
        const float *src = static_cast<const float *>(a.q) + (t.begin + tok) * a.q_stride + (int64_t)(head * group + r % group) * D + 8 * h;
        float x[C][8];
        float big = 0.0f, lo, up;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            *reinterpret_cast<float4 *>(&x[i][0]) = *reinterpret_cast<const float4 *>(src + 16 * i);
            *reinterpret_cast<float4 *>(&x[i][4]) = *reinterpret_cast<const float4 *>(src + 16 * i + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) big = fmaxf(big, finite_abs(x[i][e]));
        }
        both_halves(big, lo, up);
        const int exponent = row_exponent(fmaxf(lo, up)), most = exponent < kMostQuery ? exponent : kMostQuery;
        large_q = power_of_two(exponent - most);
        c = logit_factor(a.scale * power_of_two(kKeyShift) * power_of_two(most));
        float inv = power_of_two(-exponent);
        if (!(a.scale > 0.0f)) inv = a.scale == 0.0f ? 0.0f : -inv;  // 0: every logit 0, also where q . k overflows
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                _Float16 hi, lo16;
                split_f16(x[i][e] * inv, hi, lo16);
                qh[i][e] = hi;
                ql[i][e] = lo16;
            }
    }
    int k_at[C], v_at[DT];
#pragma unroll
    for (int i = 0; i < C; ++i) k_at[i] = (32 * b0 + col) * (D * 2) + (((2 * i + h) ^ k_swizzle<D>(col)) << 4);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
        const int key = 4 * h + ((lane & 15) >> 2), chunk = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        v_at[d] = (32 * b0 + key) * (D * 2) + ((chunk ^ v_swizzle<D>(key)) << 4) + (lane & 1) * 8;
    }
    auto v_fragment = [&](uint32_t plane, int n, int d) {
        v4s part[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(uintptr_t)(
                plane + v_at[d] + (16 * n + 8 * e) * D * 2));
        return __builtin_bit_cast(v8h, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };

    v16f o[DT];
    float mx = kNegInf, sum = 0.0f, ref_w = 0.0f;  // o is relative to ref_w, which is relative to 2^mx as sum is
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = v16f{};

    const int cut = __any(large_q != 1.0f) ? 0 : wave_masked;
    int aside = 0;  // negative: a tile of V held values that are not finite
    for (int tile = 0; tile < tiles; ++tile) {
        ring_barrier<0>();
        if (tile + 1 < tiles) request(tile + 1);
        const char *stage = lds + (tile & 1) * kStage;
        const uint32_t vt = base + (tile & 1) * kStage + 2 * kPlane;

        v16f s = {};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const v8h kh = *reinterpret_cast<const v8h *>(stage + k_at[i]), kl = *reinterpret_cast<const v8h *>(stage + kPlane + k_at[i]);
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kl, qh[i], s, 0, 0, 0);
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kh, ql[i], s, 0, 0, 0);
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kh, qh[i], s, 0, 0, 0);
        }
        // the operand reads run kAhead pairs ahead of the products
        constexpr int kAhead = 4;
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 2 * kAhead, 0);
#pragma unroll
        for (int i = 0; i < C - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 3, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 3 * kAhead, 0);
        // scales of keys 8g + 4h .. +3
        const float *sc = reinterpret_cast<const float *>(stage + 4 * kPlane) + 32 * b0 + 4 * h;
        aside |= reinterpret_cast<const int *>(stage + 4 * kPlane)[64 + lane];
        float gv[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 k4 = *reinterpret_cast<const float4 *>(sc + 8 * g), v4 = *reinterpret_cast<const float4 *>(sc + 64 + 8 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[4 * g + i] *= (&k4.x)[i];
                gv[4 * g + i] = fabsf((&v4.x)[i]);
            }
        }
        if (tile >= cut) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool seen = tile * KEYS + 32 * b0 + 8 * (i >> 2) + 4 * h + (i & 3) <= tok;
                s[i] = seen ? s[i] * large_q : kNegInf;
                gv[i] = seen ? gv[i] : 0.0f;
            }
        }
        float big = kNegInf, lo, up;
#pragma unroll
        for (int i = 0; i < 16; ++i) big = fmaxf(big, s[i]);
        both_halves(big, lo, up);
        big = fmaxf(lo, up) * c;
        if (__any(big > mx + kSlackF32)) {
            // only where it has grown: a row's result does not depend on its neighbours
            const float now = big > mx + kSlackF32 ? big : mx;
            const float keep = now == mx ? 1.0f : __builtin_amdgcn_exp2f(mx - now);
            mx = now;
            sum *= keep;
            ref_w *= keep;
        }
        const float ref = mx == kNegInf ? 0.0f : mx;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -ref));
            sum += e;
            gv[i] *= e;
            top = fmaxf(top, gv[i]);
        }
        both_halves(top, lo, up);
        top = fmaxf(lo, up);
        if (__any(top > kMostWeight * ref_w)) {
            const float now = top > kMostWeight * ref_w ? top : ref_w;
            const float keep = now == ref_w ? 1.0f : ref_w / now;
            ref_w = now;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= keep;
        }
        const float to_w = ref_w == 0.0f ? 0.0f : kWeightOne / ref_w;  // 0: no key with a weight yet
        v8h ph[2], pl[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            _Float16 hi, lo16;
            const float w = rounded(gv[i] * to_w);
            hi = (_Float16)w;
            lo16 = (_Float16)(w - (float)hi);
            ph[i >> 3][i & 7] = hi;
            pl[i >> 3][i & 7] = lo16;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const v8h vh = v_fragment(vt, n, d), vl = v_fragment(vt + kPlane, n, d);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vl, ph[n], o[d], 0, 0, 0);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vh, pl[n], o[d], 0, 0, 0);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vh, ph[n], o[d], 0, 0, 0);
            }
        // V's operand reads all go ahead of the weights
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 8 * DT, 0);
    }

    const int r = r_wave + col;
    float *dst = static_cast<float *>(a.out) + ((t.begin + tok) * a.q_heads + head * group + r % group) * D + 4 * h;
    const bool any_aside = __any(aside < 0);
    float all = 0.0f, norm = 0.0f;
    auto store = [&](int i, const v4f &v, float inv, float scale) {
        *reinterpret_cast<v4f *>(dst + 32 * (i >> 2) + 8 * (i & 3)) = v4f{v[0] * inv * scale, v[1] * inv * scale, v[2] * inv * scale, v[3] * inv * scale};
        all += (v[0] + v[1]) + (v[2] + v[3]);
        norm = inv;
    };
    if constexpr (KS == 1) {
        float lo, up;
        both_halves(sum, lo, up);
        const float inv = 1.0f / (lo + up);
        if (r < rows)
#pragma unroll
            for (int i = 0; i < 4 * DT; ++i) store(i, o_group(o, i), inv, ref_w / kWeightOne);
    } else {
        join_waves<DT, KS>(lds, o, mx, sum, ref_w / kWeightOne,
                           [&](int i, const v4f &v, float inv, float scale) { if (r < rows) store(i, v, inv, scale); });
    }
    const bool wanted = (any_aside || all - all != 0.0f) && norm - norm == 0.0f && r < rows;
    if (__any(wanted))
        settle(dst, static_cast<const float *>(a.v) + t.begin * a.v_stride + head * D + 4 * h, a.v_stride, tok + 1, wave % KS * (4 * DT / KS), 4 * DT / KS, any_aside, wanted);
}

// Few workgroups: a tile's keys are split over two waves (KS = 2), so that there
// are twice as many and the longest takes half as long. It pays up to 420 workgroups
// in bf16, 340 in fp32 (whose KS = 2 fills a CU's LDS), and half as many again of
// 64-wide heads. One prompt, KS = 1 / 2, 20/5 heads of 128: bf16 1024 tokens 24.2 /
// 19.5 us, 2300 48.6 / 44.0, 2600 (415 workgroups) 56.1 / 54.1, 2900 (460) 63.7 /
// 64.9, 4096 99 / 107; fp32 1300 tokens 74.6 / 56.0, 2048 (325) 116 / 114. 16/4 heads
// of 64: bf16 4096 tokens (516) 62.3 / 53.0, 5000 (629) 80.6 / 80.8, fp32 2500 tokens
// 90.8 / 67.7, 4096 (516) 160 / 154.
static int key_splits(const AttentionProblem &p)
{
    const int64_t groups = (p.m * (p.q_heads / p.kv_heads) / 128 + p.seqs) * p.kv_heads;
    return groups <= (p.bf16 ? 420 : 340) * (p.head_dim == 64 ? 3 : 2) / 2 ? 2 : 1;
}

int64_t attention_workspace(const AttentionProblem &p)
{
    const int64_t rows = p.m * p.kv_heads;
    return p.bf16 ? 0 : round_up(2 * rows * p.head_dim * 4, 256) + round_up(2 * rows * 4, 256);
}

hipError_t launch_attention(const AttentionProblem &p, void *ws, hipStream_t st)
{
    const int group = (int)(p.q_heads / p.kv_heads);
    const int64_t rows = p.m * p.kv_heads;
    char *planes = static_cast<char *>(ws);
    float *scales = p.bf16 ? nullptr : reinterpret_cast<float *>(planes + round_up(2 * rows * p.head_dim * 4, 256));
    auto go = [&](auto width, auto splits) {
        constexpr int D = decltype(width)::value, KS = decltype(splits)::value;
        const int64_t rows_each = 128 / KS;
        if (!p.bf16)
            in_launches(ceil_div(rows * (D / 4), 256), [&](int first, unsigned n) {
                hipLaunchKernelGGL((attention_split_kernel<D>), dim3(n, 2), dim3(256), 0, st, p, planes, scales, first);
            });
        in_launches((p.m * group / rows_each + p.seqs) * p.kv_heads, [&](int first, unsigned n) {
            if (p.bf16) hipLaunchKernelGGL((attention_bf16_kernel<D, KS>), dim3(n), dim3(256), 0, st, p, group, first);
            else hipLaunchKernelGGL((attention_f32_kernel<D, KS>), dim3(n), dim3(256), 0, st, p, group, first, (const char *)planes,
                                    (const float *)scales);
        });
    };
    auto go_width = [&](auto width) {
        key_splits(p) == 1 ? go(width, Width<1>{}) : go(width, Width<2>{});
    };
    if (p.head_dim == 128) go_width(Width<128>{});
    else go_width(Width<64>{});
    return hipGetLastError();
}

}  // namespace bl
