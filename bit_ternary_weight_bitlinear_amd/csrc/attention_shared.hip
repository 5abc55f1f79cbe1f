// attention_shared.hip -- attention of new tokens over a prefix that the whole batch
// shares and over each sequence's own cache behind it.
//
// A softmax over the two together is their results joined by their maxima and sums, so
// the prefix is read once for all sequences: their query rows of a kv head, m * group of
// them, are the rows of one matrix product with it. One launch holds the prefix's
// workgroups (32 rows and a part of the prefix each) and those of the sequences' own pages
// (attention_cached_tile), a second one joins their parts.
//
// With 32 query rows a wave the arithmetic counts, not the bytes, so over the prefix the
// codes meet the queries as fp16, on v_mfma_f32_32x32x16_f16: a code is an integer and exact,
// a row of q times a power of two that puts its largest at 2^14 to 2^15 is exact in fp16 for
// bf16 elements down to 2^-31 of the largest, and in two fp16 parts good to 2^-22 for fp32
// (elements below 2^-17 of the largest: to 2^-39 of that). Weights are relative to a power
// of two at or above their page's and row's largest, times 2^15: rounded to fp16 (2^-11)
// for bf16 results, in two parts (2^-22) for fp32 ones; their sum is that of the rounded
// weights, by a product with ones. Sums are fp32, a page's scaled by its V scale when they are
// added to the row's.
//
// Layout: S^T = K Q^T has a query row per lane and 32 of a page's 64 tokens in its two
// times 16 registers, which after the exponential are the second operand of O^T = V^T P^T
// as they lie: the product's order of tokens is free, so row rho of a K operand is token
//   16 * bit 2 + 8 * bit 4 + 4 * bit 3 + (bits 1, 0) of rho
// of its 32, which gives a lane half h the 16 tokens that one 16-byte piece of V holds. The
// dims of the first product are ordered likewise by 16-byte pieces of K.
//
// What bounds it: a page and 32 rows are 36 matrix instructions (1150 cycles) and about 550
// vector ones (32 of them exponentials, 2600 cycles) in bf16, which take turns rather than
// overlap: 1.85 us a page (16 pages a wave beside 8), 2.4 in fp32. 64 tokens of 32/8 heads behind
// 16384, up to 700 of their own: 40.4 us with the join (with one of their own each 40.8, without
// the prefix 16.9; prefix and own pages in launches one behind the other 52). One workgroup of
// the prefix per CU leaves room for one of own pages, which wait for memory. Not
// kept, beside 31 us for the prefix then: codes as fp16 through LDS for 128 rows, a barrier a page
// (40); 64 rows per wave (35). Codes raised by 128 (K's 2.5 us less in all, V's 0.5), but a
// channel that sets a page's scale would round the logits of the others, and the largest finite
// number in V would turn every dim into an infinity. For bf16 results weights in two
// parts, 49.0 us beside 41.6: the results' rms error against 64 bits is 1.675e-3 of their rms with
// one part, and 1.663e-3 with two, with fp32 weights or by attention_cached.hip's digits, the
// rounding to bf16 being that.
#include "attention_cached.hpp"

namespace bl {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kPrefixRows = 32;

struct PrefixArgs {
    const void *q;
    int64_t q_stride;
    uint32_t rows;  // of a kv head: m * group
    int q_heads, kv_heads, group, splits;
    const int32_t *table, *len;
    int64_t blocks, pages, total_rows;
    const int8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    float scale;  // of the logits, times log2 e
    float *part_o, *part_ml;
};

// Eight codes as fp16: 1024 + (code + 128) is the bits 0x6400 with the biased code in the low byte.
__device__ inline v8h codes_f16(uint32_t lo, uint32_t hi)
{
    union {
        uint32_t w[4];
        v2h h[4];
        v8h v;
    } u;
    constexpr uint32_t kTop = 0x64646464u;
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    u.w[0] = __builtin_amdgcn_perm(kTop, lo, 0x04010400u);
    u.w[1] = __builtin_amdgcn_perm(kTop, lo, 0x04030402u);
    u.w[2] = __builtin_amdgcn_perm(kTop, hi, 0x04010400u);
    u.w[3] = __builtin_amdgcn_perm(kTop, hi, 0x04030402u);
    const v2h bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) u.h[i] += bias;
    return u.v;
}

// the weights of a page's 64 tokens, register r of tile t being token 32 t + 16 half + r
template <int PARTS>
struct Weights {
    v8h hi[2][2], lo[2][2];
};

// Weights from sums s of products (times f: the logits, in powers of two) of the `left` tokens
// that the page holds (none without a page, of whose stand-in nothing may enter). Returns
// their reference exponent.
template <int PARTS>
__device__ inline float page_weights(v16f (&s)[2], float f, int left, int half, Weights<PARTS> &w)
{
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[t][r] *= f;
    if (left < kBlock)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[t][r] = 32 * t + 16 * half + r < left ? s[t][r] : kNegInf;
    float big = kNegInf;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) big = fmaxf(big, s[t][r]);
    big = fmaxf(big, __shfl_xor(big, 32));
    // No weight passes 2^15: below 2^22 the difference to 15 is exact, and a sum with it that rounds
    // rounds to 15 at most. Beyond, where it would not be, the logits lose their reference before
    // (exact near it), and are raised by 15 then.
    const float ref = ceilf(big);
    float shift = ref == kNegInf ? 0.0f : 15.0f - ref;
    const bool far = fabsf(ref) >= 0x1p22f && ref != kNegInf;
    if (__any(far)) {
        asm volatile("");  // a branch, not 32 more differences
        const float less = far ? ref : 0.0f;
        shift = far ? 15.0f : shift;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[t][r] -= less;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float e = __builtin_amdgcn_exp2f(s[t][r] + shift);
            const _Float16 e16 = (_Float16)e;
            w.hi[t][r >> 3][r & 7] = e16;
            if constexpr (PARTS == 2) w.lo[t][r >> 3][r & 7] = (_Float16)(e - (float)e16);
        }
    return ref;
}

// A query row as fp16, row r of an operand of 32: an eighth of it by thread c of eight. Returns
// the row's factor, NaN where it is not finite.
template <typename T, int D, int PARTS>
__device__ inline float query_row(const PrefixArgs &a, uint32_t row, int head, int r, int c, _Float16 *qh)
{
    constexpr int E = D / 8, U = D / 32;
    const bool there = row < a.rows;
    const uint32_t at = there ? row : 0, tok = at / (uint32_t)a.group, hq = head * a.group + (at - tok * a.group);
    const T *src = static_cast<const T *>(a.q) + tok * a.q_stride + (int64_t)hq * D + E * c;
    T raw[E];
#pragma unroll
    for (int i = 0; i < (int)(E * sizeof(T) / 16); ++i) reinterpret_cast<uint4 *>(raw)[i] = reinterpret_cast<const uint4 *>(src)[i];
    float x[E], big = 0.0f, bad = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        x[i] = there ? to_f32(raw[i]) : 0.0f;
        if (!(fabsf(x[i]) <= 3.402823466e38f)) {
            bad = 1.0f;
            x[i] = 0.0f;
        }
        big = fmaxf(big, fabsf(x[i]));
    }
    auto of8 = [](float v, auto f) {
        v = f(v, __int_as_float(dpp_mov<kDppQuadXor1>(__float_as_int(v))));
        v = f(v, __int_as_float(dpp_mov<kDppQuadXor2>(__float_as_int(v))));
        return f(v, __int_as_float(dpp_mov<kDppRowHalfMirror>(__float_as_int(v))));
    };
    big = of8(big, [](float x, float y) { return fmaxf(x, y); });
    bad = of8(bad, [](float x, float y) { return fmaxf(x, y); });
    const int e = 14 - ((int)(__float_as_uint(fmaxf(big, 1e-30f)) >> 23) - 127);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23) * (a.scale < 0.0f ? -1.0f : 1.0f);
#pragma unroll
    for (int g = 0; g < E / 8; ++g) {
        const int piece = c * (E / 8) + g;  // of 8 dims: 32 * pair + 16 * half + 8 * s
        _Float16 *dst = qh + (((piece >> 2) * 2 + (piece & 1)) * 64 + (piece >> 1 & 1) * 32 + r) * 8;
        v8h hi, lo;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = x[8 * g + i] * up;
            hi[i] = (_Float16)v;
            lo[i] = (_Float16)(v - (float)hi[i]);
        }
        *reinterpret_cast<v8h *>(dst) = hi;
        if constexpr (PARTS == 2) *reinterpret_cast<v8h *>(dst + U * 2 * 64 * 8) = lo;
    }
    return bad > 0.0f ? __builtin_nanf("") : __uint_as_float((uint32_t)(127 - e) << 23) * fabsf(a.scale);
}

// A workgroup has 32 query rows of a kv head and part of the prefix, whose pages go to its
// waves in turn.
template <int D, int PARTS>
struct PrefixLds {
    static constexpr int stride = D + 4;                   // of a row in the join
    static constexpr int query = PARTS * (D / 32) * 2 * 64;  // 16-byte pieces of the rows' operands
    static constexpr int join = kPrefixWaves * kPrefixRows * stride * 4;
    static constexpr int bytes = query * 16 > join ? query * 16 : join;
};

template <typename T, int D>
__device__ inline void attention_prefix_tile(const PrefixArgs &a, int64_t tile, int head, int split, char *lds, float *row_scale,
                                             float2 (*jm)[kPrefixRows])
{
    constexpr int W = kPrefixWaves, R = kPrefixRows;
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    constexpr int U = D / 32;  // pairs of 16-dim pieces of K; 32-dim tiles of the output
    constexpr int kStride = PrefixLds<D, PARTS>::stride;
    v8h *qh = reinterpret_cast<v8h *>(lds);  // [part][2 * pair + s][lane], in operand order

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const uint32_t row0 = (uint32_t)tile * R;  // rows are counted in 31 bits
    const int len = *a.len, npages = prefix_pages(a.len, a.blocks);
    const int chunk = prefix_chunk(npages, a.splits);
    const int p0 = split * chunk, p1 = p0 + chunk < npages ? p0 + chunk : npages;
    if (p0 >= npages) return;  // the join knows

    // place of this lane's K row in its 32 tokens, and of its pieces in a page and head
    const int token = 16 * (col >> 2 & 1) + 8 * (col >> 4) + 4 * (col >> 3 & 1) + (col & 3);
    const int k_at = k_code_at<D>(token, 16 * half);
    const int v_at = v_code_at(16 * half, col);
    // ids and scales of 64 of the wave's pages, one per lane
    int page = 0, ok = 0;
    float my_ks = 0.0f, my_vs = 0.0f;
    auto fetch_ids = [&](int base) {
        const int mine = base + W * lane, id = mine < p1 ? a.table[mine] : -1;
        ok = id >= 0 && id < a.pages;
        page = ok ? id : 0;  // a block without a page reads page 0
        const int64_t at = (int64_t)page * a.kv_heads + head;
        my_ks = a.k_scale[at];
        my_vs = a.v_scale[at];
    };
    // K of a page is asked for when the one before has met the queries (the first while they are
    // made ready), V of a page before its K does
    uint4 kf[2][U];
    auto load_k = [&](int i) {
        const int id = __builtin_amdgcn_readlane(page, i);
        const int8_t *kp = a.k_codes + ((int64_t)id * a.kv_heads + head) * (kBlock * D) + k_at;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u) kf[t][u] = *reinterpret_cast<const uint4 *>(kp + t * 8 * 16 + u * 2 * 256);
    };
    if (p0 + wave < p1) {
        fetch_ids(p0 + wave);
        load_k(0);
    }

    {
        const float f = query_row<T, D, PARTS>(a, row0 + (tid >> 3), head, tid >> 3, tid & 7, reinterpret_cast<_Float16 *>(qh));
        if ((tid & 7) == 0) row_scale[tid >> 3] = f;
    }
    __syncthreads();
    const bool poor = !(row_scale[col] == row_scale[col]);
    const float qs = poor ? 0.0f : row_scale[col];
    float top = kNegInf, sum = 0.0f;
    v16f acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[u][i] = 0.0f;

    v8h ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = (_Float16)1.0f;

    for (int base = p0 + wave; base < p1; base += 64 * W) {
        if (base != p0 + wave) {
            fetch_ids(base);
            load_k(0);
        }
        my_ks = ok ? my_ks / 127.0f : 0.0f;  // nothing of page 0 may enter for a missing one
        my_vs = ok ? my_vs / 127.0f : 0.0f;
        for (int p = base, i = 0; p < p1 && i < 64; p += W, ++i) {
            const int id = __builtin_amdgcn_readlane(page, i);
            const int8_t *vp = a.v_codes + ((int64_t)id * a.kv_heads + head) * (kBlock * D) + v_at;
            uint4 vf[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) vf[u][t] = *reinterpret_cast<const uint4 *>(vp + (u * 2 * 4 + t * 2) * 256);
            const bool there = __builtin_amdgcn_readlane(ok, i) != 0;
            const float ks = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_ks), i));
            const float vs = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_vs), i));
            const int left = there ? len - p * kBlock : 0;

            v16f s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
            for (int u = 0; u < U * 2; ++u) {
                const v8h q0 = qh[u * 64 + lane];
                v8h q1;
                if constexpr (PARTS == 2) q1 = qh[(U * 2 + u) * 64 + lane];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint4 c = kf[t][u >> 1];
                    const v8h k8 = u & 1 ? codes_f16(c.z, c.w) : codes_f16(c.x, c.y);
                    if constexpr (PARTS == 2) s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, q1, s[t], 0, 0, 0);
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, q0, s[t], 0, 0, 0);
                }
            }
            if (p + W < p1 && i < 63) load_k(i + 1);

            Weights<PARTS> w;
            const float ref = page_weights<PARTS>(s, qs * ks, left, half, w);
            const float now = fmaxf(top, ref), to = now == kNegInf ? 0.0f : now;
            const float add = __builtin_amdgcn_exp2f(ref - to) * 0x1p-15f, g = add * vs;  // of the page's weights and sums
            if (__any(now != top)) {
                asm volatile("");  // a branch, not 64 products and a choice
                const float keep = __builtin_amdgcn_exp2f(top - to);
                sum *= keep;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[u][r] *= keep;
            }
            top = now;
            auto product = [&](const v8h &c, int t, int b, v16f o) {
                if constexpr (PARTS == 2) o = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, w.lo[t][b], o, 0, 0, 0);
                return __builtin_amdgcn_mfma_f32_32x32x16_f16(c, w.hi[t][b], o, 0, 0, 0);
            };
            // the weights' sum as they are after rounding: every register the same
            v16f all;
#pragma unroll
            for (int r = 0; r < 16; ++r) all[r] = 0.0f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int b = 0; b < 2; ++b) all = product(ones, t, b, all);
            sum = __builtin_fmaf(all[0], add, sum);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v16f o;
#pragma unroll
                for (int r = 0; r < 16; ++r) o[r] = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        o = product(b ? codes_f16(vf[u][t].z, vf[u][t].w) : codes_f16(vf[u][t].x, vf[u][t].y), t, b, o);
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[u][r] = __builtin_fmaf(o[r], g, acc[u][r]);
            }
        }
    }

    // ---- join the waves, in wave order
    __syncthreads();
    float *jo = reinterpret_cast<float *>(lds);  // [wave][row][kStride]
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            v4f o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = acc[u][r + i];
            *reinterpret_cast<v4f *>(jo + (wave * R + col) * kStride + 32 * u + 2 * r + 4 * half) = o;
        }
    if (half == 0) jm[wave][col] = make_float2(top, poor ? __builtin_nanf("") : sum);
    __syncthreads();
    for (int it = tid; it < R * (D / 4); it += 64 * W) {
        const int r = it / (D / 4), dim = it % (D / 4) * 4;
        if (row0 + r >= a.rows) break;
        float best = kNegInf;
#pragma unroll
        for (int w = 0; w < W; ++w) best = fmaxf(best, jm[w][r].x);
        const float to = best == kNegInf ? 0.0f : best;
        v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = __builtin_amdgcn_exp2f(jm[w][r].x - to);
            const v4f v = *reinterpret_cast<const v4f *>(jo + (w * R + r) * kStride + dim);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(f, v[i], o[i]);
            l = __builtin_fmaf(f, jm[w][r].y, l);
        }
        const uint32_t tok = (row0 + r) / (uint32_t)a.group;
        const int64_t row = (int64_t)tok * a.q_heads + head * a.group + (row0 + r - tok * a.group);
        *reinterpret_cast<v4f *>(a.part_o + ((int64_t)split * a.total_rows + row) * D + dim) = o;
        if (dim == 0) reinterpret_cast<float2 *>(a.part_ml)[(int64_t)split * a.total_rows + row] = make_float2(best, l);
    }
}

// a / b of workgroup numbers, which rarely need 64 bits
__device__ inline int64_t over(int64_t a, int b) { return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b); }

// The prefix's workgroups first, which take longest, then the sequences' own pages: the one
// waits for arithmetic, the other for memory.
template <typename T, int D, int RT>
__global__ __launch_bounds__(64 * kPrefixWaves, 2) void attention_shared_kernel(PrefixArgs f, CachedArgs a, int64_t prefix_groups, int64_t first)
{
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    constexpr int kOwnBytes = CachedLds<D, RT, kPrefixWaves>::words * 4, kPrefixBytes = PrefixLds<D, PARTS>::bytes;
    __shared__ __align__(16) char lds[kPrefixBytes > kOwnBytes ? kPrefixBytes : kOwnBytes];
    __shared__ float row_scale[kPrefixRows];
    __shared__ float2 jm[kPrefixWaves][kPrefixRows];
    int64_t group = first + blockIdx.x;
    if (group < prefix_groups) {
        const int64_t unit = over(group, f.splits), tile = over(unit, f.kv_heads);
        attention_prefix_tile<T, D>(f, tile, (int)(unit - tile * f.kv_heads), (int)(group - unit * f.splits), lds, row_scale, jm);
        return;
    }
    group -= prefix_groups;
    const int64_t unit = over(group, a.splits), tile = over(unit, a.kv_heads);
    attention_cached_tile<T, D, RT, kPrefixWaves, false, kBehindPrefix>(a, (int)tile, (int)(unit - tile * a.kv_heads), (int)(group - unit * a.splits),
                                                                       reinterpret_cast<uint32_t *>(lds), row_scale);
}

// ---------------------------------------------------------------- launcher

// Workgroups per unit, a tile of rows and a kv head: of the prefix, and of the sequences' own
// pages, about `target` in all and with a page per wave at least
static int64_t splits_of(int64_t units, int64_t blocks, int64_t target)
{
    const int64_t most = ceil_div(blocks, kPrefixWaves), s = target / units < most ? target / units : most;
    return s < 1 ? 1 : s > 256 ? 256 : s;
}
// About one per CU. With targets of 128, 256 and 512: 64 rows of 32/8 heads behind 16384 tokens
// 63.4, 42.8 and 49.5 us in bf16, 77.5, 53.8 and 58.8 in fp32; 12 x 4 of 20/5 behind 6001, fp32
// 25.4, 23.2 and 30.5; 16 of 32/8 behind 32768 38.2, 29.6 and 35.0. Hundreds of rows per
// sequence leave no splits (8 x 64 of 32/8 behind 8000, bf16: 147 us with any)
static int64_t prefix_splits(const SharedProblem &p)
{
    return splits_of(ceil_div(p.c.m * (p.c.q_heads / p.c.kv_heads), kPrefixRows) * p.c.kv_heads, p.prefix_blocks, 256);
}
// About one per CU: beside a workgroup of the prefix there is room for one. With targets of 128, 256
// and 512: 64 rows of 32/8 heads behind 16384, up to 700 of their own, 42.4, 42.5 and 42.5 us; 12 x 4 of
// 20/5 behind 6001 20.4, 20.4 and 21.9 in fp32, 19.7, 19.6 and 21.8 in bf16; 16 of 32/8 behind 32768, 1500
// own, 32.7, 31.0 and 31.4; 4 behind 8000, 8000 own, 19.1, 18.6 and 20.8; 20 x 2 behind 3000, 1000
// own, 21.9, 21.8 and 25.5; 48 of 12/4 heads of 64 behind 5000 13.0, 13.1 and 15.2
static int64_t own_splits(const CachedProblem &c)
{
    return splits_of(units_of(c, row_tiles(c)), c.max_blocks, 256);
}

struct SharedLayout {
    int64_t part_ml, own_o, own_ml, bytes;
};
static SharedLayout shared_layout(const SharedProblem &p)
{
    const int64_t rows = p.c.m * p.c.q_heads, before = prefix_splits(p) * rows, own = own_splits(p.c) * rows;
    SharedLayout L{};
    L.part_ml = round_up(before * p.c.head_dim * 4, 256);
    L.own_o = L.part_ml + round_up(before * 8, 256);
    L.own_ml = L.own_o + round_up(own * p.c.head_dim * 4, 256);
    L.bytes = L.own_ml + round_up(own * 8, 256);
    return L;
}

int64_t attention_shared_workspace(const SharedProblem &p) { return shared_layout(p).bytes; }

hipError_t launch_attention_shared(const SharedProblem &p, void *ws, hipStream_t st)
{
    const CachedProblem &c = p.c;
    const int rt = row_tiles(c);
    const SharedLayout L = shared_layout(p);
    char *base = static_cast<char *>(ws);
    PrefixArgs f{};
    f.q = c.q; f.q_stride = c.q_stride; f.group = (int)(c.q_heads / c.kv_heads); f.rows = (uint32_t)(c.m * f.group);
    f.q_heads = (int)c.q_heads; f.kv_heads = (int)c.kv_heads; f.splits = (int)prefix_splits(p);
    f.table = p.prefix_table; f.len = p.prefix_len; f.blocks = p.prefix_blocks; f.pages = c.pages; f.total_rows = c.m * c.q_heads;
    f.k_codes = c.k_codes; f.v_codes = c.v_codes; f.k_scale = c.k_scale; f.v_scale = c.v_scale; f.scale = c.scale * kLog2e;
    f.part_o = reinterpret_cast<float *>(base);
    f.part_ml = reinterpret_cast<float *>(base + L.part_ml);
    CachedArgs a = cached_args(c, Shape{kPrefixWaves, own_splits(c)}, rt);
    a.prefix_o = f.part_o; a.prefix_ml = f.part_ml; a.prefix_len = p.prefix_len; a.prefix_blocks = p.prefix_blocks;
    a.prefix_splits = f.splits;
    a.part_o = reinterpret_cast<float *>(base + L.own_o);
    a.part_ml = reinterpret_cast<float *>(base + L.own_ml);
    const int64_t prefix_groups = ceil_div(f.rows, kPrefixRows) * c.kv_heads * f.splits;
    const int64_t groups = prefix_groups + query_tiles(c, rt) * c.kv_heads * a.splits;
    auto go = [&](auto type, auto width) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value;
        for (int64_t first = 0; first < groups; first += kMostGroups) {
            const dim3 grid((unsigned)(groups - first < kMostGroups ? groups - first : kMostGroups)), threads(64 * kPrefixWaves);
            if (rt == 1) hipLaunchKernelGGL((attention_shared_kernel<T, D, 1>), grid, threads, 0, st, f, a, prefix_groups, first);
            else if (rt == 2) hipLaunchKernelGGL((attention_shared_kernel<T, D, 2>), grid, threads, 0, st, f, a, prefix_groups, first);
            else hipLaunchKernelGGL((attention_shared_kernel<T, D, 4>), grid, threads, 0, st, f, a, prefix_groups, first);
        }
        launch_join<kBehindPrefix, T, D>(c, a, a.splits + f.splits, st);
    };
    if (c.bf16) c.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
    else c.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    return hipGetLastError();
}

}  // namespace bl
