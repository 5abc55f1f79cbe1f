// attention_cached.hpp -- the kernels of attention over the 8-bit cache: of new tokens
// over a whole cache (attention_cached.hip), over the blocks that a list names for
// each row and kv head (attention_selected.hip), and over a sequence's own cache behind
// a prefix that the batch shares (attention_shared.hip).
#pragma once

#include "attention.hpp"

namespace bl {

// What the kernels of this file walk over: a sequence's whole table; the blocks listed
// for one row (kSelectedPast: read past the caches); the whole table, to be joined with the
// results of a shared prefix.
enum CachedMode { kWhole, kSelected, kSelectedPast, kBehindPrefix };
constexpr bool listed(CachedMode m) { return m == kSelected || m == kSelectedPast; }

constexpr float kDigitMax = 8355711.0f;  // 0x7F7F7F: every digit within -128..127

// Signed base-256 digits: with 0x80 added to each, the bytes of n + 0x808080. For
// |x * scale| <= kDigitMax the fp32 sum x * scale + 0x808080 is at least 2^23, where
// fp32 holds integers only, or (for x * scale < -32896) is cut to one by the
// conversion: one fma and one conversion per value, off by less than 1 where x * scale
// is below -32896 and by at most a half elsewhere. For q the factor to its largest rounds
// by up to 0.5 and the product with it by 0.25 besides: less than 1.75 of 8355711.
__device__ inline uint32_t biased_digits(float x, float scale)
{
    return (uint32_t)__builtin_fmaf(x, scale, 8421504.0f);
}
// digit k of four values, one per byte
template <int K>
__device__ inline uint32_t digit_bytes(const uint32_t n[4])
{
    const uint32_t lo = __builtin_amdgcn_perm(n[1], n[0], 0x0C0C0400u + 0x0101u * K);
    const uint32_t hi = __builtin_amdgcn_perm(n[3], n[2], 0x04000C0Cu + 0x01010000u * K);
    return (lo | hi) ^ 0x80808080u;
}

// digits' sums to one fp32 value; the lower two meet exactly (|c1| <= 2^21)
__device__ inline float join_digits(v4i c)
{
    return __builtin_fmaf((float)c[2], 65536.0f, (float)(c[0] + (c[1] << 8)));
}

// How the pages of a sequence are split: in pages per workgroup. At least one for
// each of its waves, and at most `splits` workgroups.
__device__ inline int pages_per_split(int npages, int splits, int waves)
{
    const int c = (npages + splits - 1) / splits;
    return c < waves ? waves : c;
}

__device__ inline int pages_of(int64_t have, int n, int64_t max_blocks)
{
    const int64_t np = (have + n + kBlock - 1) / kBlock;
    return (int)(np < max_blocks ? np : max_blocks);
}

struct CachedArgs {
    const void *q;
    int64_t q_stride, m;
    const int32_t *cu, *lens, *table;
    int seqs, q_heads, kv_heads, group, splits, waves, tiles_per_seq;
    int64_t max_blocks, pages;
    const int8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    float scale;      // of the logits, times log2 e
    void *out;
    float *part_o;    // [splits][m * q_heads][D]
    float *part_ml;   // [splits][m * q_heads][2]: reference exponent, sum
    float *stat;      // [m * q_heads][max_blocks][2]: a page's largest exponent, sum
    float *final_ml;  // [m * q_heads][2]: a row's reference exponent, 1 / sum (0: adds no weight)
    // listed: [m][kv_heads][keep] blocks
    const int32_t *selected;
    int64_t keep;
    // kBehindPrefix: the prefix's parts, laid out as part_o and part_ml, and what gives their number
    const float *prefix_o, *prefix_ml;
    const int32_t *prefix_len;
    int64_t prefix_blocks;
    int prefix_splits;
};

__device__ inline int parts_of(int npages, int splits, int waves)
{
    const int chunk = pages_per_split(npages, splits, waves);
    return npages <= chunk ? 1 : (npages + chunk - 1) / chunk;
}

// A prefix's pages, those of a workgroup (whole rounds of its waves: a part less to write and
// to join costs no time), and the parts that its results come in (none for an empty one)
constexpr int kPrefixWaves = 4;
__device__ inline int prefix_chunk(int npages, int splits)
{
    return (pages_per_split(npages, splits, kPrefixWaves) + kPrefixWaves - 1) / kPrefixWaves * kPrefixWaves;
}
__device__ inline int prefix_pages(const int32_t *len, int64_t blocks) { return *len <= 0 ? 0 : pages_of(*len, 0, blocks); }
__device__ inline int prefix_parts(const CachedArgs &a)
{
    const int np = prefix_pages(a.prefix_len, a.prefix_blocks), chunk = prefix_chunk(np, a.prefix_splits);
    return (np + chunk - 1) / chunk;
}

// tiles of 4*RT query rows: row r of a sequence is token r / group, head r % group.
// Listed: a token's tiles hold no rows of the next one, whose blocks are others; t is
// that token alone, `tok` its place in the sequence
template <int RT, CachedMode MODE>
__device__ inline bool find_rows(const CachedArgs &a, int idx, SeqTile &t, int &tok)
{
    tok = 0;
    if (listed(MODE) && a.cu) {
        t.begin = idx / a.tiles_per_seq;
        t.tile = idx % a.tiles_per_seq;
        t.n = 1;
        int have;
        return find_row(a.cu, a.lens, a.seqs, a.m, t.begin, t.seq, tok, have) && have >= 0;
    }
    if (!a.cu) {
        t.seq = idx / a.tiles_per_seq;
        t.tile = idx % a.tiles_per_seq;
        t.begin = t.seq;
        t.n = 1;
        return t.seq < a.seqs && a.lens[t.seq] >= 0;
    }
    const int group = a.group;
    const int32_t *lens = a.lens;
    return find_tile(a.cu, a.seqs, a.m, idx, [=](int s, int n) {
        return lens[s] < 0 ? 0 : (int)(((int64_t)n * group + 4 * RT - 1) / (4 * RT));
    }, t);
}

// what a row adds to the blocks' weights: nothing if it sees nothing or is not finite
__device__ inline float2 final_of(float top, float l) { return make_float2(top, l > 0.0f ? 1.0f / l : 0.0f); }

template <CachedMode MODE>
__device__ inline v4i codes_at(const uint4 *p)
{
    if constexpr (MODE == kSelectedPast) return __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p));
    else return *reinterpret_cast<const v4i *>(p);
}

// words of LDS that a workgroup of attention_cached_tile needs: digits of q in operand
// order, [row tile][step][lane][16 bytes]; per wave the digits of p, [16 rows][16 dwords of
// 4 tokens]; at the end the waves' results
template <int D, int RT, int W>
struct CachedLds {
    static constexpr int query = RT * (D / 64) * 256, digits = W * 256, join = W * 4 * RT * (D + 2);
    static constexpr int words = query + digits > join ? query + digits : join;
};

// One workgroup's work: split `split` of tile idx of kv head `head`. row_scale: 4 * RT floats of LDS
template <typename T, int D, int RT, int W, bool STAT, CachedMode MODE>
__device__ inline void attention_cached_tile(const CachedArgs &a, int idx, int head, int split, uint32_t *lds, float *row_scale)
{
    constexpr int H = D / 64;   // matrix steps over the head width
    constexpr int N = D / 16;   // 16-dim tiles of the output
    constexpr int R = 4 * RT;   // query rows
    constexpr int E = D / 16;   // elements of a query row per thread
    constexpr int kQueryWords = CachedLds<D, RT, W>::query;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane >> 4, c = lane & 15;
    SeqTile t;
    int at_tok;
    if (!find_rows<RT, MODE>(a, idx, t, at_tok)) return;
    const int32_t *table = a.table + (int64_t)t.seq * a.max_blocks;
    const int32_t *chosen = listed(MODE) ? a.selected + (t.begin * a.kv_heads + head) * a.keep : nullptr;
    // one split: the wave's pages do not depend on the length, which is on its way
    int ids = -1, blocks = 0;  // listed: which block of the sequence a page is
    if (!listed(MODE) && a.splits == 1 && wave + W * lane < a.max_blocks) ids = table[wave + W * lane];
    const int64_t have = a.lens[t.seq] + (int64_t)at_tok;
    const int npages = listed(MODE) ? (int)a.keep : pages_of(have, t.n, a.max_blocks);
    const int chunk = pages_per_split(npages, a.splits, W);
    const int p0 = split * chunk, p1 = p0 + chunk < npages ? p0 + chunk : npages;
    if (p0 >= npages && split > 0) return;  // the join knows; split 0 writes rows that see nothing
    // row r of the tile is query `head * group + h` of the sequence's row `tok`
    const int64_t first = (int64_t)t.tile * R, left = (int64_t)t.n * a.group - first;
    const int rows = left < R ? (int)left : R;
    const int tok0 = (int)(first / a.group);
    const uint32_t rem0 = (uint32_t)(first - (int64_t)tok0 * a.group), group = (uint32_t)a.group;
    auto place = [&](int r, int &tok, int &hq) {
        const uint32_t u = rem0 + (uint32_t)r, q = u / group;
        tok = tok0 + (int)q;
        hq = head * a.group + (int)(u - q * group);
    };

    // ---- the wave's pages: ids and scales of 64 of them, one per lane
    float my_ks = 0.0f, my_vs = 0.0f;
    auto fetch_ids = [&](int base) {
        const int mine = base + W * lane;
        if constexpr (listed(MODE)) {
            blocks = mine < p1 ? chosen[mine] : -1;
            // entries that name no block, or one behind the row, hold nothing that it sees
            const bool sees = blocks >= 0 && blocks < a.max_blocks && (int64_t)blocks * kBlock <= have;
            ids = sees ? table[blocks] : -1;
        } else if (a.splits > 1 || base != wave) ids = mine < p1 ? table[mine] : -1;
        const bool ok = mine < p1 && ids >= 0 && ids < a.pages;
        const int64_t my_at = ok ? (int64_t)ids * a.kv_heads + head : 0;
        // a block without a page reads page 0, of which nothing may enter
        my_ks = ok ? a.k_scale[my_at] : 0.0f;
        my_vs = ok ? a.v_scale[my_at] : 0.0f;
    };
    auto page_at = [&](int i, bool &there) {
        const int id = __builtin_amdgcn_readlane(ids, i);
        there = id >= 0 && id < a.pages;
        return ((int64_t)(there ? id : 0) * a.kv_heads + head) * (kBlock * D);
    };
    v4i kf[4][H];
    auto load_k = [&](int i) {
        bool there;
        const uint4 *kp = reinterpret_cast<const uint4 *>(a.k_codes + page_at(i, there)) + lane;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int h = 0; h < H; ++h) kf[tt][h] = codes_at<MODE>(kp + (tt * H + h) * 64);
    };
    // K of a page is asked for as soon as the one before has been used, the first while
    // the query rows are made ready (one token over 1024, 20/5 heads: 6.3 us beside 6.7);
    // 16 rows leave no registers for it
    constexpr bool EARLY = RT < 4;
    int base = p0 + wave;
    if (EARLY && base < p1) {
        fetch_ids(base);
        load_k(0);
    }

    // ---- query rows as digits, 16 lanes per row
    for (int r = tid >> 4; r < R; r += 4 * W) {
        const bool there = r < rows;
        int tok, hq;
        place(there ? r : 0, tok, hq);
        const T *src = static_cast<const T *>(a.q) + (t.begin + tok) * a.q_stride + (int64_t)hq * D + E * c;
        T raw[E];
        if constexpr (E * sizeof(T) == 8) *reinterpret_cast<uint2 *>(raw) = *reinterpret_cast<const uint2 *>(src);
        else
#pragma unroll
            for (int i = 0; i < (int)(E * sizeof(T) / 16); ++i)
                reinterpret_cast<uint4 *>(raw)[i] = reinterpret_cast<const uint4 *>(src)[i];
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
        big = fmaxf(row16_max(big), 1e-30f);
        bad = row16_max(bad);
        const float inv = kDigitMax / big;
        uint32_t w[3][E / 4];
#pragma unroll
        for (int g = 0; g < E / 4; ++g) {
            uint32_t n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = biased_digits(fminf(fmaxf(x[4 * g + i] * inv, -kDigitMax), kDigitMax), 1.0f);
            w[0][g] = digit_bytes<0>(n);
            w[1][g] = digit_bytes<1>(n);
            w[2][g] = digit_bytes<2>(n);
        }
        // operand lane of (row, digit k, dim): 16 * (dim % 64 / 16) + 4 * (r % 4) + k of step dim / 64
        const int dim = E * c;
        uint32_t *dst = lds + (((r >> 2) * H + dim / 64) * 64 + (dim % 64 / 16) * 16 + (r & 3) * 4) * 4 + dim % 16 / 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int g = 0; g < E / 4; ++g) dst[k * 4 + g] = k < 3 ? w[k < 3 ? k : 0][g] : 0u;
        if (c == 0) row_scale[r] = bad > 0.0f ? __builtin_nanf("") : (big / kDigitMax) * a.scale;
    }
    uint32_t *dig = lds + kQueryWords + wave * 256;
#pragma unroll
    for (int i = 0; i < 4; ++i) dig[i * 64 + lane] = 0;  // rows 4j+3 stay 0
    __syncthreads();
    float qs[RT];          // scale of query row j of each tile
    int limit[RT];         // last token that it sees (-1: none; tokens past the table are in no page)
    bool poor[RT];         // it is not finite
    float2 *stat[RT];      // its blocks' largest exponents and sums
    v4i qd[RT][H];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const bool there = 4 * rt + j < rows;
        int tok, hq;
        place(there ? 4 * rt + j : 0, tok, hq);
        const int64_t last = have + tok;
        limit[rt] = !there ? -1 : last < 0x7FFFFFFF ? (int)last : 0x7FFFFFFF;
        if (STAT) stat[rt] = there ? reinterpret_cast<float2 *>(a.stat) + ((t.begin + tok) * a.q_heads + hq) * a.max_blocks : nullptr;
        qs[rt] = row_scale[4 * rt + j];
        poor[rt] = !(qs[rt] == qs[rt]);
        if (poor[rt]) qs[rt] = 0.0f;
        if constexpr (RT == 1)
#pragma unroll
            for (int h = 0; h < H; ++h) qd[rt][h] = *reinterpret_cast<const v4i *>(lds + (h * 64 + lane) * 4);
    }

    float mx[RT], sum[RT], acc[RT][N];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        mx[rt] = kNegInf;
        sum[rt] = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[rt][n] = 0.0f;
    }

    for (; base < p1; base += 64 * W) {
        if (!EARLY || base != p0 + wave) {
            fetch_ids(base);
            if (EARLY) load_k(0);
        }
        for (int p = base, i = 0; p < p1 && i < 64; p += W, ++i) {
            bool there;
            const uint4 *vp = reinterpret_cast<const uint4 *>(a.v_codes + page_at(i, there)) + lane;
            if (listed(MODE) && !there) {
                if (EARLY && p + W < p1 && i < 63) load_k(i + 1);
                continue;
            }
            const int block = listed(MODE) ? __builtin_amdgcn_readlane(blocks, i) : p;
            if (!EARLY) load_k(i);
            v4i vf[N];
#pragma unroll
            for (int n = 0; n < N; ++n) vf[n] = codes_at<MODE>(vp + n * 64);
            const float ks = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_ks), i)) / 127.0f;
            const float vs = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_vs), i)) / 127.0f;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if constexpr (RT > 1)
#pragma unroll
                    for (int h = 0; h < H; ++h) qd[rt][h] = *reinterpret_cast<const v4i *>(lds + ((rt * H + h) * 64 + lane) * 4);
                float x[4];
                float big = kNegInf;
                const float f = qs[rt] * ks;
                const int last = there ? limit[rt] - block * kBlock : -1;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    v4i s = {0, 0, 0, 0};
#pragma unroll
                    for (int h = 0; h < H; ++h) s = __builtin_amdgcn_mfma_i32_16x16x64_i8(qd[rt][h], kf[tt][h], s, 0, 0, 0);
                    const bool seen = 4 * c + tt <= last;
                    x[tt] = seen ? join_digits(s) * f : kNegInf;
                    big = fmaxf(big, x[tt]);
                }
                if (EARLY && rt == RT - 1 && p + W < p1 && i < 63) load_k(i + 1);  // the next page's
                big = row16_max(big);
                const float ref = big == kNegInf ? 0.0f : big;
                float total = 0.0f;
                uint32_t n4[4];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    const float e = __builtin_amdgcn_exp2f(x[tt] - ref);
                    total += e;
                    n4[tt] = biased_digits(e, kDigitMax);
                }
                total = row16_sum(total);
                dig[4 * j * 16 + c] = digit_bytes<0>(n4);
                dig[(4 * j + 1) * 16 + c] = digit_bytes<1>(n4);
                dig[(4 * j + 2) * 16 + c] = digit_bytes<2>(n4);
                // the lanes of a wave exchange through LDS, which serves them in order
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                const v4i pd = *reinterpret_cast<const v4i *>(&dig[c * 16 + 4 * j]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (STAT && c == 0 && stat[rt]) stat[rt][p] = make_float2(big, total);
                const float now = fmaxf(mx[rt], big);
                const float to = now == kNegInf ? 0.0f : now;
                const float keep = __builtin_amdgcn_exp2f(mx[rt] - to), add = __builtin_amdgcn_exp2f(big - to);
                mx[rt] = now;
                sum[rt] = __builtin_fmaf(sum[rt], keep, total * add);
                const float g = add * vs * (1.0f / kDigitMax);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const v4i o = __builtin_amdgcn_mfma_i32_16x16x64_i8(pd, vf[n], v4i{0, 0, 0, 0}, 0, 0, 0);
                    acc[rt][n] = __builtin_fmaf(acc[rt][n], keep, join_digits(o) * g);
                }
            }
        }
    }

    // ---- join the waves, in wave order
    __syncthreads();
    float *jo = reinterpret_cast<float *>(lds);              // [wave][row][D]
    float *jm = jo + W * R * D;                              // [wave][row][2]
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = wave * R + 4 * rt + j;
#pragma unroll
        for (int n = 0; n < N; ++n) jo[r * D + 16 * n + c] = acc[rt][n];
        if (c == 0) {
            jm[2 * r] = mx[rt];
            jm[2 * r + 1] = poor[rt] ? __builtin_nanf("") : sum[rt];
        }
    }
    __syncthreads();
    const int64_t total_rows = a.m * a.q_heads;
    for (int it = tid; it < R * D; it += 64 * W) {
        const int r = it / D, dim = it % D;
        if (r >= rows) break;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, jm[2 * (w * R + r)]);
        const float to = top == kNegInf ? 0.0f : top;
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = __builtin_amdgcn_exp2f(jm[2 * (w * R + r)] - to);
            o = __builtin_fmaf(f, jo[(w * R + r) * D + dim], o);
            l = __builtin_fmaf(f, jm[2 * (w * R + r) + 1], l);
        }
        int tok, hq;
        place(r, tok, hq);
        const int64_t row = (t.begin + tok) * a.q_heads + hq;
        if (a.splits > 1 || MODE == kBehindPrefix) {
            a.part_o[((int64_t)split * total_rows + row) * D + dim] = o;
            if (dim == 0) reinterpret_cast<float2 *>(a.part_ml)[(int64_t)split * total_rows + row] = make_float2(top, l);
        } else {
            store_out(static_cast<T *>(a.out) + row * D + dim, l == 0.0f ? 0.0f : o / l);
            if (STAT && dim == 0) reinterpret_cast<float2 *>(a.final_ml)[row] = final_of(top, l);
        }
    }
}

template <typename T, int D, int RT, int W, bool STAT, CachedMode MODE = kWhole>
__global__ __launch_bounds__(64 * W, RT == 1 ? 4 : 2) void attention_cached_kernel(CachedArgs a, int first_tile)
{
    __shared__ __align__(16) uint32_t lds[CachedLds<D, RT, W>::words];
    __shared__ float row_scale[4 * RT];
    attention_cached_tile<T, D, RT, W, STAT, MODE>(a, first_tile + (int)blockIdx.z, blockIdx.y, blockIdx.x, lds, row_scale);
}

// Adds the attention weight of 64 blocks of a sequence, a block per lane and the
// rows over the waves; their sums meet in LDS, in a fixed order. PARTS: the rows'
// final exponents and sums are joined from the splits here (a few hundred values),
// in the launch that joins their results, rather than in another one behind it.
template <int W, bool PARTS>
__device__ inline void add_weights(const CachedArgs &a, int s, int chunk64, float *weights, float2 *fin, float *part)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t begin;
    int n;
    seq_rows(a.cu, s, a.m, begin, n);
    const int64_t have = a.lens[s];
    if (have < 0 || n == 0) return;
    const int npages = pages_of(have, n, a.max_blocks), p = chunk64 * 64 + lane;
    if (chunk64 * 64 >= npages) return;
    const int chunk = pages_per_split(npages, a.splits, a.waves);
    const int parts = npages <= chunk ? 1 : (npages + chunk - 1) / chunk;
    const int64_t row0 = begin * a.q_heads, rows = (int64_t)n * a.q_heads, total_rows = a.m * a.q_heads;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml), *stat = reinterpret_cast<const float2 *>(a.stat);
    float w = 0.0f;
    // a thread adds kRows rows per round; LANES lanes join a row's splits
    auto add = [&](auto lanes) {
        constexpr int LANES = decltype(lanes)::value, kRows = 64 / LANES;
        for (int64_t r0 = 0; r0 < rows; r0 += kRows * W) {
            float2 st[kRows];  // asked for before the rows' exponents and sums
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = r0 + wave + W * i;
                st[i] = r < rows && p < npages ? stat[(row0 + r) * a.max_blocks + p] : make_float2(0.0f, 0.0f);
            }
            if constexpr (PARTS) {
                const int64_t r = r0 + tid / LANES;
                float mx = kNegInf, l = 0.0f;
                if (r < rows)
                    for (int i = tid % LANES; i < parts; i += LANES) {
                        const float2 v = ml[i * total_rows + row0 + r];
                        const float now = fmaxf(mx, v.x), to = now == kNegInf ? 0.0f : now;
                        l = __builtin_fmaf(l, __builtin_amdgcn_exp2f(mx - to), v.y * __builtin_amdgcn_exp2f(v.x - to));
                        mx = now;
                    }
                float top = mx;
#pragma unroll
                for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
                l *= __builtin_amdgcn_exp2f(mx - (top == kNegInf ? 0.0f : top));
#pragma unroll
                for (int d = 1; d < LANES; d <<= 1) l += __shfl_xor(l, d);
                __syncthreads();
                if (tid % LANES == 0) fin[tid / LANES] = final_of(top, l);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = r0 + wave + W * i;
                if (r >= rows) continue;
                const float2 f = PARTS ? fin[wave + W * i] : reinterpret_cast<const float2 *>(a.final_ml)[row0 + r];
                const float share = st[i].y * f.y * __builtin_amdgcn_exp2f(st[i].x - f.x);
                w += f.y > 0.0f && st[i].y > 0.0f ? share : 0.0f;
            }
        }
    };
    if (rows > 4 * W) add(Width<4>{});
    else add(Width<16>{});
    part[tid] = w;
    __syncthreads();
    if (wave || p >= npages) return;
#pragma unroll
    for (int i = 1; i < W; ++i) w += part[i * 64 + lane];
    weights[(int64_t)s * a.max_blocks + p] += w;
}

// Joins the splits. Up to kFewSplits, a thread per dim of a row does by itself, all its
// loads independent; otherwise one workgroup per query row: the splits' sums become
// factors in LDS, then every thread adds one dim of every fourth split (or eighth, of
// 64 dims). The workgroups behind those add the blocks' weights. 12 sequences of four
// tokens and 8 splits, 20 heads: 4.1 us beside 6.1 with a workgroup per row.
constexpr int kFewSplits = 16;

template <typename T, int D, bool FEW, CachedMode MODE = kWhole>
__global__ __launch_bounds__(512) void attention_join_kernel(CachedArgs a, float *__restrict__ weights, int blocks64, int64_t first)
{
    constexpr int G = 512 / D;
    __shared__ float factor[512], jo[512];
    __shared__ float red[2][8];
    __shared__ float2 fin[128];
    const int tid = threadIdx.x, wave = tid >> 6, dim = tid % D;
    const int64_t total_rows = a.m * a.q_heads, groups = FEW ? (total_rows + G - 1) / G : total_rows;
    const int64_t group = first + blockIdx.x;
    if (group >= groups) {
        const int w = (int)(group - groups);
        add_weights<8, true>(a, w / blocks64, w % blocks64, weights, fin, jo);
        return;
    }
    const int64_t row = FEW ? group * G + tid / D : group;
    if (row >= total_rows) return;
    SeqTile t;
    const int tok = (int)(row / a.q_heads);
    if (!a.cu) {
        t.seq = tok;
        t.n = 1;
    } else {
        const int first = a.cu[0] < 0 ? 0 : a.cu[0];
        if (!find_tile(a.cu, a.seqs, a.m, tok - first, [](int, int n) { return n; }, t)) return;
        if (t.begin + t.tile != tok) return;
    }
    const int64_t have = a.lens[t.seq];
    if (have < 0) return;
    const int own = parts_of(listed(MODE) ? (int)a.keep : pages_of(have, t.n, a.max_blocks), a.splits, a.waves);
    const int parts = MODE == kBehindPrefix ? own + prefix_parts(a) : own;
    const float2 *own_ml = reinterpret_cast<const float2 *>(a.part_ml) + row;
    const float *own_o = a.part_o + row * D + dim;
    auto ml_of = [&](int s) {
        if (MODE == kBehindPrefix && s >= own) return reinterpret_cast<const float2 *>(a.prefix_ml)[(s - own) * total_rows + row];
        return own_ml[s * total_rows];
    };
    auto o_of = [&](int s) {
        if (MODE == kBehindPrefix && s >= own) return a.prefix_o[((s - own) * total_rows + row) * D + dim];
        return own_o[s * total_rows * D];
    };
    float o = 0.0f, l = 0.0f;
    if constexpr (FEW) {
        float2 ml[kFewSplits];
        float part[kFewSplits], top = kNegInf;
#pragma unroll
        for (int s = 0; s < kFewSplits; ++s) {
            ml[s] = s < parts ? ml_of(s) : make_float2(kNegInf, 0.0f);
            part[s] = s < parts ? o_of(s) : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kFewSplits; ++s) top = fmaxf(top, ml[s].x);
        const float to = top == kNegInf ? 0.0f : top;
#pragma unroll
        for (int s = 0; s < kFewSplits; ++s) {
            const float f = __builtin_amdgcn_exp2f(ml[s].x - to);
            o = __builtin_fmaf(f, part[s], o);
            l = __builtin_fmaf(f, ml[s].y, l);
        }
    } else {
        float2 ml = make_float2(kNegInf, 0.0f);
        if (tid < parts) ml = ml_of(tid);
        const float wave_top = wave_max(ml.x);
        if ((tid & 63) == 0) red[0][wave] = wave_top;
        __syncthreads();
        float top = red[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) top = fmaxf(top, red[0][w]);
        const float f = tid < parts ? __builtin_amdgcn_exp2f(ml.x - (top == kNegInf ? 0.0f : top)) : 0.0f;
        factor[tid] = f;
        l = f * ml.y;
#pragma unroll
        for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
        if ((tid & 63) == 0) red[1][wave] = l;
        __syncthreads();
        l = red[1][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) l += red[1][w];
#pragma unroll 8
        for (int s = tid / D; s < parts; s += G) o = __builtin_fmaf(factor[s], o_of(s), o);
        jo[tid] = o;
        __syncthreads();
        if (tid >= D) return;
#pragma unroll
        for (int g = 1; g < G; ++g) o += jo[g * D + tid];
    }
    store_out(static_cast<T *>(a.out) + row * D + dim, l == 0.0f ? 0.0f : o / l);
}

// ---------------------------------------------------------------- launcher

// rows of a kv head that a sequence has on average
inline int64_t rows_each(const CachedProblem &p) { return ceil_div(p.m * (p.q_heads / p.kv_heads), p.seqs); }

// tiles of 4 * rt query rows, of all sequences and heads
inline int64_t units_of(const CachedProblem &p, int rt) { return p.seqs * ceil_div(rows_each(p), 4 * rt) * p.kv_heads; }

// A bound of the tiles per head, whatever the sequences' rows are
inline int64_t query_tiles(const CachedProblem &p, int rt)
{
    const int64_t group = p.q_heads / p.kv_heads, r = 4 * rt;
    return p.cu ? p.m * group / r + p.seqs : p.seqs * ceil_div(group, r);
}

// Row tiles per workgroup: 4 * rt query rows share a page's loads, but a wave works on
// them one after the other (0.5 us per page and tile of rows, 16 rows 2.3). Where four
// rows give no more workgroups than CUs and there is little to read, that spreads the
// work (4 tokens of 20/5 heads over 1000: 6.8 us with 4 rows, 8.8 with 8, 12.3 with
// 16); where there is much, the pages are read less often (32 x 8 tokens of 32/8 heads
// over 2500: 74, 56, 47 us). In between it is 8 rows (16 x 4 tokens of 32/8 heads over
// 2500: 20.0, 18.5, 28.1 us). Pages counted for every tile, as of 128-wide heads. When
// the rule was fitted 482 shapes took 1.04 times their best on average by it (16 rows
// wherever a sequence has more than 8: 1.42).
inline int row_tiles(const CachedProblem &p)
{
    const int64_t rows = rows_each(p), pages = p.max_blocks * p.head_dim / 64;  // twice them
    if (rows <= 4) return 1;
    if (rows > 8 && units_of(p, 4) * pages >= 20000) return 4;
    return units_of(p, 1) <= 256 && units_of(p, 1) * pages <= 12000 ? 1 : 2;
}

// Waves per workgroup, and workgroups per sequence, head and tile of query rows
// (a unit). 16 waves per workgroup (as many as their results fit LDS for: 16 / RT)
// are a CU's share for 4 query rows, and need few or no launches to join:
//  - no more blocks than two per wave (four of 64-wide heads): one workgroup per unit,
//    no joining launch (one sequence of 1023 tokens, 20/5 heads: 6.8 us, split over 4
//    10.0; 2500 tokens 9.6 and 9.6; 3999 12.4 and 9.8; 3000 of 16/4 heads of 64 8.1 and
//    8.5);
//  - up to one unit per CU: as many workgroups as give every CU 16 waves (8 with 8 and
//    16 query rows, whose registers allow no more), but at least a page per wave;
//  - between one and one and a half, where whole workgroups would leave the second
//    round half empty: four waves, split for a thousand workgroups (35 sequences of
//    7800 tokens, 32/8 heads: 107 against 122 us); up to two, where there are more
//    blocks than two per wave, whole ones again (48 x 2 tokens over 300: 14.8 us, with
//    four waves 11.4);
//  - two and more: one workgroup per unit, of four waves, which even out unequal
//    lengths (200 sequences of 2000: 118 against 124 us; 64 of 7800: 168 and 167).
struct Shape {
    int waves;
    int64_t splits;
};
inline Shape launch_shape(const CachedProblem &p, int rt)
{
    const int64_t units = units_of(p, rt), cus = 256;
    const bool lengthy = p.max_blocks * p.head_dim > 256 * 16 / rt;
    const bool wide = units <= cus || (lengthy && 2 * units >= 3 * cus && units < 2 * cus);
    const int waves = wide ? 16 / rt : 4;
    if (p.max_blocks * p.head_dim <= 256 * waves) return {waves, 1};
    int64_t s = (rt == 1 ? 16 : 8) * cus / (waves * units);
    const int64_t most = ceil_div(p.max_blocks, waves);
    s = s > most ? most : s;
    if (units >= 2 * cus || s < 1) s = 1;
    return {waves, s > 256 ? 256 : s};
}

// What a launch takes from a problem
inline CachedArgs cached_args(const CachedProblem &p, const Shape &shape, int rt)
{
    const int64_t group = p.q_heads / p.kv_heads;
    CachedArgs a{};
    a.q = p.q; a.q_stride = p.q_stride; a.m = p.m;
    a.cu = p.cu; a.lens = p.lens; a.table = p.table;
    a.seqs = (int)p.seqs; a.q_heads = (int)p.q_heads; a.kv_heads = (int)p.kv_heads; a.group = (int)group;
    a.splits = (int)shape.splits;
    a.waves = shape.waves;
    a.tiles_per_seq = (int)ceil_div(group, 4 * rt);
    a.max_blocks = p.max_blocks; a.pages = p.pages;
    a.k_codes = p.k_codes; a.v_codes = p.v_codes; a.k_scale = p.k_scale; a.v_scale = p.v_scale;
    a.scale = p.scale * kLog2e; a.out = p.out;
    return a;
}

// The joining launch (launches, where there are more rows than one may have threads for);
// most_parts: a bound of the results that it joins
template <CachedMode MODE, typename T, int D>
inline void launch_join(const CachedProblem &p, const CachedArgs &a, int64_t most_parts, hipStream_t st)
{
    const bool few = most_parts <= kFewSplits;
    const int64_t rows = p.m * p.q_heads, blocks64 = ceil_div(p.max_blocks, 64), extra = p.weights ? p.seqs * blocks64 : 0;
    const int64_t groups = (few ? ceil_div(rows, 512 / D) : rows) + extra;
    for (int64_t first = 0; first < groups; first += kMostGroups) {
        const dim3 grid((unsigned)(groups - first < kMostGroups ? groups - first : kMostGroups));
        if (few) hipLaunchKernelGGL((attention_join_kernel<T, D, true, MODE>), grid, dim3(512), 0, st, a, p.weights, (int)blocks64, first);
        else hipLaunchKernelGGL((attention_join_kernel<T, D, false, MODE>), grid, dim3(512), 0, st, a, p.weights, (int)blocks64, first);
    }
}

// The kernel over `tiles_in_all` tiles per head, and the joining launch where there are splits
template <CachedMode MODE>
inline void launch_tiles(const CachedProblem &p, const CachedArgs &a, const Shape &shape, int rt, int64_t tiles_in_all, hipStream_t st)
{
    auto go_waves = [&](auto type, auto width, auto tiles, auto waves) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value, RT = decltype(tiles)::value, W = decltype(waves)::value;
        in_launches(tiles_in_all, [&](int first, unsigned n) {
            const dim3 grid((unsigned)a.splits, (unsigned)p.kv_heads, n);
            if constexpr (MODE == kWhole) {
                if (p.weights) {
                    hipLaunchKernelGGL((attention_cached_kernel<T, D, RT, W, true, MODE>), grid, dim3(64 * W), 0, st, a, first);
                    return;
                }
            }
            hipLaunchKernelGGL((attention_cached_kernel<T, D, RT, W, false, MODE>), grid, dim3(64 * W), 0, st, a, first);
        }, kMostInZ);
        if (a.splits > 1) launch_join<MODE == kSelectedPast ? kSelected : MODE, T, D>(p, a, a.splits, st);
    };
    auto go = [&](auto type, auto width, auto tiles) {
        constexpr int RT = decltype(tiles)::value;
        if (shape.waves == 4) go_waves(type, width, tiles, Width<4>{});
        else if constexpr (RT < 4) go_waves(type, width, tiles, Width<16 / RT>{});
    };
    auto go_rt = [&](auto type, auto width) {
        if (rt == 1) go(type, width, Width<1>{});
        else if (rt == 2) go(type, width, Width<2>{});
        else go(type, width, Width<4>{});
    };
    if (p.bf16) p.head_dim == 128 ? go_rt(bf16_t{}, Width<128>{}) : go_rt(bf16_t{}, Width<64>{});
    else p.head_dim == 128 ? go_rt(float{}, Width<128>{}) : go_rt(float{}, Width<64>{});
}

}  // namespace bl
