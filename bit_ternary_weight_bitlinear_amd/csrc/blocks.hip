// blocks.hip -- which blocks of the 8-bit cache a new token's attention goes to: the
// bounds of every block's keys, and the choice by them.
//
// Bounds: per page, kv head and dim the largest and the smallest code of K. For a query
// row c of integers no key of the block has a larger product with it than
//   sum_d max(high_d c_d, low_d c_d)
// and summed over the query heads h of a kv head that is
//   T = sum_d high_d P_d + low_d N_d,  P_d = sum_h max(c_hd, 0),  N_d = sum_h min(c_hd, 0),
// 256 bytes (head_dim 128) for a block of 8 KB of K, and work that does not grow with the
// group. With c as the framework quantizes activations (127 for the largest of the group's
// rows) T is a whole number and exact, so the choice has one answer: score = fp32(T) times the
// page's K scale, ties to the lower block.
#include "attention.hpp"

namespace bl {

// ---------------------------------------------------------------- bounds

// A dword of codes as two pairs of 16-bit numbers, 256 times the code: bytes 1 and 3, 0 and 2
typedef short v2s __attribute__((ext_vector_type(2)));
__device__ inline v2s pk_max(v2s a, v2s b) { return __builtin_elementwise_max(a, b); }
__device__ inline v2s pk_min(v2s a, v2s b) { return __builtin_elementwise_min(a, b); }
__device__ inline v2s bits_v2s(uint32_t v) { return __builtin_bit_cast(v2s, v); }
__device__ inline uint32_t v2s_bits(v2s v) { return __builtin_bit_cast(uint32_t, v); }

// One wave per (reached block, kv head). A lane's 16-byte pieces are 16 dims of the tokens
// that share its place in a tile, so what is left are 16 neighbouring lanes. Bound by HBM
// where there are many blocks (55059 tokens of 8 heads of 128: 12.7 us a call, 4.6 TB/s), by
// latency with a token per sequence (32 of them: 3.7 us on the device, 4.2 a call).
template <int D>
__global__ __launch_bounds__(64) void cache_bounds_kernel(const int8_t *__restrict__ k_codes, int8_t *__restrict__ bounds, int64_t pages,
                                                          int64_t m, const int32_t *__restrict__ cu, const int32_t *__restrict__ lens,
                                                          int seqs, const int32_t *__restrict__ table, int64_t max_blocks)
{
    constexpr int G = D / 64;  // 4-tile groups of dims that a lane has
    SeqTile t;
    int64_t block;
    if (!find_block(cu, lens, seqs, m, max_blocks, blockIdx.x, t, block)) return;
    const int head = blockIdx.y, heads = gridDim.y, lane = threadIdx.x;
    const int64_t page = table[(int64_t)t.seq * max_blocks + block];
    if (page < 0 || page >= pages) return;
    const int64_t left = (int64_t)lens[t.seq] + t.n - block * kBlock;  // tokens that the block holds, at least one
    const int held = left < kBlock ? (int)left : kBlock;
    const uint4 *src = reinterpret_cast<const uint4 *>(k_codes + (page * heads + head) * (kBlock * D)) + lane;
    uint4 c[4][G];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int g = 0; g < G; ++g) c[q][g] = src[(q * G + g) * 64];
    // [odd, even bytes] of the lane's 16 dims
    v2s high[G][4][2], low[G][4][2];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                high[g][w][b] = bits_v2s(0x80008000u);
                low[g][w][b] = bits_v2s(0x7F007F00u);
            }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (4 * (lane & 15) + q >= held) continue;  // the token of this lane's pieces
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t w4[4] = {c[q][g].x, c[q][g].y, c[q][g].z, c[q][g].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const v2s odd = bits_v2s(w4[w] & 0xFF00FF00u), even = bits_v2s((w4[w] << 8) & 0xFF00FF00u);
                high[g][w][0] = pk_max(high[g][w][0], odd);
                high[g][w][1] = pk_max(high[g][w][1], even);
                low[g][w][0] = pk_min(low[g][w][0], odd);
                low[g][w][1] = pk_min(low[g][w][1], even);
            }
        }
    }
    auto over = [](v2s v, auto f) {
        v = f(v, bits_v2s((uint32_t)dpp_mov<kDppQuadXor1>((int)v2s_bits(v))));
        v = f(v, bits_v2s((uint32_t)dpp_mov<kDppQuadXor2>((int)v2s_bits(v))));
        v = f(v, bits_v2s((uint32_t)dpp_mov<kDppRowHalfMirror>((int)v2s_bits(v))));
        return f(v, bits_v2s((uint32_t)dpp_mov<kDppRowMirror>((int)v2s_bits(v))));
    };
    int8_t *dst = bounds + (page * heads + head) * (2 * D);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t h1 = v2s_bits(over(high[g][w][0], pk_max)), h0 = v2s_bits(over(high[g][w][1], pk_max));
            const uint32_t l1 = v2s_bits(over(low[g][w][0], pk_min)), l0 = v2s_bits(over(low[g][w][1], pk_min));
            h[w] = h1 | (h0 >> 8 & 0x00FF00FFu);
            l[w] = l1 | (l0 >> 8 & 0x00FF00FFu);
        }
        const int dim = (4 * g + (lane >> 4)) * 16;
        if ((lane & 15) == 0) *reinterpret_cast<uint4 *>(dst + dim) = make_uint4(h[0], h[1], h[2], h[3]);
        if ((lane & 15) == 1) *reinterpret_cast<uint4 *>(dst + D + dim) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// ---------------------------------------------------------------- selection

struct SelectArgs {
    const void *q;
    int64_t q_stride, m;
    const int32_t *cu, *lens, *table;
    int seqs, q_heads, kv_heads, group;
    int64_t max_blocks, pages, keep, first, recent;
    const int8_t *bounds;
    const float *k_scale;
    int32_t *selected;
    uint32_t *keys;  // [m][kv_heads][max_blocks], where a workgroup's LDS does not hold them
};

constexpr int kKeysInLds = 8192;
constexpr float kLargest = 3.402823466e38f;

// The sums of the group's positive and negative parts, as a lane's digits of 7 bits and a sign: of
// the 2 * D / 16 lanes that have a block's bounds the first half has P, the other N. Every element
// is looked at twice, for the largest and then for its integer, with the largest on the way
// through LDS between. `sums`: D words, zero at the start; at most 127 * 128 in either half.
template <typename T, int D, int THREADS>
struct QueryDigits {
    static constexpr int E = 16 / sizeof(T), KEEP = 2;  // elements of a piece; pieces kept in registers
    T raw[KEEP][E];
    const T *src;
    int pieces;

    __device__ void load(const SelectArgs &a, int64_t row, int head)
    {
        pieces = a.group * D / E;
        src = static_cast<const T *>(a.q) + row * a.q_stride + (int64_t)head * a.group * D;  // a kv head's query heads are adjacent
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if ((int)threadIdx.x + k * THREADS < pieces)
                *reinterpret_cast<uint4 *>(raw[k]) = reinterpret_cast<const uint4 *>(src)[threadIdx.x + k * THREADS];
    }
    // f(piece, elements) for every piece of this thread
    template <typename F>
    __device__ void each(F f)
    {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if ((int)threadIdx.x + k * THREADS < pieces) f((int)threadIdx.x + k * THREADS, raw[k]);
        for (int i = threadIdx.x + KEEP * THREADS; i < pieces; i += THREADS) {
            T more[E];
            *reinterpret_cast<uint4 *>(more) = reinterpret_cast<const uint4 *>(src)[i];
            f(i, more);
        }
    }
    // NaN counts as 0 and infinities as the largest finite number
    static __device__ float value(T x)
    {
        const float v = to_f32(x);
        return v == v ? fminf(fmaxf(v, -kLargest), kLargest) : 0.0f;
    }
    __device__ float largest()
    {
        float big = 0.0f;
        each([&](int, const T *x) {
#pragma unroll
            for (int i = 0; i < E; ++i) big = fmaxf(big, fabsf(value(x[i])));
        });
        return wave_max(big);
    }
    __device__ void add(float big, uint32_t *sums)
    {
        const float inv = 127.0f / fmaxf(big, 1e-30f);
        each([&](int piece, const T *x) {
            const int dim = piece * E % D;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = (int)rintf(value(x[i]) * inv);
                atomicAdd(&sums[dim + i], c < 0 ? (uint32_t)-c << 16 : (uint32_t)c);
            }
        });
    }
    static __device__ void digits(const uint32_t *sums, v4i &lo, v4i &hi)
    {
        const int at = (threadIdx.x & 63) % (D / 8), dim = at % (D / 16) * 16, down = at < D / 16 ? 0 : 16;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sums + dim + 4 * w);
            const uint32_t x[4] = {v.x >> down & 0xFFFFu, v.y >> down & 0xFFFFu, v.z >> down & 0xFFFFu, v.w >> down & 0xFFFFu};
            uint32_t l = 0, h = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = at < D / 16 ? (int)x[i] : -(int)x[i];
                l |= (uint32_t)(v % 128 & 0xFF) << (8 * i);
                h |= (uint32_t)(v / 128 & 0xFF) << (8 * i);
            }
            lo[w] = (int)l;
            hi[w] = (int)h;
        }
    }
};

// Bounds of 64 blocks of a sequence: D / 8 lanes have one block's, so a wave's load holds
// B = 64 / (D / 8) blocks. After the products a lane has the sum of its block alone: in a
// step of the reduction a lane keeps one of two loads' sums, by a bit of its number, and gets
// the other lane's share of it. Its block is `place` of the 64.
template <int D>
struct BlockBounds {
    static constexpr int L = D / 8, B = 64 / L;  // L loads
    v4i c[L];
    float scale;
    bool ok;

    // The steps' partners are mirrored rows, halves of rows and pairs in quads, in this order, so
    // that a partner differs in bits that have not been used yet: bits 3 (or 2) to 0 of the
    // lane, the first of them the lowest of its load's number
    static constexpr __host__ __device__ int reversed(int i)
    {
        return L == 16 ? (i & 1) << 3 | (i & 2) << 1 | (i & 4) >> 1 | (i & 8) >> 3 : (i & 1) << 2 | (i & 2) | (i & 4) >> 2;
    }
    static __device__ int place() { return reversed((int)threadIdx.x & (L - 1)) * B + ((int)threadIdx.x & 63) / L; }

    // id: of the lane's block
    __device__ void load(const SelectArgs &a, int id, int head)
    {
        const int lane = threadIdx.x & 63;
        ok = id >= 0 && id < a.pages;
        const int page = ok ? id : 0;  // a block without a page reads page 0
        const int8_t *src = a.bounds + lane % L * 16;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            // the lane whose block is i * B + lane / L
            const int64_t at = (int64_t)__shfl(page, lane / L * L + reversed(i)) * a.kv_heads + head;
            c[i] = *reinterpret_cast<const v4i *>(src + at * (2 * D));
        }
        scale = a.k_scale[(int64_t)page * a.kv_heads + head];
    }
    template <int CTRL, int N>
    static __device__ void halve(int (&v)[L], int bit)
    {
        const bool odd = threadIdx.x >> bit & 1;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const int stays = odd ? v[2 * i + 1] : v[2 * i], goes = odd ? v[2 * i] : v[2 * i + 1];
            v[i] = stays + dpp_mov<CTRL>(goes);
        }
    }
    // the key of the lane's block: its score in order, as the weights of an eviction are
    __device__ uint32_t key(const v4i &lo, const v4i &hi) const
    {
        int v[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            int l = 0, h = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                l = __builtin_amdgcn_sdot4(c[i][w], lo[w], l, false);
                h = __builtin_amdgcn_sdot4(c[i][w], hi[w], h, false);
            }
            v[i] = l + (h << 7);
        }
        if constexpr (L == 16) halve<kDppRowMirror, 16>(v, 3);
        halve<kDppRowHalfMirror, 8>(v, 2);
        halve<kDppQuadXor2, 4>(v, 1);
        halve<kDppQuadXor1, 2>(v, 0);
        return ok ? weight_key((float)v[0] * scale) : weight_key(kNegInf);
    }
};

// What a row and kv head choose from
struct Choice {
    int used, mid0, mid1, want;  // blocks; those that a score decides on, and how many of them stay

    __device__ Choice(const SelectArgs &a, int64_t have, int place)
    {
        const int64_t blocks = (have + place) / kBlock + 1;
        used = blocks < a.max_blocks ? (int)blocks : (int)a.max_blocks;
        const bool all = used <= a.keep;
        mid0 = all ? used : (int)a.first;
        mid1 = all ? used : (int)(used - a.recent);
        want = all ? 0 : (int)(a.keep - a.first - a.recent);
    }
};

__device__ inline uint32_t wave_max_u32(uint32_t v)
{
    auto up = [&](int o) { v = (uint32_t)o > v ? (uint32_t)o : v; };
    up(dpp_mov<kDppQuadXor1>((int)v));
    up(dpp_mov<kDppQuadXor2>((int)v));
    up(dpp_mov<kDppRowHalfMirror>((int)v));
    up(dpp_mov<kDppRowMirror>((int)v));
    up(__builtin_amdgcn_update_dpp((int)v, (int)v, kDppRowBcast15, 0xA, 0xF, false));
    up(__builtin_amdgcn_update_dpp((int)v, (int)v, kDppRowBcast31, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// LDS of choose(): three histograms, zero at the start, and counts of 64 blocks each
template <int THREADS>
struct ChooseLds {
    __align__(16) int hist[3][kDigitBins];
    uint32_t ends[2][THREADS / 64];
    int sums[2][64];
};

// The list of a row and kv head, in block order, from its blocks' keys: the `want` largest of
// those at mid0 .. mid1-1, of equals the lower blocks, and everything outside. The least that
// stays is found by digits of 11 bits from the highest in which the keys differ (their sign,
// exponent and first bits are mostly the same, and counts of one digit stand in line), until
// a digit's count is what is left to keep. low, high: the wave's least and largest key of
// the middle. The keys, and the histograms' zeros, are behind the caller's writes, not yet behind a barrier.
template <int THREADS>
__device__ inline void choose(const SelectArgs &a, const Choice &ch, const uint32_t *keys, uint32_t low, uint32_t high, int32_t *out,
                              ChooseLds<THREADS> &lds)
{
    constexpr int W = THREADS / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // keys without their lowest `shift` bits: above `prefix` they stay, and `left` of those that equal it
    uint32_t prefix = 0;
    int shift = 0, left = ch.want;
    if (ch.want > 0) {
        high = wave_max_u32(high);
        low = ~wave_max_u32(~low);
        if (lane == 0) {
            lds.ends[0][wave] = low;
            lds.ends[1][wave] = high;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) {
            low = lds.ends[0][w] < low ? lds.ends[0][w] : low;
            high = lds.ends[1][w] > high ? lds.ends[1][w] : high;
        }
        shift = low == high ? 0 : 32 - __builtin_clz(low ^ high);
        prefix = shift < 32 ? high >> shift : 0;
        for (int round = 0; round < 3 && shift > 0; ++round) {
            int *hist = lds.hist[round];
            const int down = shift > kDigitBits ? shift - kDigitBits : 0, bits = shift - down;
            for (int b = ch.mid0 + tid; b < ch.mid1; b += THREADS) {
                const uint32_t key = keys[b];
                if (shift == 32 || key >> shift == prefix) atomicAdd(&hist[key >> down & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            const uint32_t digit = pick_digit(hist, left);
            prefix = prefix << bits | digit;
            shift = down;
            if (hist[digit] == left) break;  // all of them stay
        }
    }
    // which blocks stay, C times THREADS of them at a time: a count for every 64 of them, and what
    // stands before them by one scan of the counts
    constexpr int C = W == 16 ? 4 : 2;
    int sure_at = 0, equal_at = 0;  // of the blocks before: those that stay anyway, and the cut's equals
    for (int b0 = 0, buf = 0; b0 < ch.used; b0 += C * THREADS, buf ^= 1) {
        uint64_t equals[C], sures[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int b = b0 + c * THREADS + tid;
            const bool in = b < ch.used, mid = in && b >= ch.mid0 && b < ch.mid1;
            const uint32_t key = ch.want > 0 && mid ? keys[b] >> shift : 0;
            equals[c] = __ballot(ch.want > 0 && mid && key == prefix);
            sures[c] = __ballot(in && (!mid || (ch.want > 0 && key > prefix)));
            if (lane == 0) lds.sums[buf][c * W + wave] = __popcll(sures[c]) << 16 | __popcll(equals[c]);
        }
        __syncthreads();
        const int incl = wave_scan(lane < C * W ? lds.sums[buf][lane] : 0);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = c * W + wave, mine = at ? __builtin_amdgcn_readlane(incl, at - 1) : 0;
            const uint64_t below = lane ? ~0ull >> (64 - lane) : 0;
            const int eq = equal_at + (mine & 0xFFFF) + __popcll(equals[c] & below);
            const int sure = sure_at + (mine >> 16) + __popcll(sures[c] & below);
            if (sures[c] >> lane & 1 || (equals[c] >> lane & 1 && eq < left)) out[sure + (eq < left ? eq : left)] = b0 + c * THREADS + tid;
        }
        const int all = __builtin_amdgcn_readlane(incl, 63);
        sure_at += all >> 16;
        equal_at += all & 0xFFFF;
    }
    const int stayed = sure_at + (equal_at < left ? equal_at : left);
    for (int64_t i = stayed + tid; i < a.keep; i += THREADS) out[i] = -1;
}

// least and largest key of the middle
__device__ inline void widen(const Choice &ch, int b, uint32_t key, uint32_t &low, uint32_t &high)
{
    if (b < ch.mid0 || b >= ch.mid1) return;
    low = key < low ? key : low;
    high = key > high ? key : high;
}

// A workgroup per (row, kv head): the keys of its blocks into LDS, and the list. The queries
// and the first bounds are asked for before either is needed. Workgroups go to the eight XCDs
// in turn; each XCD has neighbouring rows of a head, which read the same bounds where they are
// of one sequence (64 x 2 tokens over up to 500 blocks: 14.0 us beside 17.1).
template <typename T, int D, int THREADS, int KEYS>
__global__ __launch_bounds__(THREADS, 4) void block_select_kernel(SelectArgs a, int64_t first, int64_t items)
{
    constexpr int W = THREADS / 64;
    __shared__ uint32_t keys[KEYS];
    __shared__ ChooseLds<THREADS> lds;
    __shared__ __align__(16) uint32_t digits[D];
    __shared__ float red[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t each = gridDim.x / 8, item = first + blockIdx.x % 8 * each + blockIdx.x / 8;
    if (item >= items) return;
    const int head = (int)(item / a.m);
    const int64_t row = item - head * a.m;
    QueryDigits<T, D, THREADS> q;
    q.load(a, row, head);
    for (int i = tid; i < 3 * kDigitBins; i += THREADS) lds.hist[0][i] = 0;
    for (int i = tid; i < D; i += THREADS) digits[i] = 0;
    int seq, place, have;
    if (!find_row(a.cu, a.lens, a.seqs, a.m, row, seq, place, have) || have < 0) return;
    const Choice ch(a, have, place);
    const int32_t *table = a.table + (int64_t)seq * a.max_blocks;
    uint32_t low = ~0u, high = 0;
    if (ch.want > 0) {
        BlockBounds<D> bounds;
        int b0 = wave * 64;
        auto id_of = [&](int at) { return at + bounds.place() < ch.used ? table[at + bounds.place()] : -1; };
        int id = id_of(b0);
        if (b0 < ch.used) bounds.load(a, id, head);
        id = id_of(b0 + THREADS);
        float most = q.largest();
        if (lane == 0) red[wave] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) most = fmaxf(most, red[w]);
        q.add(most, digits);
        __syncthreads();
        v4i lo, hi;
        q.digits(digits, lo, hi);
        for (; b0 < ch.used; b0 += THREADS) {
            const uint32_t key = bounds.key(lo, hi);
            if (b0 + THREADS < ch.used) {
                bounds.load(a, id, head);
                id = id_of(b0 + 2 * THREADS);
            }
            const int b = b0 + bounds.place();
            if (b < ch.used) keys[b] = key;
            widen(ch, b < ch.used ? b : -1, key, low, high);
        }
    }
    choose<THREADS>(a, ch, keys, low, high, a.selected + (row * a.kv_heads + head) * a.keep, lds);
}

// The same by two launches, for few rows and heads or tables too wide for LDS: the keys into
// the workspace, four waves of 64 blocks per workgroup, and a workgroup per (row, kv head) that
// chooses by them.
template <typename T, int D>
__global__ __launch_bounds__(256, 4) void block_score_kernel(SelectArgs a, int first_row)
{
    __shared__ __align__(16) uint32_t digits[D];
    __shared__ float red[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, head = blockIdx.y;
    const int64_t row = (int64_t)first_row + blockIdx.z;
    QueryDigits<T, D, 256> q;
    q.load(a, row, head);
    for (int i = tid; i < D; i += 256) digits[i] = 0;
    int seq, place, have;
    if (!find_row(a.cu, a.lens, a.seqs, a.m, row, seq, place, have) || have < 0) return;
    const Choice ch(a, have, place);
    const int group0 = (int)blockIdx.x * 256, b = group0 + wave * 64 + BlockBounds<D>::place();
    if (ch.want == 0 || group0 >= ch.used) return;
    BlockBounds<D> bounds;
    bounds.load(a, b < ch.used ? a.table[(int64_t)seq * a.max_blocks + b] : -1, head);
    float most = q.largest();
    if (lane == 0) red[wave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) most = fmaxf(most, red[w]);
    q.add(most, digits);
    __syncthreads();
    v4i lo, hi;
    q.digits(digits, lo, hi);
    const uint32_t key = bounds.key(lo, hi);
    if (b < ch.used) a.keys[(row * a.kv_heads + head) * a.max_blocks + b] = key;
}

template <int KEYS>
__global__ __launch_bounds__(1024) void block_choose_kernel(SelectArgs a, int first_row)
{
    constexpr int THREADS = 1024;
    __shared__ uint32_t held[KEYS ? KEYS : 1];
    __shared__ ChooseLds<THREADS> lds;
    const int tid = threadIdx.x, head = blockIdx.y;
    const int64_t row = (int64_t)first_row + blockIdx.x;
    for (int i = tid; i < 3 * kDigitBins; i += THREADS) lds.hist[0][i] = 0;
    int seq, place, have;
    if (!find_row(a.cu, a.lens, a.seqs, a.m, row, seq, place, have) || have < 0) return;
    const Choice ch(a, have, place);
    const uint32_t *keys = a.keys + (row * a.kv_heads + head) * a.max_blocks;
    uint32_t low = ~0u, high = 0;
    if (ch.want > 0)
        for (int b = tid; b < ch.used; b += THREADS) {
            const uint32_t key = keys[b];
            if (KEYS) held[b] = key;
            widen(ch, b, key, low, high);
        }
    choose<THREADS>(a, ch, KEYS ? held : keys, low, high, a.selected + (row * a.kv_heads + head) * a.keep, lds);
}

// ---------------------------------------------------------------- launchers

hipError_t launch_cache_bounds(const CacheBounds &p, hipStream_t st)
{
    // reached blocks of a batch: at most n / 64 + 2 of a sequence with n rows
    const int64_t most = p.cu ? p.m / kBlock + 2 * p.seqs : p.seqs;
    const dim3 grid((unsigned)most, (unsigned)p.kv_heads);
    auto go = [&](auto width) {
        hipLaunchKernelGGL((cache_bounds_kernel<decltype(width)::value>), grid, dim3(64), 0, st, p.k_codes, p.bounds, p.pages, p.m, p.cu,
                           p.lens, (int)p.seqs, p.table, p.max_blocks);
    };
    p.head_dim == 128 ? go(Width<128>{}) : go(Width<64>{});
    return hipGetLastError();
}

// One workgroup reads a head's bounds at 64 bytes a cycle and takes 6 us of arithmetic for
// 2048 blocks: where rows and heads leave CUs idle, the scores are a launch of their own. On the
// device, of 8 heads with 4 rows each (m x heads: two launches and one, us):
//   550 blocks   16: 10.2, 10.1   64: 11.3, 11.0   96: 14.0, 12.2
//   1000         32: 11.5, 12.3   64: 13.3, 14.2   96: 15.6, 14.5   192: 18.8, 17.3
//   1100         64: 14.7, 15.7   96: 15.5, 16.1   128: 17.3, 16.8  192: 20.5, 19.0
//   1500         64: 15.3, 17.3   96: 17.8, 18.1   160: 20.8, 20.6  192: 23.3, 22.5
//   2048         8: 11.2, 17.1    64: 16.7, 21.0   96: 19.3, 21.9   192: 29.8, 31.0   256: 39.0, 37.9
//   4096         64: 22.8, 29.6   96: 30.6, 43.4   192: 52.3, 53.6  256: 65.3, 64.6
//   8192         64: 43.2, 79.1   128: 68.6, 87.1  192: 93.7, 100.9
// 300 blocks of one token 10.6 and 8.7.
static bool two_launches(int64_t m, int64_t kv_heads, int64_t max_blocks)
{
    return max_blocks > kKeysInLds || (max_blocks > 512 && m * kv_heads <= (max_blocks < 1500 ? 64 : 192));
}

int64_t block_select_workspace(int64_t m, int64_t kv_heads, int64_t max_blocks)
{
    return two_launches(m, kv_heads, max_blocks) ? m * kv_heads * max_blocks * 4 : 0;
}

hipError_t launch_block_select(const SelectProblem &p, void *ws, hipStream_t st)
{
    SelectArgs a{};
    a.q = p.q; a.q_stride = p.q_stride; a.m = p.m; a.cu = p.cu; a.lens = p.lens; a.table = p.table; a.seqs = (int)p.seqs;
    a.q_heads = (int)p.q_heads; a.kv_heads = (int)p.kv_heads; a.group = (int)(p.q_heads / p.kv_heads);
    a.max_blocks = p.max_blocks; a.pages = p.pages; a.keep = p.keep; a.first = p.first; a.recent = p.recent;
    a.bounds = p.bounds; a.k_scale = p.k_scale; a.selected = p.selected; a.keys = static_cast<uint32_t *>(ws);
    auto go = [&](auto type, auto width) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value;
        const bool apart = two_launches(p.m, p.kv_heads, p.max_blocks);
        if (apart)
            in_launches(p.m, [&](int first, unsigned n) {
                const dim3 grid((unsigned)ceil_div(p.max_blocks, 256), (unsigned)p.kv_heads, n);
                hipLaunchKernelGGL((block_score_kernel<T, D>), grid, dim3(256), 0, st, a, first);
            }, kMostInZ);
        if (apart) {
            in_launches(p.m, [&](int first, unsigned n) {
                const dim3 grid(n, (unsigned)p.kv_heads);
                if (p.max_blocks <= kKeysInLds) hipLaunchKernelGGL((block_choose_kernel<kKeysInLds>), grid, dim3(1024), 0, st, a, first);
                else hipLaunchKernelGGL((block_choose_kernel<0>), grid, dim3(1024), 0, st, a, first);
            });
            return;
        }
        const int64_t items = p.m * p.kv_heads;
        for (int64_t first = 0; first < items; first += kMostGroups) {
            const int64_t end = first + kMostGroups < items ? first + kMostGroups : items;
            const dim3 grid((unsigned)round_up(end - first, 8));
            // Small workgroups overlap each other's waits: 512 of 500 blocks take 15.7 us with 256
            // threads and 26.0 with 1024, of 1000 blocks 24.2 and 36.7, of 2000 41.6 and 47.6
            if (p.max_blocks <= 2048) hipLaunchKernelGGL((block_select_kernel<T, D, 256, 2048>), grid, dim3(256), 0, st, a, first, end);
            else hipLaunchKernelGGL((block_select_kernel<T, D, 1024, kKeysInLds>), grid, dim3(1024), 0, st, a, first, end);
        }
    };
    if (p.bf16) p.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
    else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    return hipGetLastError();
}

}  // namespace bl
