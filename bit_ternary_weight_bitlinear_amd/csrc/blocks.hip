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
// where there are many blocks, by latency with a token per sequence.
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
    int seqs, q_heads, kv_heads, group, splits;
    int64_t max_blocks, pages, keep, first, recent;
    const int8_t *bounds;
    const float *k_scale;
    int32_t *selected;
    uint32_t *keys;  // [m][kv_heads][max_blocks], where a workgroup's LDS does not hold them
};

constexpr int kSelectThreads = 512;
constexpr int kKeysInLds = 8192;

// The sums of the group's positive and negative parts as a lane's digits of 7 bits: lanes
// 0 .. D/16-1 of a 16-byte piece's 2 * D/16 lanes have P, the others -N. `lds`: D words.
template <typename T, int D>
__device__ inline void query_digits(const SelectArgs &a, int64_t row, int head, uint32_t *lds, float *red, v4i &lo, v4i &hi)
{
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 63, n = a.group * D;
    const T *src = static_cast<const T *>(a.q) + row * a.q_stride + (int64_t)head * n;  // a kv head's query heads are adjacent
    constexpr float kMost = 3.402823466e38f;
    auto value = [&](int i) {  // NaN counts as 0 and infinities as the largest finite number
        const float v = to_f32(src[i]);
        return v == v ? fminf(fmaxf(v, -kMost), kMost) : 0.0f;
    };
    float big = 0.0f;
    for (int i = tid; i < n; i += threads) big = fmaxf(big, fabsf(value(i)));
    big = wave_max(big);
    if (lane == 0) red[tid >> 6] = big;
    __syncthreads();
    for (int w = 0; w < threads / 64; ++w) big = fmaxf(big, red[w]);
    const float inv = 127.0f / fmaxf(big, 1e-30f);
    for (int d = tid; d < D; d += threads) {
        int p = 0, q = 0;
        for (int h = 0; h < a.group; ++h) {
            const int c = (int)rintf(value(h * D + d) * inv);
            p += c > 0 ? c : 0;
            q += c < 0 ? -c : 0;
        }
        lds[d] = (uint32_t)p | (uint32_t)q << 16;  // at most 127 * 128
    }
    __syncthreads();
    const int at = lane % (D / 8), dim = at % (D / 16) * 16, down = at < D / 16 ? 0 : 16;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t l = 0, h = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = lds[dim + 4 * w + i] >> down & 0xFFFFu;
            l |= (v & 127u) << (8 * i);
            h |= (v >> 7) << (8 * i);
        }
        lo[w] = (int)l;
        hi[w] = (int)h;
    }
}

// Keys of blocks b0 .. b0+63 of a sequence, one per lane: their scores in order, as the
// weights of an eviction are. D/8 lanes have a block's bounds, so a wave's load is 64 / (D/8)
// blocks.
template <int D>
__device__ inline uint32_t block_keys(const SelectArgs &a, const int32_t *table, int head, int b0, int used, const v4i &lo, const v4i &hi)
{
    constexpr int L = D / 8, B = 64 / L;  // lanes of a block, blocks of a load
    const int lane = threadIdx.x & 63, mine = b0 + lane;
    const int id = mine < used ? table[mine] : -1;
    const bool ok = id >= 0 && id < a.pages;
    const int64_t my_at = ok ? (int64_t)id * a.kv_heads + head : 0;
    const float scale = ok ? a.k_scale[my_at] : 0.0f;
    const int page = ok ? id : 0;
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < 64 / B; ++i) {
        const int64_t at = (int64_t)__shfl(page, i * B + lane / L) * a.kv_heads + head;
        const v4i c = *reinterpret_cast<const v4i *>(a.bounds + at * (2 * D) + lane % L * 16);
        int l = 0, h = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            l = __builtin_amdgcn_sdot4(c[w], lo[w], l, false);
            h = __builtin_amdgcn_sdot4(c[w], hi[w], h, false);
        }
        int v = l + (h << 7);
        if (lane % L >= L / 2) v = -v;  // low_d N_d, by -N
        if constexpr (L == 16) v = row16_sum(v);
        else v = group8_sum(v);
        const int got = __shfl(v, lane % B * L);
        if (lane / B == i) sum = got;
    }
    return ok ? weight_key((float)sum * scale) : weight_key(kNegInf);
}

// The blocks that stay of those at mid0 .. mid1-1, `want` of them: every key above `prefix`
// (without its lowest `shift` bits) and the first `left` that equal it. By digits from the
// top, until a digit's count is what is left to keep.
struct Cut {
    uint32_t prefix;
    int shift, left;
};
template <int THREADS>
__device__ inline Cut find_cut(const uint32_t *keys, int mid0, int mid1, int want, int *hist, int *wave_sums, int *pick)
{
    constexpr int W = THREADS / 64, kBins = 2048, PER = kBins / THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Cut r{0, 32, want};
    while (want > 0 && r.shift > 0) {
        const int bits = r.shift > 10 ? 11 : 10, down = r.shift - bits;
#pragma unroll
        for (int i = 0; i < PER; ++i) hist[tid + i * THREADS] = 0;
        __syncthreads();
        for (int b = mid0 + tid; b < mid1; b += THREADS) {
            const uint32_t key = keys[b];
            if (r.shift == 32 || key >> r.shift == r.prefix) atomicAdd(&hist[key >> down & ((1u << bits) - 1)], 1);
        }
        __syncthreads();
        // thread i has the i-th largest PER digits; what lies above them
        const int top = (1 << bits) - 1 - PER * tid;
        int h[PER], mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            h[i] = top - i >= 0 ? hist[top - i] : 0;
            mine += h[i];
        }
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 63) wave_sums[wave] = incl;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (w < wave) incl += wave_sums[w];
        int above = incl - mine;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (above < r.left && above + h[i] >= r.left) {
                pick[0] = top - i;
                pick[1] = r.left - above;
                pick[2] = h[i];
            }
            above += h[i];
        }
        __syncthreads();
        r.prefix = r.prefix << bits | (uint32_t)pick[0];
        r.left = pick[1];
        r.shift = down;
        if (pick[2] == r.left) break;  // all of them stay
        __syncthreads();
    }
    return r;
}

// One workgroup per (row, kv head): the keys of its blocks into LDS (or, of tables too
// wide for it, into the workspace), the cut, and the list in block order.
template <typename T, int D, bool LDS>
__global__ __launch_bounds__(kSelectThreads) void block_select_kernel(SelectArgs a, int first_row)
{
    constexpr int THREADS = kSelectThreads, W = THREADS / 64;
    __shared__ uint32_t held[LDS ? kKeysInLds : 1];
    __shared__ int hist[2048];
    __shared__ uint32_t digits[D];
    __shared__ float red[W];
    __shared__ int wave_sums[W], pick[3], sums[2][2][W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, head = blockIdx.y;
    const int64_t row = (int64_t)first_row + blockIdx.x;
    int seq, place;
    if (!find_row(a.cu, a.seqs, a.m, row, seq, place)) return;
    const int64_t have = a.lens[seq];
    if (have < 0) return;
    const int64_t blocks = (have + place) / kBlock + 1;
    const int used = blocks < a.max_blocks ? (int)blocks : (int)a.max_blocks;
    const bool all = used <= a.keep;
    const int mid0 = all ? used : (int)a.first, mid1 = all ? used : (int)(used - a.recent);
    const int want = all ? 0 : (int)(a.keep - a.first - a.recent);
    const int32_t *table = a.table + (int64_t)seq * a.max_blocks;
    uint32_t *keys = LDS ? held : a.keys + (row * a.kv_heads + head) * a.max_blocks;
    Cut cut{0, 32, 0};
    if (want > 0) {
        v4i lo, hi;
        query_digits<T, D>(a, row, head, digits, red, lo, hi);
        for (int b0 = wave * 64; b0 < used; b0 += THREADS) {
            const uint32_t key = block_keys<D>(a, table, head, b0, used, lo, hi);
            if (b0 + lane < used) keys[b0 + lane] = key;
        }
        __syncthreads();
        cut = find_cut<THREADS>(keys, mid0, mid1, want, hist, wave_sums, pick);
    }
    int32_t *out = a.selected + (row * a.kv_heads + head) * a.keep;
    int stay_at = 0, equal_at = 0;
    for (int b0 = 0, buf = 0; b0 < used; b0 += THREADS, buf ^= 1) {
        const int b = b0 + tid;
        const bool in = b < used, mid = in && b >= mid0 && b < mid1;
        const uint32_t key = want > 0 && mid ? keys[b] >> cut.shift : 0;
        const bool equal = mid && want > 0 && key == cut.prefix;
        const uint64_t below = lane ? ~0ull >> (64 - lane) : 0;
        const uint64_t eq_mask = __ballot(equal);
        if (lane == 0) sums[buf][0][wave] = __popcll(eq_mask);
        __syncthreads();
        int eq = equal_at + __popcll(eq_mask & below);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < wave) eq += sums[buf][0][i];
            equal_at += sums[buf][0][i];
        }
        const bool stay = in && (!mid || (want > 0 && (key > cut.prefix || (equal && eq < cut.left))));
        const uint64_t stay_mask = __ballot(stay);
        if (lane == 0) sums[buf][1][wave] = __popcll(stay_mask);
        __syncthreads();
        int at = stay_at + __popcll(stay_mask & below);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < wave) at += sums[buf][1][i];
            stay_at += sums[buf][1][i];
        }
        if (stay) out[at] = b;
    }
    for (int64_t i = stay_at + tid; i < a.keep; i += THREADS) out[i] = -1;
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

int64_t block_select_workspace(int64_t m, int64_t kv_heads, int64_t max_blocks)
{
    return max_blocks <= kKeysInLds ? 0 : m * kv_heads * max_blocks * 4;
}

hipError_t launch_block_select(const SelectProblem &p, void *ws, hipStream_t st)
{
    SelectArgs a{};
    a.q = p.q; a.q_stride = p.q_stride; a.m = p.m; a.cu = p.cu; a.lens = p.lens; a.table = p.table; a.seqs = (int)p.seqs;
    a.q_heads = (int)p.q_heads; a.kv_heads = (int)p.kv_heads; a.group = (int)(p.q_heads / p.kv_heads);
    a.max_blocks = p.max_blocks; a.pages = p.pages; a.keep = p.keep; a.first = p.first; a.recent = p.recent;
    a.bounds = p.bounds; a.k_scale = p.k_scale; a.selected = p.selected; a.keys = static_cast<uint32_t *>(ws);
    in_launches(p.m, [&](int first, unsigned n) {
        const dim3 grid(n, (unsigned)p.kv_heads), threads(kSelectThreads);
        auto go = [&](auto type, auto width) {
            using T = decltype(type);
            constexpr int D = decltype(width)::value;
            if (p.max_blocks <= kKeysInLds) hipLaunchKernelGGL((block_select_kernel<T, D, true>), grid, threads, 0, st, a, first);
            else hipLaunchKernelGGL((block_select_kernel<T, D, false>), grid, threads, 0, st, a, first);
        };
        if (p.bf16) p.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
        else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    });
    return hipGetLastError();
}

}  // namespace bl
