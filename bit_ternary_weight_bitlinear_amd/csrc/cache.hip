// cache.hip -- the 8-bit key/value cache: append, read back, eviction of blocks.
//
// A page holds 64 tokens; per page and kv head there is one scale for K and one
// for V, and the codes lie in the operand order of the int8 matrix instructions
// (include/bitlinear.h), so that the attention kernel reads whole pages with
// contiguous 16-byte loads and no shuffles. The cost of that order is paid here:
// one token's V codes are bytes 16 apart.
#include "attention.hpp"

namespace bl {

constexpr float kSmallestScale = 1e-30f;  // keeps 127 / s finite

// an earlier token's code under a scale that has grown by 1 / ratio
__device__ inline int rescale_code(int c, float ratio) { return (int)rintf((float)c * ratio); }

// One workgroup per (touched block, kv head), K and V together: the new rows are
// read once into registers, their largest magnitudes give the two scales, the
// codes meet in LDS and leave in the cache's order. Traffic-bound: the rows in,
// a quarter (fp32) or half (bf16) of that out; earlier codes are read only where
// a scale grew, and for the 16-token groups of V that the new tokens share.
template <typename T, int D>
__global__ __launch_bounds__(256) void cache_append_kernel(const T *__restrict__ k, int64_t k_stride,
                                                           const T *__restrict__ v, int64_t v_stride, int64_t m,
                                                           const int32_t *__restrict__ cu, const int32_t *__restrict__ lens,
                                                           int seqs, const int32_t *__restrict__ table, int64_t max_blocks,
                                                           int8_t *__restrict__ k_codes, int8_t *__restrict__ v_codes,
                                                           float *__restrict__ k_scale, float *__restrict__ v_scale,
                                                           int64_t pages)
{
    constexpr int Q = D / 4;                       // 4-element pieces of a row
    constexpr int ITER = kBlock * Q / 256;         // pieces of K, and of V, that a thread may hold
    __shared__ __align__(16) uint32_t codes[2][kBlock][Q];
    __shared__ float red[2][4];
    SeqTile t;
    int64_t block;
    if (!find_block(cu, lens, seqs, m, max_blocks, blockIdx.x, t, block)) return;
    const int head = blockIdx.y, heads = gridDim.y, tid = threadIdx.x;
    const int64_t page = table[(int64_t)t.seq * max_blocks + block];  // waited for after the rows
    const int64_t have = lens[t.seq], t0 = block * kBlock;
    const int64_t lo = have > t0 ? have : t0, hi = have + t.n < t0 + kBlock ? have + t.n : t0 + kBlock;
    const int used = (int)(lo - t0), cnt = (int)(hi - lo), end = used + cnt;
    const int64_t row0 = t.begin + (lo - have);

    // x[0] is K, x[1] V: item i * 256 + tid is 4 elements of a row
    const int items = cnt * Q;
    T raw[2][ITER][4];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const T *src = (w ? v + row0 * v_stride : k + row0 * k_stride) + head * D;
        const int64_t stride = w ? v_stride : k_stride;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int it = i * 256 + tid;
            if (it >= items) continue;
            const T *at_row = src + (it / Q) * stride + it % Q * 4;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(raw[w][i]) = *reinterpret_cast<const float4 *>(at_row);
            else *reinterpret_cast<uint2 *>(raw[w][i]) = *reinterpret_cast<const uint2 *>(at_row);
        }
    }
    if (page < 0 || page >= pages) return;
    const int64_t at = page * heads + head;
    const float old_k = used ? k_scale[at] : 0.0f, old_v = used ? v_scale[at] : 0.0f;
    float x[2][ITER][4];
    uint32_t top[2] = {0, 0};  // largest magnitude as bits: NaN above inf above every number
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if (i * 256 + tid >= items) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[w][i][j] = to_f32(raw[w][i][j]);
                const uint32_t b = __float_as_uint(x[w][i][j]) & 0x7FFFFFFFu;
                top[w] = b > top[w] ? b : top[w];
            }
        }
    if (__any(top[0] > 0x7F7FFFFFu || top[1] > 0x7F7FFFFFu)) {
        top[0] = top[1] = 0;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                if (i * 256 + tid >= items) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f = x[w][i][j];
                    f = f == f ? fminf(fmaxf(f, -3.402823466e38f), 3.402823466e38f) : 0.0f;
                    x[w][i][j] = f;
                    const uint32_t b = __float_as_uint(f) & 0x7FFFFFFFu;
                    top[w] = b > top[w] ? b : top[w];
                }
            }
    }
    const float mk = wave_max(__uint_as_float(top[0])), mv = wave_max(__uint_as_float(top[1]));
    if ((tid & 63) == 0) {
        red[0][tid >> 6] = mk;
        red[1][tid >> 6] = mv;
    }
    __syncthreads();
    float sk = fmaxf(old_k, kSmallestScale), sv = fmaxf(old_v, kSmallestScale);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        sk = fmaxf(sk, red[0][w]);
        sv = fmaxf(sv, red[1][w]);
    }
    const float inv_k = 127.0f / sk, inv_v = 127.0f / sv;
    const float ratio_k = old_k / sk, ratio_v = old_v / sv;
    const bool grow_k = used && ratio_k != 1.0f, grow_v = used && ratio_v != 1.0f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float inv = w ? inv_v : inv_k;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int it = i * 256 + tid;
            if (it >= items) continue;
            codes[w][used + it / Q][it % Q] = pack_low_bytes(quant_bits(x[w][i][0], inv), quant_bits(x[w][i][1], inv),
                                                             quant_bits(x[w][i][2], inv), quant_bits(x[w][i][3], inv));
        }
    }
    __syncthreads();

    int8_t *kp = k_codes + at * (kBlock * D), *vp = v_codes + at * (kBlock * D);
    // K: 16 dims of a token are one 16-byte piece
    for (int it = tid; it < end * (D / 16); it += 256) {
        const int tok = it / (D / 16), j = it % (D / 16);
        uint4 *dst = reinterpret_cast<uint4 *>(kp + k_code_at<D>(tok, 16 * j));
        if (tok >= used) {
            *dst = *reinterpret_cast<const uint4 *>(&codes[0][tok][4 * j]);
        } else if (grow_k) {
            uint4 c = *dst;
            int8_t *b = reinterpret_cast<int8_t *>(&c);
#pragma unroll
            for (int i = 0; i < 16; ++i) b[i] = (int8_t)rescale_code(b[i], ratio_k);
            *dst = c;
        }
    }
    // V: 16 tokens of a dim are one piece. Groups of 16 new tokens: 4 dims per
    // thread, bytes transposed in registers
    const int full0 = (used + 15) / 16, full1 = end / 16;
    for (int it = tid; it < (full1 - full0) * Q; it += 256) {
        const int first = 16 * (full0 + it / Q), piece = it % Q;
        uint32_t o[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = codes[1][first + 4 * q + i][piece];
            const uint32_t a01 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), a23 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
            const uint32_t b01 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u), b23 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
            o[0][q] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
            o[1][q] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
            o[2][q] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
            o[3][q] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
            *reinterpret_cast<uint4 *>(vp + v_code_at(first, 4 * piece + d)) = make_uint4(o[d][0], o[d][1], o[d][2], o[d][3]);
    }
    // the others, at most one before and one behind unless the scale grew: a dim per thread,
    // of whose 16 codes those of [0, used) are rescaled, of [used, end) replaced, the rest kept
    const int g0 = grow_v ? 0 : used / 16, ng = (end + 15) / 16 - g0;
    for (int it = tid; it < ng * D; it += 256) {
        const int g = g0 + it / D, dim = it % D, first = 16 * g;
        if (g >= full0 && g < full1) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(vp + v_code_at(first, dim));
        uint4 c = *dst;
        int8_t *b = reinterpret_cast<int8_t *>(&c);
        const int8_t *fresh = reinterpret_cast<const int8_t *>(&codes[1][0][0]) + dim;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int tok = first + i;
            if (tok < used) {
                if (grow_v) b[i] = (int8_t)rescale_code(b[i], ratio_v);
            } else if (tok < end) {
                b[i] = fresh[tok * D];
            }
        }
        *dst = c;
    }
    if (tid == 0) {
        k_scale[at] = sk;
        v_scale[at] = sv;
    }
}

// One workgroup per (reached block, kv head). K leaves as 4 dims of a token per
// lane; V as 16 tokens of one dim per lane, 64 neighbouring dims per store. The
// stores pass the caches by, which keeps lines that are still to be read in them. With
// plain stores beside it, 8 heads of 128: 2000 tokens in fp32 read 7.1 / 8.4 us, read and
// then passed over once 15.1 / 16.6; 8195 tokens 15.5 / 16.1 and 34.1 / 32.3 (in bf16
// 11.2 / 12.1 and 27.1 / 23.2: those results would have stayed in the last-level cache);
// 16 x 3000 appended and read 211 / 245, read and passed over 211 / 211.
template <typename T, int D>
__global__ __launch_bounds__(256) void cache_read_kernel(const int8_t *__restrict__ k_codes,
                                                         const int8_t *__restrict__ v_codes,
                                                         const float *__restrict__ k_scale,
                                                         const float *__restrict__ v_scale, int64_t pages,
                                                         const int32_t *__restrict__ table, int64_t max_blocks,
                                                         const int32_t *__restrict__ cu, const int32_t *__restrict__ begin,
                                                         int seqs, int64_t m, T *__restrict__ k_out, T *__restrict__ v_out)
{
    SeqTile t;
    int64_t block;
    // blocks past the table hold no tokens but are still written (as 0)
    if (!find_block(cu, begin, seqs, m, (int64_t)1 << 40, blockIdx.x, t, block)) return;
    const int head = blockIdx.y, heads = gridDim.y, tid = threadIdx.x;
    const int64_t page = block < max_blocks ? table[(int64_t)t.seq * max_blocks + block] : -1;
    const bool there = page >= 0 && page < pages;
    const int64_t from = begin[t.seq], t0 = block * kBlock;
    const int64_t lo = from > t0 ? from : t0, hi = from + t.n < t0 + kBlock ? from + t.n : t0 + kBlock;
    const int used = (int)(lo - t0), cnt = (int)(hi - lo), end = used + cnt;
    const int64_t row0 = t.begin + (lo - from), at = there ? page * heads + head : 0;
    const float sk = there ? k_scale[at] / 127.0f : 0.0f, sv = there ? v_scale[at] / 127.0f : 0.0f;
    const int8_t *kp = k_codes + at * (kBlock * D), *vp = v_codes + at * (kBlock * D);

    for (int it = tid; it < cnt * (D / 4); it += 256) {
        const int tok = it / (D / 4), dim = it % (D / 4) * 4;
        const uint32_t c = there ? *reinterpret_cast<const uint32_t *>(kp + k_code_at<D>(used + tok, dim)) : 0;
        typedef T v4t __attribute__((ext_vector_type(4)));
        v4t o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (T)((float)(int8_t)(c >> (8 * i)) * sk);
        __builtin_nontemporal_store(o, reinterpret_cast<v4t *>(k_out + ((row0 + tok) * heads + head) * D + dim));
    }
    const int g0 = used / 16, ng = (end + 15) / 16 - g0;
    for (int it = tid; it < ng * D; it += 256) {
        const int first = 16 * (g0 + it / D), dim = it % D;
        uint4 c = make_uint4(0, 0, 0, 0);
        if (there) c = *reinterpret_cast<const uint4 *>(vp + v_code_at(first, dim));
        const int8_t *b = reinterpret_cast<const int8_t *>(&c);
        T *dst = v_out + ((row0 + first - used) * heads + head) * D + dim;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (first + i >= used && first + i < end) __builtin_nontemporal_store((T)((float)b[i] * sv), dst + (int64_t)i * heads * D);
    }
}

// ---------------------------------------------------------------- eviction
constexpr int kEvictThreads = 1024;

// One workgroup per sequence. The weight that the last kept block has is found by
// its digits from the top, 11, 11 and 10 bits (counts in LDS, integers, so the
// order does not matter), until a digit's count is all that is left to keep: two
// rounds for most. Then one pass in block order keeps everything above it, as many
// of its equals as are left, and compacts both lists by ballots. Latency-bound:
// 48 blocks 5.1 us, 64 x 2048 blocks 7.0 us (8-bit digits without the early end:
// 5.7 and 8.2).
__global__ __launch_bounds__(kEvictThreads) void cache_evict_kernel(
    const int32_t *__restrict__ table, const int32_t *__restrict__ lens, const float *__restrict__ weights,
    int64_t max_blocks, int64_t keep, int64_t first, int64_t recent, int32_t *__restrict__ table_out,
    int32_t *__restrict__ lens_out, float *__restrict__ weights_out, int32_t *__restrict__ evicted,
    int32_t *__restrict__ evicted_count, int first_seq)
{
    constexpr int W = kEvictThreads / 64, kBins = 2048;
    __shared__ int hist[kBins];
    __shared__ int wave_sums[W];
    __shared__ int pick[3];
    __shared__ int sums[2][2][W];
    const int s = first_seq + (int)blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = (int64_t)s * max_blocks;
    table += row; weights += row; table_out += row; weights_out += row; evicted += row;
    const int have = lens[s], wide = (int)max_blocks;
    const int64_t blocks = ((int64_t)have + kBlock - 1) / kBlock;
    const int used = have <= 0 ? 0 : blocks < wide ? (int)blocks : wide;
    const bool all = used <= keep;
    const int mid0 = all ? used : (int)first, mid1 = all ? used : (int)(used - recent);
    const int want = all ? 0 : (int)(keep - first - recent);

    // keys are compared without their lowest `shift` bits
    uint32_t prefix = 0;
    int shift = 32, left = want;  // of the blocks whose key begins with prefix, how many stay
    while (want > 0 && shift > 0) {
        const int bits = shift > 10 ? 11 : 10, down = shift - bits;
        hist[2 * tid] = 0;
        hist[2 * tid + 1] = 0;
        __syncthreads();
        for (int b = mid0 + tid; b < mid1; b += kEvictThreads) {
            const uint32_t key = weight_key(weights[b]);
            if (shift == 32 || key >> shift == prefix) atomicAdd(&hist[key >> down & ((1u << bits) - 1)], 1);
        }
        __syncthreads();
        // thread i has the i-th largest two digits; what lies above them
        const int top = (1 << bits) - 1 - 2 * tid;
        const int h0 = top >= 0 ? hist[top] : 0, h1 = top >= 0 ? hist[top - 1] : 0;
        int incl = h0 + h1;
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
        const int above = incl - h0 - h1;
        if (above < left && incl >= left) {
            const bool second = above + h0 < left;
            pick[0] = top - (second ? 1 : 0);
            pick[1] = left - above - (second ? h0 : 0);
            pick[2] = second ? h1 : h0;
        }
        __syncthreads();
        prefix = prefix << bits | (uint32_t)pick[0];
        left = pick[1];
        shift = down;
        if (pick[2] == left) break;  // all of them stay
    }

    int stay_at = 0, gone_at = 0, equal_at = 0;
    for (int b0 = 0, buf = 0; b0 < used; b0 += kEvictThreads, buf ^= 1) {
        const int b = b0 + tid;
        const bool in = b < used, mid = in && b >= mid0 && b < mid1;
        const float w = in ? weights[b] : 0.0f;
        const uint32_t key = want > 0 ? weight_key(w) >> shift : 0;
        const bool equal = mid && want > 0 && key == prefix;
        const uint64_t below = lane ? ~0ull >> (64 - lane) : 0;
        const uint64_t eq_mask = __ballot(equal);
        if (lane == 0) sums[buf][0][wave] = __popcll(eq_mask);
        __syncthreads();
        int eq = equal_at + __popcll(eq_mask & below);
        int eq_all = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < wave) eq += sums[buf][0][i];
            eq_all += sums[buf][0][i];
        }
        equal_at += eq_all;
        const bool stay = in && (!mid || (want > 0 && (key > prefix || (equal && eq < left))));
        const uint64_t stay_mask = __ballot(stay);
        if (lane == 0) sums[buf][1][wave] = __popcll(stay_mask);
        __syncthreads();
        int at = __popcll(stay_mask & below), before = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < wave) at += sums[buf][1][i];
            before += sums[buf][1][i];
        }
        if (stay) {
            table_out[stay_at + at] = table[b];
            weights_out[stay_at + at] = w;
        } else if (in) {
            evicted[gone_at + (tid - at)] = table[b];
        }
        const int here = used - b0 < kEvictThreads ? used - b0 : kEvictThreads;
        stay_at += before;
        gone_at += here - before;
    }
    for (int b = stay_at + tid; b < wide; b += kEvictThreads) {
        table_out[b] = -1;
        weights_out[b] = 0.0f;
    }
    for (int b = gone_at + tid; b < wide; b += kEvictThreads) evicted[b] = -1;
    if (tid == 0) {
        lens_out[s] = have - kBlock * gone_at;
        evicted_count[s] = gone_at;
    }
}

// ---------------------------------------------------------------- launchers

// touched blocks of a batch: at most n / 64 + 2 of a sequence with n rows
static int64_t most_blocks(const int32_t *cu, int64_t m, int64_t seqs) { return cu ? m / kBlock + 2 * seqs : seqs; }

hipError_t launch_cache_append(const CacheAppend &p, hipStream_t st)
{
    const dim3 grid((unsigned)most_blocks(p.cu, p.m, p.seqs), (unsigned)p.kv_heads);
    auto go = [&](auto type, auto width) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value;
        hipLaunchKernelGGL((cache_append_kernel<T, D>), grid, dim3(256), 0, st, static_cast<const T *>(p.k), p.k_stride,
                           static_cast<const T *>(p.v), p.v_stride, p.m, p.cu, p.lens, (int)p.seqs, p.table,
                           p.max_blocks, p.k_codes, p.v_codes, p.k_scale, p.v_scale, p.pages);
    };
    if (p.bf16) p.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
    else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    return hipGetLastError();
}

hipError_t launch_cache_read(const CacheRead &p, hipStream_t st)
{
    const dim3 grid((unsigned)most_blocks(p.cu, p.m, p.seqs), (unsigned)p.kv_heads);
    auto go = [&](auto type, auto width) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value;
        hipLaunchKernelGGL((cache_read_kernel<T, D>), grid, dim3(256), 0, st, p.k_codes, p.v_codes, p.k_scale, p.v_scale,
                           p.pages, p.table, p.max_blocks, p.cu, p.begin, (int)p.seqs, p.m,
                           static_cast<T *>(p.k_out), static_cast<T *>(p.v_out));
    };
    if (p.bf16) p.head_dim == 128 ? go(__bf16{}, Width<128>{}) : go(__bf16{}, Width<64>{});
    else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    return hipGetLastError();
}

hipError_t launch_cache_evict(const int32_t *table, const int32_t *lens, const float *weights, int64_t seqs,
                              int64_t max_blocks, int64_t keep, int64_t first, int64_t recent, int32_t *table_out,
                              int32_t *lens_out, float *weights_out, int32_t *evicted, int32_t *evicted_count,
                              hipStream_t st)
{
    in_launches(seqs, [&](int at, unsigned n) {
        hipLaunchKernelGGL(cache_evict_kernel, dim3(n), dim3(kEvictThreads), 0, st, table, lens, weights, max_blocks, keep,
                           first, recent, table_out, lens_out, weights_out, evicted, evicted_count, at);
    });
    return hipGetLastError();
}

}  // namespace bl
