// attention_shared.hip -- attention of new tokens over a prefix that the whole batch
// shares and over each sequence's own cache behind it.
//
// A softmax over the two together is their results joined by their maxima and sums, so
// the prefix is read once for all sequences: their query rows of a kv head, m * group of
// them, are the rows of one matrix product with it. The kernel here writes the prefix's
// parts (maximum, sum and sum of values of every row), attention_cached_kernel adds them
// to the results of the sequences' own pages as it stores them, or the joining launch
// does where those come in parts too.
//
// With 32 query rows a wave the arithmetic counts, not the bytes, so here the codes meet
// the queries as fp16, on v_mfma_f32_32x32x16_f16: a code is an integer and exact, a row of
// q times a power of two that puts its largest at 2^14 to 2^15 is exact in fp16 for bf16
// elements down to 2^-31 of the largest, and in two fp16 parts good to 2^-22 for fp32
// (elements below 2^-17 of the largest: to 2^-39 of that). Weights are relative to a power
// of two at or above their page's and row's largest, times 2^15: rounded to fp16 (2^-11)
// for bf16 results, in two parts (2^-22) for fp32 ones. Sums are fp32, a page's scaled by
// its V scale when they are added to the row's.
//
// Layout: S^T = K Q^T has a query row per lane and 32 of a page's 64 tokens in its two
// times 16 registers, which after the exponential are the second operand of O^T = V^T P^T
// as they lie: the product's order of tokens is free, so row rho of a K operand is token
//   16 * bit 2 + 8 * bit 4 + 4 * bit 3 + (bits 1, 0) of rho
// of its 32, which gives a lane half h the 16 tokens that one 16-byte piece of V holds. The
// dims of the first product are ordered likewise by 16-byte pieces of K.
#include "attention_cached.hpp"

namespace bl {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kPrefixRows = 32, kPrefixWaves = 4;

struct PrefixArgs {
    const void *q;
    int64_t q_stride, rows;  // rows of a kv head: m * group
    int q_heads, kv_heads, group, splits;
    const int32_t *table, *len;
    int64_t blocks, pages, total_rows;
    const int8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    float scale;  // of the logits, times log2 e
    float *part_o, *part_ml;
};

// eight codes as fp16: 1024 + (code + 128) is the bits 0x6400 with the biased code in the low byte
__device__ inline v8h codes_f16(uint32_t lo, uint32_t hi)
{
    union {
        uint32_t w[4];
        v2h h[4];
        v8h v;
    } u;
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    u.w[0] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u);
    u.w[1] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u);
    u.w[2] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u);
    u.w[3] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u);
    const v2h bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) u.h[i] += bias;
    return u.v;
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kPrefixWaves) void attention_prefix_kernel(PrefixArgs a, int first_tile)
{
    constexpr int W = kPrefixWaves, R = kPrefixRows;
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    constexpr int U = D / 32;      // pairs of 16-dim pieces of K; 32-dim tiles of the output
    constexpr int E = D / 8;       // elements of a query row per thread
    constexpr int kStride = D + 4;  // of a row in the join
    constexpr int kQueryHalfs = PARTS * U * 2 * 64 * 8, kJoinFloats = W * R * kStride;
    __shared__ __align__(16) char lds[kQueryHalfs * 2 > kJoinFloats * 4 ? kQueryHalfs * 2 : kJoinFloats * 4];
    __shared__ float row_scale[R];
    __shared__ float2 jm[W][R];
    _Float16 *qh = reinterpret_cast<_Float16 *>(lds);  // [part][2 * pair + s][lane][8], in operand order

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int head = blockIdx.y, split = blockIdx.x;
    const int64_t row0 = ((int64_t)first_tile + blockIdx.z) * R;
    const int len = *a.len, npages = prefix_pages(a.len, a.blocks);
    const int chunk = pages_per_split(npages, a.splits, W);
    const int p0 = split * chunk, p1 = p0 + chunk < npages ? p0 + chunk : npages;
    if (p0 >= npages) return;  // the join knows

    // ---- query rows as fp16, eight threads a row
    {
        const int r = tid >> 3, c = tid & 7;
        const bool there = row0 + r < a.rows;
        const int64_t row = there ? row0 + r : 0;
        const int64_t tok = row / a.group;
        const int hq = head * a.group + (int)(row - tok * a.group);
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
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            big = fmaxf(big, __shfl_xor(big, d));
            bad = fmaxf(bad, __shfl_xor(bad, d));
        }
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
        if (c == 0) row_scale[r] = bad > 0.0f ? __builtin_nanf("") : __uint_as_float((uint32_t)(127 - e) << 23) * fabsf(a.scale);
    }
    __syncthreads();
    const float qs_raw = row_scale[col];
    const bool poor = !(qs_raw == qs_raw);
    const float qs = poor ? 0.0f : qs_raw;

    float top = kNegInf, sum = 0.0f;
    v16f acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[u][i] = 0.0f;

    // place of this lane's K row in its 32 tokens, and of its pieces in a page and head
    const int token = 16 * (col >> 2 & 1) + 8 * (col >> 4) + 4 * (col >> 3 & 1) + (col & 3);
    const int k_at = k_code_at<D>(token, 16 * half);
    const int v_at = v_code_at(16 * half, col);

    for (int base = p0 + wave; base < p1; base += 64 * W) {
        const int mine = base + W * lane;
        const int ids = mine < p1 ? a.table[mine] : -1;
        const bool ok = ids >= 0 && ids < a.pages;
        const int64_t my_at = ok ? (int64_t)ids * a.kv_heads + head : 0;
        const float my_ks = ok ? a.k_scale[my_at] : 0.0f, my_vs = ok ? a.v_scale[my_at] : 0.0f;
        for (int p = base, i = 0; p < p1 && i < 64; p += W, ++i) {
            const int id = __builtin_amdgcn_readlane(ids, i);
            if (id < 0 || id >= a.pages) continue;  // a block without a page holds no tokens
            const int64_t at = ((int64_t)id * a.kv_heads + head) * (kBlock * D);
            const int8_t *kp = a.k_codes + at + k_at, *vp = a.v_codes + at + v_at;
            uint4 kf[2][U], vf[U][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = 0; u < U; ++u) kf[t][u] = *reinterpret_cast<const uint4 *>(kp + t * 8 * 16 + u * 2 * 256);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) vf[u][t] = *reinterpret_cast<const uint4 *>(vp + (u * 2 * 4 + t * 2) * 256);
            const float ks = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_ks), i)) / 127.0f;
            const float vs = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_vs), i)) / 127.0f;

            v16f s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const v8h q0 = *reinterpret_cast<const v8h *>(qh + ((u * 2 + b) * 64 + lane) * 8);
                    v8h q1;
                    if constexpr (PARTS == 2) q1 = *reinterpret_cast<const v8h *>(qh + ((U * 2 + u * 2 + b) * 64 + lane) * 8);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const v8h k8 = b ? codes_f16(kf[t][u].z, kf[t][u].w) : codes_f16(kf[t][u].x, kf[t][u].y);
                        if constexpr (PARTS == 2) s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, q1, s[t], 0, 0, 0);
                        s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k8, q0, s[t], 0, 0, 0);
                    }
                }

            // register r of tile t is token 32 t + 16 half + r
            const float f = qs * ks;  // not negative: the sign of the scale is in q
            const int left = len - p * kBlock;
            float big = kNegInf;
            if (left >= kBlock) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) big = fmaxf(big, s[t][r]);
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (32 * t + 16 * half + r < left) big = fmaxf(big, s[t][r]);
            }
            big = fmaxf(big, __shfl_xor(big, 32));
            // raised by more than the rounding of its difference to 15, so that no weight passes 2^15
            const float ref = ceilf(__builtin_fmaf(fabsf(big * f), 0x1p-22f, big * f)), shift = 15.0f - ref;
            float total = 0.0f;
            v8h ph[2][2], pl[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], f, shift));
                    if (left < kBlock && 32 * t + 16 * half + r >= left) w = 0.0f;
                    total += w;
                    const _Float16 w16 = (_Float16)w;
                    ph[t][r >> 3][r & 7] = w16;
                    if constexpr (PARTS == 2) pl[t][r >> 3][r & 7] = (_Float16)(w - (float)w16);
                }
            total += __shfl_xor(total, 32);
            const float now = fmaxf(top, ref);
            const float keep = __builtin_amdgcn_exp2f(top - now), add = __builtin_amdgcn_exp2f(ref - now) * 0x1p-15f;
            top = now;
            sum = __builtin_fmaf(sum, keep, total * add);
            const float g = add * vs;
            const bool same = !__any(keep != 1.0f);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v16f o;
#pragma unroll
                for (int r = 0; r < 16; ++r) o[r] = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const v8h v8 = b ? codes_f16(vf[u][t].z, vf[u][t].w) : codes_f16(vf[u][t].x, vf[u][t].y);
                        if constexpr (PARTS == 2) o = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, pl[t][b], o, 0, 0, 0);
                        o = __builtin_amdgcn_mfma_f32_32x32x16_f16(v8, ph[t][b], o, 0, 0, 0);
                    }
                if (same) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[u][r] = __builtin_fmaf(o[r], g, acc[u][r]);
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[u][r] = __builtin_fmaf(o[r], g, acc[u][r] * keep);
                }
            }
        }
    }

    // ---- join the waves, in wave order
    __syncthreads();
    float *jo = reinterpret_cast<float *>(lds);  // [wave][row][kStride]
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            *reinterpret_cast<v4f *>(jo + (wave * R + col) * kStride + 32 * u + 2 * r + 4 * half) =
                v4f{acc[u][r], acc[u][r + 1], acc[u][r + 2], acc[u][r + 3]};
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
        const int64_t tok = (row0 + r) / a.group;
        const int64_t row = tok * a.q_heads + head * a.group + (row0 + r - tok * a.group);
        *reinterpret_cast<v4f *>(a.part_o + ((int64_t)split * a.total_rows + row) * D + dim) = o;
        if (dim == 0) reinterpret_cast<float2 *>(a.part_ml)[(int64_t)split * a.total_rows + row] = make_float2(best, l);
    }
}

// ---------------------------------------------------------------- launcher

// Workgroups per tile of 32 rows and kv head: two per CU in all, but at least a page per wave
static int64_t prefix_splits(const SharedProblem &p)
{
    const int64_t units = ceil_div(p.c.m * (p.c.q_heads / p.c.kv_heads), kPrefixRows) * p.c.kv_heads;
    const int64_t most = ceil_div(p.prefix_blocks, kPrefixWaves);
    int64_t s = 512 / units;
    s = s > most ? most : s;
    return s < 1 ? 1 : s > 256 ? 256 : s;
}

struct SharedLayout {
    int64_t part_ml, own_o, own_ml, bytes;
};
static SharedLayout shared_layout(const SharedProblem &p)
{
    const int64_t splits = launch_shape(p.c, row_tiles(p.c)).splits, before = prefix_splits(p), rows = p.c.m * p.c.q_heads;
    SharedLayout L{};
    L.part_ml = round_up(before * rows * p.c.head_dim * 4, 256);
    L.own_o = L.part_ml + round_up(before * rows * 8, 256);
    L.own_ml = L.own_o + (splits > 1 ? round_up(splits * rows * p.c.head_dim * 4, 256) : 0);
    L.bytes = L.own_ml + (splits > 1 ? round_up(splits * rows * 8, 256) : 0);
    return L;
}

int64_t attention_shared_workspace(const SharedProblem &p) { return shared_layout(p).bytes; }

hipError_t launch_attention_shared(const SharedProblem &p, void *ws, hipStream_t st)
{
    const CachedProblem &c = p.c;
    const int rt = row_tiles(c);
    const Shape shape = launch_shape(c, rt);
    const SharedLayout L = shared_layout(p);
    char *base = static_cast<char *>(ws);
    PrefixArgs f{};
    f.q = c.q; f.q_stride = c.q_stride; f.group = (int)(c.q_heads / c.kv_heads); f.rows = c.m * f.group;
    f.q_heads = (int)c.q_heads; f.kv_heads = (int)c.kv_heads; f.splits = (int)prefix_splits(p);
    f.table = p.prefix_table; f.len = p.prefix_len; f.blocks = p.prefix_blocks; f.pages = c.pages; f.total_rows = c.m * c.q_heads;
    f.k_codes = c.k_codes; f.v_codes = c.v_codes; f.k_scale = c.k_scale; f.v_scale = c.v_scale; f.scale = c.scale * kLog2e;
    f.part_o = reinterpret_cast<float *>(base);
    f.part_ml = reinterpret_cast<float *>(base + L.part_ml);
    in_launches(ceil_div(f.rows, kPrefixRows), [&](int first, unsigned n) {
        const dim3 grid((unsigned)f.splits, (unsigned)c.kv_heads, n), threads(64 * kPrefixWaves);
        auto go = [&](auto type) {
            using T = decltype(type);
            if (c.head_dim == 128) hipLaunchKernelGGL((attention_prefix_kernel<T, 128>), grid, threads, 0, st, f, first);
            else hipLaunchKernelGGL((attention_prefix_kernel<T, 64>), grid, threads, 0, st, f, first);
        };
        c.bf16 ? go(bf16_t{}) : go(float{});
    }, kMostInZ);

    CachedArgs a = cached_args(c, shape, rt);
    a.prefix_o = f.part_o; a.prefix_ml = f.part_ml; a.prefix_len = p.prefix_len; a.prefix_blocks = p.prefix_blocks;
    a.prefix_splits = f.splits; a.prefix_waves = kPrefixWaves;
    if (a.splits > 1) {
        a.part_o = reinterpret_cast<float *>(base + L.own_o);
        a.part_ml = reinterpret_cast<float *>(base + L.own_ml);
    }
    launch_tiles<kBehindPrefix>(c, a, shape, rt, query_tiles(c, rt), a.splits + f.splits, st);
    return hipGetLastError();
}

}  // namespace bl
