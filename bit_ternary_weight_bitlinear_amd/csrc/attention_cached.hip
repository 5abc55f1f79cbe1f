// attention_cached.hip -- attention of new tokens over the 8-bit cache.
//
//   x_ij = scale * (q_i . kc_j) * (ks / 127),  p = softmax over the seen j,
//   out_i = sum_j p_ij * vc_j * (vs / 127)
//
// kc, vc are int8 codes and ks, vs one scale per page of 64 tokens. Both products
// run on v_mfma_i32_16x16x64_i8 with the codes as they lie in memory: q and p
// become three signed base-256 digits (23 bits and a sign, relative to the
// largest of the row of q, and to the page's largest p), so the codes need no
// conversion, the sums are exact integers, and the result is as good as fp32.
// The 16 rows of the first operand hold 4 query rows x (3 digits + a zero row):
// row 4j+i is digit i of query row j. The result's row 4j+i lies in register i of
// the lanes with lane / 16 = j, so a lane joins the digits of its own query row
// in registers, and all per-row state (maximum, sum, rescaling) is per lane.
//
// A page is one step of a wave: 8 KB of K, 8 KB of V (head_dim 128), each lane
// 16 bytes per load, every load of a wave contiguous. Bound by HBM for up to 16
// query rows a page: ~170 VALU operations and 16 matrix instructions per 16 KB
// and four query rows.
#include "attention.hpp"

namespace bl {

constexpr int kWaves = 4;
constexpr float kDigitMax = 8355711.0f;  // 0x7F7F7F: every digit within -128..127

// signed base-256 digits of an integer of at most kDigitMax: digit i in byte 0 of d[i]
__device__ inline void digits3(int n, int d[3])
{
    d[0] = n;
    const int n1 = (n - (int)(int8_t)n) >> 8;
    d[1] = n1;
    d[2] = (n1 - (int)(int8_t)n1) >> 8;
}

// digits' sums to one fp32 value
__device__ inline float join_digits(v4i c)
{
    return __builtin_fmaf((float)c[2], 65536.0f, __builtin_fmaf((float)c[1], 256.0f, (float)c[0]));
}

// How the pages of a sequence are split: in pages per workgroup. At least one for
// each of its waves, and at most `splits` workgroups.
__device__ inline int pages_per_split(int npages, int splits)
{
    const int c = (npages + splits - 1) / splits;
    return c < kWaves ? kWaves : c;
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
    int seqs, q_heads, kv_heads, group, splits, tiles_per_seq;
    int64_t max_blocks, pages;
    const int8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    float scale;      // of the logits, times log2 e
    void *out;
    float *part_o;    // [splits][m * q_heads][D]
    float *part_ml;   // [splits][m * q_heads][2]: reference exponent, sum
    float *stat;      // [m * q_heads][max_blocks][2]: a page's largest exponent, sum
};

// tiles of 4*RT query rows: row r of a sequence is token r / group, head r % group
template <int RT>
__device__ inline bool find_rows(const CachedArgs &a, int idx, SeqTile &t)
{
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

template <typename T, int D, int RT, bool STAT>
__global__ __launch_bounds__(64 * kWaves) void attention_cached_kernel(CachedArgs a)
{
    constexpr int H = D / 64;   // matrix steps over the head width
    constexpr int N = D / 16;   // 16-dim tiles of the output
    constexpr int R = 4 * RT;   // query rows
    // per wave: digits of p, [16 rows][16 dwords of 4 tokens]; the join at the end
    constexpr int kDigitWords = kWaves * RT * 256, kJoinWords = kWaves * R * (D + 2);
    __shared__ __align__(16) uint32_t lds[kDigitWords > kJoinWords ? kDigitWords : kJoinWords];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane >> 4, c = lane & 15;
    SeqTile t;
    if (!find_rows<RT>(a, blockIdx.x, t)) return;
    const int head = blockIdx.y, split = blockIdx.z;
    const int64_t have = a.lens[t.seq];
    const int npages = pages_of(have, t.n, a.max_blocks);
    const int chunk = pages_per_split(npages, a.splits);
    const int p0 = split * chunk, p1 = p0 + chunk < npages ? p0 + chunk : npages;
    if (p0 >= npages && split > 0) return;  // the join knows; split 0 writes rows that see nothing
    const int64_t rows = (int64_t)t.n * a.group;

    // ---- query rows as digits. Lane (j, c) builds row c of the operand: digit
    // c % 4 of query row c / 4, dims 16*j .. 16*j+15 of every 64.
    v4i qd[RT][H];
    float qs[RT];          // per lane of the result: scale of query row j
    int64_t limit[RT];     // last token that query row j sees (-1: none)
    bool poor[RT];         // query row j is not finite
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int64_t r = (int64_t)t.tile * R + 4 * rt + (c >> 2);
        const bool there = r < rows;
        const int tok = there ? (int)(r / a.group) : 0, hq = head * a.group + (there ? (int)(r % a.group) : 0);
        const T *src = static_cast<const T *>(a.q) + (t.begin + tok) * a.q_stride + (int64_t)hq * D + 16 * j;
        float x[H][16];
        float big = 0.0f;
        bool ok = true;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            T raw[16];
            constexpr int V = 16 * sizeof(T) / 16;
#pragma unroll
            for (int i = 0; i < V; ++i)
                reinterpret_cast<uint4 *>(raw)[i] = reinterpret_cast<const uint4 *>(src + 64 * h)[i];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[h][i] = there ? to_f32(raw[i]) : 0.0f;
                ok = ok && fabsf(x[h][i]) <= 3.402823466e38f;
                big = fmaxf(big, fabsf(x[h][i]));
            }
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        const uint64_t bad = __ballot(!ok);
        big = fmaxf(big, 1e-30f);
        const float inv = kDigitMax / fminf(big, 3.402823466e38f);
        const int digit = c & 3;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = x[h][4 * g + i];
                    int d[3];
                    digits3(ok ? (int)rintf(fminf(fmaxf(f * inv, -kDigitMax), kDigitMax)) : 0, d);
                    b[i] = digit == 0 ? d[0] : digit == 1 ? d[1] : digit == 2 ? d[2] : 0;
                }
                w[g] = pack_low_bytes(b[0], b[1], b[2], b[3]);
            }
            qd[rt][h] = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        }
        // the result's lane (j, c) has query row j: that is operand row 4j of lane 4j
        const float big_j = __shfl(big, 4 * j);
        qs[rt] = (big_j / kDigitMax) * a.scale;
        const int64_t rj = (int64_t)t.tile * R + 4 * rt + j;
        limit[rt] = rj < rows ? have + rj / a.group : -1;
        poor[rt] = (bad & (0x000F000F000F000Full << (4 * j))) != 0;
    }

    uint32_t *dig = lds + wave * RT * 256;
#pragma unroll
    for (int i = 0; i < RT * 4; ++i) dig[i * 64 + lane] = 0;  // row 4j+3 of every tile stays 0

    float mx[RT], sum[RT], acc[RT][N];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        mx[rt] = kNegInf;
        sum[rt] = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[rt][n] = 0.0f;
    }

    const int32_t *table = a.table + (int64_t)t.seq * a.max_blocks;
    for (int p = p0 + wave; p < p1; p += kWaves) {
        const int64_t id = table[p];
        const bool there = id >= 0 && id < a.pages;
        const int64_t at = (there ? id : 0) * a.kv_heads + head;
        const uint4 *kp = reinterpret_cast<const uint4 *>(a.k_codes + at * (kBlock * D)) + lane;
        const uint4 *vp = reinterpret_cast<const uint4 *>(a.v_codes + at * (kBlock * D)) + lane;
        v4i kf[4][H], vf[N];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int h = 0; h < H; ++h) kf[tt][h] = *reinterpret_cast<const v4i *>(kp + (tt * H + h) * 64);
#pragma unroll
        for (int n = 0; n < N; ++n) vf[n] = *reinterpret_cast<const v4i *>(vp + n * 64);
        const float ks = a.k_scale[at] / 127.0f, vs = a.v_scale[at] / 127.0f;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x[4];
            float big = kNegInf;
            const float f = qs[rt] * ks;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                v4i s = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < H; ++h) s = __builtin_amdgcn_mfma_i32_16x16x64_i8(qd[rt][h], kf[tt][h], s, 0, 0, 0);
                const bool seen = there && (int64_t)p * kBlock + 4 * c + tt <= limit[rt];
                x[tt] = seen ? join_digits(s) * f : kNegInf;
                big = fmaxf(big, x[tt]);
            }
            big = row16_max(big);
            const float ref = big == kNegInf ? 0.0f : big;
            float total = 0.0f;
            uint32_t b[4][3];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                const float e = __builtin_amdgcn_exp2f(x[tt] - ref);
                total += e;
                int d[3];
                digits3((int)rintf(e * kDigitMax), d);
                b[tt][0] = d[0];
                b[tt][1] = d[1];
                b[tt][2] = d[2];
            }
            total = row16_sum(total);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                dig[rt * 256 + (4 * j + i) * 16 + c] = pack_low_bytes(b[0][i], b[1][i], b[2][i], b[3][i]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const v4i pd = *reinterpret_cast<const v4i *>(&dig[rt * 256 + c * 16 + 4 * j]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (STAT && c == 0) {
                const int64_t rj = (int64_t)t.tile * R + 4 * rt + j;
                if (rj < rows) {
                    const int64_t row = (t.begin + rj / a.group) * a.q_heads + head * a.group + rj % a.group;
                    reinterpret_cast<float2 *>(a.stat)[row * a.max_blocks + p] = make_float2(big, poor[rt] ? 0.0f : total);
                }
            }
            const float now = fmaxf(mx[rt], big);
            const float base = now == kNegInf ? 0.0f : now;
            const float keep = __builtin_amdgcn_exp2f(mx[rt] - base), add = __builtin_amdgcn_exp2f(big - base);
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

    // ---- join the waves, in wave order
    __syncthreads();
    float *jo = reinterpret_cast<float *>(lds);              // [wave][row][D]
    float *jm = jo + kWaves * R * D;                         // [wave][row][2]
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
    for (int it = tid; it < R * D; it += 64 * kWaves) {
        const int r = it / D, dim = it % D;
        const int64_t rj = (int64_t)t.tile * R + r;
        if (rj >= rows) break;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, jm[2 * (w * R + r)]);
        const float base = top == kNegInf ? 0.0f : top;
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(jm[2 * (w * R + r)] - base);
            o = __builtin_fmaf(f, jo[(w * R + r) * D + dim], o);
            l = __builtin_fmaf(f, jm[2 * (w * R + r) + 1], l);
        }
        const int64_t row = (t.begin + rj / a.group) * a.q_heads + head * a.group + rj % a.group;
        if (a.splits > 1) {
            a.part_o[((int64_t)split * total_rows + row) * D + dim] = o;
        } else {
            store_out(static_cast<T *>(a.out) + row * D + dim, l == 0.0f ? 0.0f : o / l);
        }
        if (dim == 0 && a.part_ml) {
            a.part_ml[2 * ((int64_t)split * total_rows + row)] = top;
            a.part_ml[2 * ((int64_t)split * total_rows + row) + 1] = l;
        }
    }
}

// Joins the splits: one workgroup per query row, its waves take the splits in
// turn and meet in LDS.
template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves) void attention_join_kernel(CachedArgs a)
{
    constexpr int E = D / 64;
    __shared__ float jo[kWaves][D];
    __shared__ float jm[kWaves][2];
    SeqTile t;
    const int64_t row = blockIdx.x;
    const int tok = (int)(row / a.q_heads), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    const int npages = pages_of(have, t.n, a.max_blocks), chunk = pages_per_split(npages, a.splits);
    const int parts = npages <= chunk ? 1 : (npages + chunk - 1) / chunk;
    const int64_t total_rows = a.m * a.q_heads;
    float mx = kNegInf, l = 0.0f, o[E] = {};
    for (int s = wave; s < parts; s += kWaves) {
        const int64_t at = s * total_rows + row;
        const float pm = a.part_ml[2 * at], pl = a.part_ml[2 * at + 1];
        float po[E];
#pragma unroll
        for (int e = 0; e < E; ++e) po[e] = a.part_o[at * D + e * 64 + lane];
        const float now = fmaxf(mx, pm), base = now == kNegInf ? 0.0f : now;
        const float keep = __builtin_amdgcn_exp2f(mx - base), add = __builtin_amdgcn_exp2f(pm - base);
        mx = now;
        l = __builtin_fmaf(l, keep, pl * add);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(o[e], keep, po[e] * add);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) jo[wave][e * 64 + lane] = o[e];
    if (lane == 0) {
        jm[wave][0] = mx;
        jm[wave][1] = l;
    }
    __syncthreads();
    if ((int)threadIdx.x >= D) return;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, jm[w][0]);
    const float base = top == kNegInf ? 0.0f : top;
    float out = 0.0f, all = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(jm[w][0] - base);
        out = __builtin_fmaf(f, jo[w][threadIdx.x], out);
        all = __builtin_fmaf(f, jm[w][1], all);
    }
    store_out(static_cast<T *>(a.out) + row * D + threadIdx.x, all == 0.0f ? 0.0f : out / all);
}

// Adds each block's attention weight: one workgroup per sequence and 256 blocks.
// The rows' final exponents and sums are joined from the splits again (a few
// hundred values) rather than in a launch of their own.
__global__ __launch_bounds__(256) void attention_weights_kernel(CachedArgs a, float *__restrict__ weights)
{
    __shared__ float2 fin[64];
    const int s = blockIdx.x, tid = threadIdx.x;
    int64_t begin;
    int n;
    seq_rows(a.cu, s, a.m, begin, n);
    const int64_t have = a.lens[s];
    if (have < 0 || n == 0) return;
    const int npages = pages_of(have, n, a.max_blocks), chunk = pages_per_split(npages, a.splits);
    const int parts = npages <= chunk ? 1 : (npages + chunk - 1) / chunk;
    const int p = blockIdx.y * 256 + tid;
    if ((int)blockIdx.y * 256 >= npages) return;
    const int64_t total_rows = a.m * a.q_heads, row0 = begin * a.q_heads, rows = (int64_t)n * a.q_heads;
    float w = 0.0f;
    for (int64_t r0 = 0; r0 < rows; r0 += 64) {
        __syncthreads();
        // four threads of a quad share a row's splits
        const int64_t r = r0 + (tid >> 2);
        float mx = kNegInf, l = 0.0f;
        if (r < rows) {
            for (int i = tid & 3; i < parts; i += 4) {
                const int64_t at = i * total_rows + row0 + r;
                const float pm = a.part_ml[2 * at], pl = a.part_ml[2 * at + 1];
                const float now = fmaxf(mx, pm), base = now == kNegInf ? 0.0f : now;
                l = __builtin_fmaf(l, __builtin_amdgcn_exp2f(mx - base), pl * __builtin_amdgcn_exp2f(pm - base));
                mx = now;
            }
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            const float om = __shfl_xor(mx, d), ol = __shfl_xor(l, d);
            const float now = fmaxf(mx, om), base = now == kNegInf ? 0.0f : now;
            l = l * __builtin_amdgcn_exp2f(mx - base) + ol * __builtin_amdgcn_exp2f(om - base);
            mx = now;
        }
        // a row that is not finite, or sees nothing, adds nothing
        if ((tid & 3) == 0) fin[tid >> 2] = make_float2(mx, l > 0.0f ? 1.0f / l : 0.0f);
        __syncthreads();
        const int here = rows - r0 < 64 ? (int)(rows - r0) : 64;
        if (p < npages) {
            for (int i = 0; i < here; ++i) {
                const float2 st = reinterpret_cast<const float2 *>(a.stat)[(row0 + r0 + i) * a.max_blocks + p];
                const float2 f = fin[i];
                if (f.y > 0.0f && st.y > 0.0f) w = __builtin_fmaf(st.y * f.y, __builtin_amdgcn_exp2f(st.x - f.x), w);
            }
        }
    }
    if (p < npages) weights[(int64_t)s * a.max_blocks + p] += w;
}

// ---------------------------------------------------------------- launcher

// query rows per workgroup: 4, 8 or 16, as many as one token's group needs; more
// tokens at once use 16
static int row_tiles(bool one_token, int64_t group) { return one_token && group <= 4 ? 1 : one_token && group <= 8 ? 2 : 4; }

static int64_t query_tiles(const CachedProblem &p, int rt)
{
    const int64_t group = p.q_heads / p.kv_heads, r = 4 * rt;
    return p.packed ? p.m * group / r + p.seqs : p.seqs * ceil_div(group, r);
}

// Workgroups wanted: four per CU, so that 16 waves of a CU keep their pages in
// flight. Splits beyond one page per wave would stay empty.
constexpr int64_t kWantedGroups = 1024;
static int64_t split_count(const CachedProblem &p, int rt)
{
    const int64_t units = query_tiles(p, rt) * p.kv_heads;
    const int64_t most = ceil_div(p.max_blocks, kWaves);
    int64_t s = kWantedGroups / units;
    if (s > most) s = most;
    if (s > 256) s = 256;
    return s < 1 ? 1 : s;
}

struct CachedLayout {
    int64_t part_o, part_ml, stat, bytes;
};
static CachedLayout cached_layout(const CachedProblem &p)
{
    const int64_t splits = split_count(p, row_tiles(!p.packed, p.q_heads / p.kv_heads)), rows = p.m * p.q_heads;
    CachedLayout L{};
    int64_t off = 0;
    if (splits > 1) off += round_up(splits * rows * p.head_dim * 4, 256);
    L.part_ml = off;
    if (splits > 1 || p.want_weights) off += round_up(splits * rows * 8, 256);
    L.stat = off;
    if (p.want_weights) off += round_up(rows * p.max_blocks * 8, 256);
    L.bytes = off;
    return L;
}

int64_t attention_cached_workspace(const CachedProblem &p) { return cached_layout(p).bytes; }

hipError_t launch_attention_cached(const CachedProblem &p, void *ws, hipStream_t st)
{
    const int64_t group = p.q_heads / p.kv_heads;
    const int rt = row_tiles(!p.packed, group);
    const CachedLayout L = cached_layout(p);
    char *base = static_cast<char *>(ws);
    CachedArgs a{};
    a.q = p.q; a.q_stride = p.q_stride; a.m = p.m;
    a.cu = p.cu; a.lens = p.lens; a.table = p.table;
    a.seqs = (int)p.seqs; a.q_heads = (int)p.q_heads; a.kv_heads = (int)p.kv_heads; a.group = (int)group;
    a.splits = (int)split_count(p, rt);
    a.tiles_per_seq = (int)ceil_div(group, 4 * rt);
    a.max_blocks = p.max_blocks; a.pages = p.pages;
    a.k_codes = p.k_codes; a.v_codes = p.v_codes; a.k_scale = p.k_scale; a.v_scale = p.v_scale;
    a.scale = p.scale * kLog2e; a.out = p.out;
    a.part_o = a.splits > 1 ? reinterpret_cast<float *>(base) : nullptr;
    a.part_ml = a.splits > 1 || p.weights ? reinterpret_cast<float *>(base + L.part_ml) : nullptr;
    a.stat = p.weights ? reinterpret_cast<float *>(base + L.stat) : nullptr;

    const dim3 grid((unsigned)query_tiles(p, rt), (unsigned)p.kv_heads, (unsigned)a.splits);
    auto go = [&](auto type, auto width, auto tiles) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value, RT = decltype(tiles)::value;
        if (p.weights) hipLaunchKernelGGL((attention_cached_kernel<T, D, RT, true>), grid, dim3(64 * kWaves), 0, st, a);
        else hipLaunchKernelGGL((attention_cached_kernel<T, D, RT, false>), grid, dim3(64 * kWaves), 0, st, a);
        if (a.splits > 1)
            hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3((unsigned)(p.m * p.q_heads)), dim3(64 * kWaves), 0, st, a);
    };
    auto go_rt = [&](auto type, auto width) {
        if (rt == 1) go(type, width, Width<1>{});
        else if (rt == 2) go(type, width, Width<2>{});
        else go(type, width, Width<4>{});
    };
    if (p.bf16) p.head_dim == 128 ? go_rt(bf16_t{}, Width<128>{}) : go_rt(bf16_t{}, Width<64>{});
    else p.head_dim == 128 ? go_rt(float{}, Width<128>{}) : go_rt(float{}, Width<64>{});
    if (p.weights)
        hipLaunchKernelGGL(attention_weights_kernel, dim3((unsigned)p.seqs, (unsigned)ceil_div(p.max_blocks, 256)),
                           dim3(256), 0, st, a, p.weights);
    return hipGetLastError();
}

}  // namespace bl
