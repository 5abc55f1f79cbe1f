// rotate.hip -- rotation of queries and keys by their tokens' positions, with an RMS
// norm of every head before it.
//
//   x^ = (x * r) * gain,  r = 1 / sqrt(mean_d x^2 + eps)          (where a gain is given)
//   (a, b) -> magnitude * (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i]
//
// for the pairs i of the head's first rotary_dim elements; the others pass. A wave works on
// one token: its 64 lanes compute the token's angles once, for all of its heads, and exchange
// the cosines and sines through LDS; a lane then holds the same two 16-byte pieces of every
// head that it gets, both elements of each pair among them, so a norm is one reduction over 4
// to 16 neighbouring lanes and a rotation none.
//
// The angle in 64 bits: the product of a position and an fp32 frequency by its rounded value
// and the remainder, less the multiple of pi / 2 next to it (two constants, 106 bits of
// pi / 2), so positions up to 2^31 cost no digits; its cosine and sine are rounded to fp32.
//
// Bound by HBM with many tokens: 8192 of 32/8 heads of 128 in bf16, normed, 168 MB in 31 us
// (5.4 TB/s; without the next round's heads on their way and one set of gains for both sides
// 5 % more), by a launch and its chain of loads with few: one token 2.7 us on the device, 192 tokens
// of 20/5 heads in fp32 3.9 (a wave per round of heads there; a call takes 5.4). The loads pass the caches by, which
// keep what is stored for the append and the attention that read it: 31.1 us beside 36.6 with
// plain loads, with an append behind it 45.2 beside 46.3 (with stores that pass them by too 50.5).
#include "attention.hpp"

namespace bl {

struct RotateArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride, m;
    int q_heads, kv_heads, seqs, pairs;  // pairs: rotary_dim / 2
    const int32_t *cu, *begin;
    const float *inv_freq, *q_gain, *k_gain;
    float eps, magnitude;
    int parts;  // waves per token
};

// Cosine and sine of position * freq: Taylor's series to r^14 and r^15 on |r| <= pi / 4 (the
// cosine's next term is 1.0e-15, the sine's 5e-17; beside exact values both are off by at most
// 1e-15 up to |t| = 2^45 and by 1.4e-14 up to 2^50), rounded to fp32 once.
__device__ inline float2 turn(int64_t position, float freq)
{
    const double p = (double)position, f = freq, t = p * f, rest = __builtin_fma(p, f, -t);
    const double n = __builtin_rint(t * 0.6366197723675814);  // 2 / pi
    double r = __builtin_fma(n, -1.5707963267948966, t);
    r = __builtin_fma(n, -6.123233995736766e-17, r) + rest;
    const double z = r * r;
    double s = -1.0 / 1307674368000.0, c = -1.0 / 87178291200.0;
    s = __builtin_fma(s, z, 1.0 / 6227020800.0);
    c = __builtin_fma(c, z, 1.0 / 479001600.0);
    s = __builtin_fma(s, z, -1.0 / 39916800.0);
    c = __builtin_fma(c, z, -1.0 / 3628800.0);
    s = __builtin_fma(s, z, 1.0 / 362880.0);
    c = __builtin_fma(c, z, 1.0 / 40320.0);
    s = __builtin_fma(s, z, -1.0 / 5040.0);
    c = __builtin_fma(c, z, -1.0 / 720.0);
    s = __builtin_fma(s, z, 1.0 / 120.0);
    c = __builtin_fma(c, z, 1.0 / 24.0);
    s = __builtin_fma(s, z, -1.0 / 6.0);
    c = __builtin_fma(c, z, -0.5);
    const float sine = (float)__builtin_fma(s * z, r, r), cosine = (float)__builtin_fma(c, z, 1.0);
    const int quarter = (int)(long long)n & 3;
    const float a = quarter & 1 ? sine : cosine, b = quarter & 1 ? cosine : sine;
    return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// 1 / sqrt(v): the hardware's (1 ulp) and a step of Newton's; by its definition in lanes whose v
// may be below the numbers that the hardware takes, or is none (a head's bits do not depend on
// another's)
__device__ inline float inverse_root(float v)
{
    const float r = __builtin_amdgcn_rsqf(v);
    const float fine = __builtin_fmaf(0.5f * r, __builtin_fmaf(-v * r, r, 1.0f), r);
    const bool usual = v >= 1e-30f && v <= 1e38f;
    if (__any(!usual)) return usual ? fine : 1.0f / sqrtf(v);
    return fine;
}

template <typename T, int D, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotate_kernel(RotateArgs a, int first)
{
    constexpr int E = 16 / sizeof(T);  // elements of a piece
    constexpr int LANES = D / (2 * E);  // of a head
    constexpr int HEADS = 64 / LANES;   // of a wave at once: a round
    __shared__ __align__(16) float2 turns[4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t item = ((int64_t)first + blockIdx.x) * 4 + wave;
    const int64_t row = item / a.parts;
    const int part = (int)(item - row * a.parts);
    if (row >= a.m) return;
    const int slot = lane % LANES;
    const bool rotary = slot * E < a.pairs;
    // elements of a lane: `lo` .. lo+E-1 and `hi` .. hi+E-1 of the head
    const int lo = INTERLEAVED ? 2 * E * slot : rotary ? E * slot : 2 * E * slot;
    const int hi = INTERLEAVED ? lo + E : rotary ? a.pairs + lo : lo + E;

    // rounds 0 .. q_rounds-1 are of q, the others of k; a round is on its way while the one before is worked on
    const int q_rounds = (a.q_heads + HEADS - 1) / HEADS, rounds = q_rounds + (a.kv_heads + HEADS - 1) / HEADS;
    struct Round {
        int head;
        bool is_q, there;
        uint4 lo, hi;
    };
    auto load = [&](int i) {
        Round r;
        r.is_q = i < q_rounds;
        r.head = (r.is_q ? i : i - q_rounds) * HEADS + lane / LANES;
        r.there = r.head < (r.is_q ? a.q_heads : a.kv_heads);
        r.lo = r.hi = make_uint4(0, 0, 0, 0);
        if (r.there) {
            const T *src = static_cast<const T *>(r.is_q ? a.q : a.k) + row * (r.is_q ? a.q_stride : a.k_stride) + (int64_t)r.head * D;
            r.lo = load_nt16(src + lo);
            r.hi = load_nt16(src + hi);
        }
        return r;
    };
    Round next = load(part);

    int seq, place, begin;
    if (!find_row(a.cu, a.begin, a.seqs, a.m, row, seq, place, begin) || begin < 0) return;  // negative: an unused slot
    if (lane < a.pairs) {
        const float2 t = turn((int64_t)begin + place, a.inv_freq[lane]);
        turns[wave][lane] = make_float2(t.x * a.magnitude, t.y * a.magnitude);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    float co[E], si[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float2 t = rotary ? turns[wave][slot * E + i] : make_float2(1.0f, 0.0f);
        co[i] = t.x;
        si[i] = t.y;
    }

    float gain[2 * E];
    const float *held = nullptr;  // whose elements `gain` has
    for (int i = part; i < rounds; i += a.parts) {
        const Round r = next;
        if (i + a.parts < rounds) next = load(i + a.parts);
        const float *g = r.is_q ? a.q_gain : a.k_gain;
        if (g && g != held) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                *reinterpret_cast<v4f *>(gain + e) = *reinterpret_cast<const v4f *>(g + lo + e);
                *reinterpret_cast<v4f *>(gain + E + e) = *reinterpret_cast<const v4f *>(g + hi + e);
            }
            held = g;
        }
        T x[2 * E];
        *reinterpret_cast<uint4 *>(x) = r.lo;
        *reinterpret_cast<uint4 *>(x + E) = r.hi;
        float f[2 * E];
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) f[e] = to_f32(x[e]);
        if (g) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
            ss += __int_as_float(dpp_mov<kDppQuadXor1>(__float_as_int(ss)));
            ss += __int_as_float(dpp_mov<kDppQuadXor2>(__float_as_int(ss)));
            if constexpr (LANES >= 8) ss += __int_as_float(dpp_mov<kDppRowHalfMirror>(__float_as_int(ss)));
            if constexpr (LANES >= 16) ss += __int_as_float(dpp_mov<kDppRowMirror>(__float_as_int(ss)));
            const float s = inverse_root(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) f[e] = (f[e] * s) * gain[e];
        }
        if (rotary) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float &u = f[INTERLEAVED ? 2 * e : e], &v = f[INTERLEAVED ? 2 * e + 1 : E + e];
                const float a0 = u, b0 = v;
                u = __builtin_fmaf(a0, co[e], -(b0 * si[e]));
                v = __builtin_fmaf(b0, co[e], a0 * si[e]);
            }
        }
        if (!r.there) continue;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) store_out(&x[e], f[e]);
        T *dst = static_cast<T *>(r.is_q ? a.q_out : a.k_out) + row * (r.is_q ? a.q_out_stride : a.k_out_stride) + (int64_t)r.head * D;
        *reinterpret_cast<uint4 *>(dst + lo) = *reinterpret_cast<const uint4 *>(x);
        *reinterpret_cast<uint4 *>(dst + hi) = *reinterpret_cast<const uint4 *>(x + E);
    }
}

hipError_t launch_rotate(const RotateProblem &p, hipStream_t st)
{
    RotateArgs a{};
    a.q = p.q; a.k = p.k; a.q_out = p.q_out; a.k_out = p.k_out;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.q_out_stride = p.q_out_stride; a.k_out_stride = p.k_out_stride;
    a.m = p.m; a.q_heads = (int)p.q_heads; a.kv_heads = (int)p.kv_heads; a.seqs = (int)p.seqs; a.pairs = (int)p.rotary_dim / 2;
    a.cu = p.cu; a.begin = p.begin; a.inv_freq = p.inv_freq; a.q_gain = p.q_gain; a.k_gain = p.k_gain;
    a.eps = p.eps; a.magnitude = p.magnitude;
    // Few tokens: a wave for every round of heads, and otherwise one for a token's. On the device,
    // normed, of 5 rounds (32/8 heads of 128 in bf16) 64 tokens take 3.1 us with a wave for each and 5.7
    // without, 512 tokens 4.3 and 6.3, 2048 tokens 13.8 and 14.2, 3000 18.4 and 17.0, 4096 22.4 and 19.8;
    // of 7 (20/5 heads in fp32) 512 tokens 4.6 and 8.1, 2048 14.5 and 17.2, 4096 26.0 and 25.0
    const int64_t per_round = 64 * 32 / (p.head_dim * (p.bf16 ? 2 : 4));
    const int64_t rounds = ceil_div(p.q_heads, per_round) + ceil_div(p.kv_heads, per_round);
    a.parts = p.m * rounds <= 12000 ? (int)rounds : 1;
    in_launches(ceil_div(p.m * a.parts, 4), [&](int first, unsigned n) {
        auto go = [&](auto type, auto width) {
            using T = decltype(type);
            constexpr int D = decltype(width)::value;
            if (p.interleaved) hipLaunchKernelGGL((rotate_kernel<T, D, true>), dim3(n), dim3(256), 0, st, a, first);
            else hipLaunchKernelGGL((rotate_kernel<T, D, false>), dim3(n), dim3(256), 0, st, a, first);
        };
        if (p.bf16) p.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
        else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    });
    return hipGetLastError();
}

}  // namespace bl
