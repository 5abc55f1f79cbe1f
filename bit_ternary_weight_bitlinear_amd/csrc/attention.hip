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

int64_t attention_workspace(const AttentionProblem &) { return 0; }

hipError_t launch_attention(const AttentionProblem &p, void *, hipStream_t st)
{
    const dim3 grid((unsigned)p.m, (unsigned)p.q_heads);
    auto go = [&](auto type, auto width) {
        using T = decltype(type);
        constexpr int D = decltype(width)::value;
        hipLaunchKernelGGL((attention_kernel<T, D>), grid, dim3(64), 0, st, p);
    };
    if (p.bf16) p.head_dim == 128 ? go(bf16_t{}, Width<128>{}) : go(bf16_t{}, Width<64>{});
    else p.head_dim == 128 ? go(float{}, Width<128>{}) : go(float{}, Width<64>{});
    return hipGetLastError();
}

}  // namespace bl
