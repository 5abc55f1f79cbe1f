// attention.hpp -- device helpers shared by the attention and cache kernels.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace bl {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.4426950408889634f;

// A sequence's rows in a packed batch, and which of its tiles a workgroup has.
struct SeqTile {
    int seq, tile;
    int64_t begin;  // first row
    int n;          // rows
};

// Rows of sequence s (values outside 0..m taken as the nearest of the two).
__device__ inline void seq_rows(const int32_t *cu, int s, int64_t m, int64_t &begin, int &n)
{
    if (!cu) {
        begin = s;
        n = 1;
        return;
    }
    int64_t a = cu[s], b = cu[s + 1];
    a = a < 0 ? 0 : a > m ? m : a;
    b = b < a ? a : b > m ? m : b;
    begin = a;
    n = (int)(b - a);
}

// The sequence and tile of the idx-th tile of a batch, where sequence s has
// tiles(s, rows) of them: every wave counts 64 sequences at a time (one round of
// loads for a batch of 64), so the host needs no lengths, only a bound of the
// number of tiles. False: there is no such tile. Wave-uniform.
template <typename F>
__device__ inline bool find_tile(const int32_t *cu, int seqs, int64_t m, int idx, F tiles, SeqTile &t)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    if (idx < 0) return false;
    for (int s0 = 0; s0 < seqs; s0 += 64) {
        const int s = s0 + lane;
        int64_t begin = 0;
        int n = 0, cnt = 0;
        if (s < seqs) {
            seq_rows(cu, s, m, begin, n);
            cnt = tiles(s, n);
        }
        int incl = cnt;
        if (seqs > 1) {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
        }
        const uint64_t hit = __ballot(incl > idx - before);
        if (hit) {
            const int w = __builtin_ctzll(hit);
            t.seq = s0 + w;
            t.tile = idx - before - (__builtin_amdgcn_readlane(incl, w) - __builtin_amdgcn_readlane(cnt, w));
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)begin, w);
            t.begin = (int64_t)lo;  // at most BL_MAX_TOKENS rows
            t.n = __builtin_amdgcn_readlane(n, w);
            // offsets out of order can make the counts wrap: no tile beyond its sequence
            return t.tile >= 0 && t.tile < __builtin_amdgcn_readlane(cnt, w);
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

__device__ inline void store_out(float *p, float v) { *p = v; }
__device__ inline void store_out(bf16_t *p, float v)
{
    const __bf16 b = (__bf16)v;
    p->bits = __builtin_bit_cast(uint16_t, b);
}

// byte of (token, dim) inside a page and head of the cache (include/bitlinear.h)
template <int D>
__device__ inline int k_code_at(int token, int dim)
{
    return ((token & 3) * (D / 16) + (dim >> 4)) * 256 + (token >> 2) * 16 + (dim & 15);
}
__device__ inline int v_code_at(int token, int dim)
{
    return ((dim >> 4) * 4 + (token >> 4)) * 256 + (dim & 15) * 16 + (token & 15);
}

// sum over each row of 16 lanes, in a fixed order (every lane of the row gets it)
__device__ inline float row16_sum(float v)
{
    v += __int_as_float(dpp_mov<kDppQuadXor1>(__float_as_int(v)));
    v += __int_as_float(dpp_mov<kDppQuadXor2>(__float_as_int(v)));
    v += __int_as_float(dpp_mov<kDppRowHalfMirror>(__float_as_int(v)));
    v += __int_as_float(dpp_mov<kDppRowMirror>(__float_as_int(v)));
    return v;
}

constexpr int kBlock = 64;  // tokens per cache page

// A launch holds fewer than 2^32 threads in x: longer grids go in several launches,
// each with the index of its first workgroup.
constexpr int64_t kMostGroups = (int64_t)1 << 21;
constexpr int64_t kMostInZ = 1 << 15;  // and in y or z no more than 2^16 workgroups
template <typename F>
inline void in_launches(int64_t groups, F launch, int64_t most = kMostGroups)
{
    for (int64_t first = 0; first < groups; first += most)
        launch((int)first, (unsigned)(groups - first < most ? groups - first : most));
}

}  // namespace bl
