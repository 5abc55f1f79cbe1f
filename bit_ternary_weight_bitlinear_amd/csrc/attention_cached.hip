// attention_cached.hip -- attention of new tokens over the 8-bit cache.
//
//   x_ij = scale * (q_i . kc_j) * (ks / 127),  p = softmax over the seen j,
//   out_i = sum_j p_ij * vc_j * (vs / 127)
//
// kc, vc are int8 codes and ks, vs one scale per page of 64 tokens. Both products
// run on v_mfma_i32_16x16x64_i8 with the codes as they lie in memory: q and p
// become three signed base-256 digits (23 bits and a sign, relative to the
// largest of the row of q, and to the page's largest p: off by less than 2^-22 and
// 2^-23 of it), so the codes need no conversion, the sums are exact integers, and
// the result is as good as fp32.
// The 16 rows of the first operand hold 4 query rows x (3 digits + a zero row):
// row 4j+i is digit i of query row j. The result's row 4j+i lies in register i of
// the lanes with lane / 16 = j, so a lane joins the digits of its own query row
// in registers, and all per-row state (maximum, sum, rescaling) is per lane.
//
// A page is one step of a wave: 8 KB of K, 8 KB of V (head_dim 128), each lane
// 16 bytes per load, every load of a wave contiguous. ~200 VALU operations and 16
// matrix instructions per 16 KB and four query rows (0.5 us of a SIMD): bound by HBM
// with four rows a page (64 tokens over 7900, 32/8 heads: 168 us, 5.8 TB/s), by the
// latency of a wave's pages with eight (16 x 4 tokens over 2500, 32/8 heads: 18.5 us,
// the VALU busy 34 % of the cycles; 12 x 4 over 1 to 4000: 13 %), by the VALU with
// sixteen (32 x 8 tokens over 2500: 47 us, VALU 59 %, matrix cores 18 %). Not kept: the
// next page's V too ahead of its use (registers spill).
#include "attention_cached.hpp"

namespace bl {

__global__ __launch_bounds__(1024) void attention_weights_kernel(CachedArgs a, float *__restrict__ weights, int first_seq)
{
    __shared__ float part[1024];
    add_weights<16, false>(a, first_seq + (int)blockIdx.x, blockIdx.y, weights, nullptr, part);
}

struct CachedLayout {
    int64_t part_ml, stat, final_ml, bytes;
};
static CachedLayout cached_layout(const CachedProblem &p)
{
    const int64_t splits = launch_shape(p, row_tiles(p)).splits, rows = p.m * p.q_heads;
    CachedLayout L{};
    int64_t off = 0;
    if (splits > 1) off += round_up(splits * rows * p.head_dim * 4, 256);
    L.part_ml = off;
    if (splits > 1) off += round_up(splits * rows * 8, 256);
    L.stat = off;
    if (p.want_weights) off += round_up(rows * p.max_blocks * 8, 256);
    L.final_ml = off;
    if (p.want_weights && splits == 1) off += round_up(rows * 8, 256);
    L.bytes = off;
    return L;
}

int64_t attention_cached_workspace(const CachedProblem &p) { return cached_layout(p).bytes; }

hipError_t launch_attention_cached(const CachedProblem &p, void *ws, hipStream_t st)
{
    const int rt = row_tiles(p);
    const Shape shape = launch_shape(p, rt);
    const CachedLayout L = cached_layout(p);
    char *base = static_cast<char *>(ws);
    CachedArgs a = cached_args(p, shape, rt);
    if (a.splits > 1) {
        a.part_o = reinterpret_cast<float *>(base);
        a.part_ml = reinterpret_cast<float *>(base + L.part_ml);
    }
    if (p.weights) {
        a.stat = reinterpret_cast<float *>(base + L.stat);
        if (a.splits == 1) a.final_ml = reinterpret_cast<float *>(base + L.final_ml);
    }

    launch_tiles<kWhole>(p, a, shape, rt, query_tiles(p, rt), st);
    if (p.weights && a.splits == 1) {
        const int64_t blocks64 = ceil_div(p.max_blocks, 64);
        in_launches(p.seqs, [&](int first, unsigned n) {
            hipLaunchKernelGGL(attention_weights_kernel, dim3(n, (unsigned)blocks64), dim3(1024), 0, st, a, p.weights, first);
        });
    }
    return hipGetLastError();
}

}  // namespace bl
