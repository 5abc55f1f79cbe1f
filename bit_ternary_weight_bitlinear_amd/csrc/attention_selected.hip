// attention_selected.hip -- attention of new tokens over the blocks of the 8-bit cache
// that a list names for each of them and each kv head.
//
// The mathematics, the digits and a wave's work on a page are those of
// attention_cached.hip; a page is found through the list and the sequence's table, and
// the rows of a workgroup are one token's query heads of one kv head.
#include "attention_cached.hpp"

namespace bl {

// For the launch rules a token and its list are a sequence and its table
static CachedProblem by_rows(const SelectedProblem &p)
{
    CachedProblem r = p.c;
    r.seqs = p.c.m;
    r.max_blocks = p.keep;
    r.cu = nullptr;
    return r;
}

struct SelectedLayout {
    int64_t part_ml, bytes;
};
static SelectedLayout selected_layout(const CachedProblem &r)
{
    const int64_t splits = launch_shape(r, row_tiles(r)).splits, rows = r.m * r.q_heads;
    SelectedLayout L{};
    if (splits == 1) return L;
    L.part_ml = round_up(splits * rows * r.head_dim * 4, 256);
    L.bytes = L.part_ml + round_up(splits * rows * 8, 256);
    return L;
}

int64_t attention_selected_workspace(const SelectedProblem &p) { return selected_layout(by_rows(p)).bytes; }

hipError_t launch_attention_selected(const SelectedProblem &p, void *ws, hipStream_t st)
{
    const CachedProblem r = by_rows(p);
    const int rt = row_tiles(r);
    const Shape shape = launch_shape(r, rt);
    CachedArgs a = cached_args(p.c, shape, rt);
    a.selected = p.selected;
    a.keep = p.keep;
    if (a.splits > 1) {
        a.part_o = static_cast<float *>(ws);
        a.part_ml = reinterpret_cast<float *>(static_cast<char *>(ws) + selected_layout(r).part_ml);
    }
    // Lists of more than a third of the last-level cache, of one row per sequence, are read past
    // it: 32 blocks of 32/8 heads of 128 for 16 rows (64 MB) 19.1 us beside 15.8 through it, for 20
    // rows 18.9 and 19.0, 24 rows 19.5 and 19.8, 64 rows 45.1 and 47.9, 128 rows 84.5 and 92.4 (other
    // inputs from call to call). Rows of one sequence mostly list the same blocks, which the cache
    // holds for them: 10 x 4 rows, 8 of their 32 blocks common 31.0 and 28.9, 24 of them 26.4 and
    // 21.8; 8 x 32 rows 78.6 and 61.8
    const int64_t bytes = p.c.m * p.c.kv_heads * p.keep * 2 * kBlock * p.c.head_dim;
    if (p.c.m == p.c.seqs && bytes >= (int64_t)96 << 20) launch_tiles<kSelectedPast>(p.c, a, shape, rt, p.c.m * a.tiles_per_seq, st);
    else launch_tiles<kSelected>(p.c, a, shape, rt, p.c.m * a.tiles_per_seq, st);
    return hipGetLastError();
}

}  // namespace bl
