// attn_division.cu -- the multi-query attention's division of work, walked on
// the host: which CTA takes which keys of which item, in the kernels' own code.
#include "attn_common.cuh"
#include "attn_simt.cuh"
#include "attn_tc.cuh"

namespace pkv {
namespace {

template <class Div>
long long items(const AttnParams& p, int grid, long long* out, long long cap) {
    long long n = 0;
    for (int cta = 0; cta < grid; ++cta) {
        AttnWalk<Div> w = attn_walk_start_host<Div>(p, cta, grid);
        AttnItem it;
        while (w.next(p, cta, it)) {
            if (n < cap) {
                const bool split = it.nparts > 1;
                const long long row[] = {cta, it.seq, it.row, it.ntok, it.pos, it.first, it.kv0, it.kv1, it.g,
                                         it.part, it.nparts, it.keys, it.per_key,
                                         split ? AttnWalk<Div>::owner(it, w.share, 0) : -1,
                                         split ? AttnWalk<Div>::owner(it, w.share, it.part) : -1,
                                         split ? attn_partial(cta, it.part) : -1};
                for (long long x : row) *out++ = x;
            }
            ++n;
        }
    }
    return n;
}

}  // namespace
}  // namespace pkv

// Not in the header: the items of a launch of `grid` CTAs as rows of 16 numbers
// (CTA, sequence, first row, tokens, position, the sequence's first position, keys from and
// to, kv head, part, parts, keys and work per key of the item, CTA of part 0 and of this
// part, place of the partial result), at most `cap` of them; returns how many there are.
// rows: of a full tile, 256 (tensor cores), 64 or 16 (CUDA cores).
extern "C" PKV_API long long pkv_internal_attn_items(int rows, const int32_t* query_start, const int32_t* context_lens,
                                                     int num_seqs, int num_tokens, int num_kv_heads, int group_log2,
                                                     int max_context, int grid, long long* out, long long cap) {
    pkv::AttnParams p = {};
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.group_log2 = group_log2;
    p.block_size = 1;
    p.max_blocks_per_seq = max_context;
    return rows == 256 ? pkv::items<pkv::atc::TcDivision>(p, grid, out, cap)
           : rows == 64 ? pkv::items<pkv::SimtDivision<64>>(p, grid, out, cap)
                        : pkv::items<pkv::SimtDivision<16>>(p, grid, out, cap);
}
