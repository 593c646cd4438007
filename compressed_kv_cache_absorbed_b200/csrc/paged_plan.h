// Where the new tokens of a paged append go: index arithmetic shared by the kernels and by
// the host tests (plain C++, no CUDA needed).
//
// Sequence b's new tokens are rows [new_offsets[b], new_offsets[b + 1]) of the call's inputs
// and the last of its seq_lens[b] tokens.  The work is cut by page: an item is the part of
// one 64-token page that receives new tokens, so that one block owns every byte (and the one
// scale) it writes.  k new tokens touch at most k / 64 + 2 pages, whatever their position in
// the first one, and floor(o1 / 64) - floor(o0 / 64) >= floor((o1 - o0) / 64), so numbering
// sequence b's items from new_offsets[b] / 64 + 2 b gives every sequence enough of them
// without a prefix sum over the lengths.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

constexpr int kPageTokensLog2 = 6;
constexpr int kPageRows = 1 << kPageTokensLog2;   // tokens per page

// first item of sequence b, whose new tokens start at row o0; items of a whole call
MLA_HD long long append_item_base(int o0, int b) { return (long long)(o0 >> kPageTokensLog2) + 2LL * b; }
MLA_HD long long append_items(int n, int B) { return (long long)(n >> kPageTokensLog2) + 2LL * B; }

// new_offsets entries of sequence b are usable: rows inside the call's n, not decreasing, the
// first sequence from row 0 and the last one up to row n
MLA_HD bool append_offsets_ok(int o0, int o1, int b, int B, int n) {
    return o0 >= 0 && o1 >= o0 && o1 <= n && (b > 0 || o0 == 0) && (b + 1 < B || o1 == n);
}

// The part of one page an item writes: rows [r0, r1) of the page at block `block` of the
// sequence, from input rows src .. src + r1 - r0 - 1, at positions 64 block + r0 ...
struct AppendItem {
    int block, r0, r1, src;
};

// Item `k` (counted from the sequence's first) of a sequence with new rows [o0, o1) and
// `len` tokens after the append.  Returns 0 if the item writes nothing, 1 if it writes *it,
// and -1 if the sequence is invalid (fewer tokens than new ones, or more than its row of the
// block table has pages for); an invalid sequence is reported by its item 0 only.
MLA_HD int append_item(int o0, int o1, int len, int max_blocks, long long k, AppendItem* it) {
    const int fresh = o1 - o0;
    if (fresh <= 0) return 0;
    if (len < fresh || (long long)len > (long long)max_blocks * kPageRows) return k == 0 ? -1 : 0;
    const int start = len - fresh;                     // position of the first new token
    const long long block = (long long)(start >> kPageTokensLog2) + k;
    const long long p0 = block * kPageRows;
    if (p0 >= len) return 0;
    it->block = (int)block;
    it->r0 = p0 < start ? (int)(start - p0) : 0;
    it->r1 = len - p0 < kPageRows ? (int)(len - p0) : kPageRows;
    it->src = (int)(o0 + (p0 + it->r0 - start));
    return 1;
}

}  // namespace mla
