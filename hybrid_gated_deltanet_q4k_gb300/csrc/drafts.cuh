// The tokens of a call over drafted tokens: each sequence's range, checked, and
// the ancestors of each of its tokens.
#pragma once

#include "common.cuh"

namespace gdn {

struct DraftTokens {
    const int32_t* cu;       // [n_seqs + 1], or null: max_new tokens each
    const uint64_t* tree;    // [n_tokens] mask words, or null: chains
    int n_tokens, max_new, n_seqs;
};

// The tokens of a sequence whose offsets are lo and hi.  Offsets out of range
// leave the sequence without tokens and say so in `skipped`.
__device__ __forceinline__ int draft_count(const DraftTokens& d, int lo, int hi, int& skipped) {
    if (lo < 0 || hi < lo || hi > d.n_tokens || hi - lo > d.max_new) {
        atomicCAS(&skipped, 0, static_cast<int>(ERR_INDEX));
        return 0;
    }
    return hi - lo;
}

// First token and number of tokens of sequence s.
__device__ __forceinline__ int draft_range(const DraftTokens& d, int s, int& first, int& skipped) {
    if (!d.cu) {
        first = s * d.max_new;
        return d.max_new;
    }
    first = d.cu[s];
    return draft_count(d, first, d.cu[s + 1], skipped);
}

// The proper ancestors of a sequence's token i (first: its token 0).
__device__ __forceinline__ uint64_t draft_ancestors(const DraftTokens& d, int first, int i) {
    const uint64_t earlier = (1ull << i) - 1;
    return d.tree ? d.tree[first + i] & earlier : earlier;
}

// The parent of a token with these ancestors (-1: none): tokens follow their ancestors.
__device__ __forceinline__ int draft_parent(uint64_t ancestors) { return 63 - __clzll(static_cast<long long>(ancestors)); }

}  // namespace gdn
