// shared_plan.cuh -- how a batch with shared prefixes is divided: what each
// group of sequences has in common, and the stream of key tiles that the
// persistent CTAs of the attention kernels cut into equal shares.
//
// Group g = sequences starts[g] .. starts[g+1]-1.  Its first C_g tokens are
// computed once for all its rows: whole blocks of min(prefix_lens[g], the
// smallest context - 1), so every sequence keeps at least one token of its
// own, and 0 where sharing does not pay.  A prefix item is (g, kv-head,
// `seqs_per_item` neighbouring sequences); its tiles are `keys_per_tile` keys
// of the prefix.  Items are listed by group, kv-head, sequences.  The own
// stream lists, by sequence and kv-head, the tiles behind C_g.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

struct SharedGroups {
    const int32_t *context_lens;   // [num_seqs]
    const int32_t *starts;         // [num_groups + 1]
    const int32_t *prefix_lens;    // [num_groups]
    int num_seqs;
    int num_groups;
    int num_kv_heads;
    int block_size;
    int64_t max_tokens;            // max_blocks * block_size
    int seqs_per_item;
    int keys_per_tile;
};

// The plan, in the workspace.
struct SharedPlan {
    int32_t *seq_group;    // [num_seqs]
    int32_t *own_len;      // [num_seqs]: tokens behind the shared ones; 0: context length out of range
    int32_t *shared_len;   // [num_groups]: C_g
    int32_t *min_ctx;      // [num_groups], scratch
    int32_t *item_start;   // [num_groups + 1]
    int64_t *tile_start;   // [num_groups + 1]: tiles of all items of the groups before
    int64_t *own_start;    // [num_seqs + 1]: own tiles (of one kv-head) of the sequences before
};

// The c-th of p equal shares of n tiles begins here; share that holds tile t.
__host__ __device__ __forceinline__ int64_t share_begin(int64_t c, int64_t n, int64_t p) { return c * n / p; }
__host__ __device__ __forceinline__ int64_t share_of(int64_t t, int64_t n, int64_t p) { return ((t + 1) * p - 1) / n; }

// Last index i in [0, n) with a[i] <= v (a[0] <= v).
template <typename V, typename X>
__device__ __forceinline__ int last_at_most(const V *a, int n, X v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace pa
