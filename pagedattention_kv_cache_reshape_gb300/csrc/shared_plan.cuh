// shared_plan.cuh -- how a batch with shared prefixes is divided: what each
// group of sequences has in common, and the stream of key tiles that the
// persistent CTAs of the attention kernels cut into equal shares.
//
// Group g = sequences starts[g] .. starts[g+1]-1.  Its first C_g tokens are
// computed once for all its rows: whole blocks of min(prefix_lens[g], the
// smallest context - 1), so every sequence keeps at least one token of its
// own, and 0 where sharing does not pay.  A prefix item is (g, kv-head,
// `seqs_per_item` neighbouring sequences); its tiles are `keys_per_tile` keys
// of the prefix.  Items of a small group (at most `pair_seqs` sequences) are (g,
// two neighbouring kv-heads) and their tiles half as many keys.  Items are
// listed by group, kv-head, sequences.
//
// Teams: items of one (g, kv-head) read the same tiles, so `width` of them at a
// time form a block, and blocks have a stream of their own: teams of `width`
// CTAs, each CTA with one item of a block, take equal shares of it, so that a
// tile is read by the whole team at about the same time and comes from HBM
// once.  Items that fill no block are in the plain stream, cut by CTAs alone.
//
// Pieces: a share's tiles of one item.  The piece that begins with the item's
// first tile is kept in the item's own rows, ordered (group, kv-head, sequence,
// q-head of the kv-head), num_seqs * num_heads rows in all.  Any other piece is
// the first of its CTA's share of its stream, and is kept in the CTA's rows for
// that stream: item_rows rows from num_seqs * num_heads + (c * streams + stream)
// * item_rows on (stream 0 plain, 1 teams).
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
    int pair_seqs;                 // 0: no items of two kv-heads
    int max_width;                 // of a team; 1: no teams
    // Estimated work, in nanoseconds of an SM: `own_keys` tokens of one sequence (all kv-heads) on their own; a tile of
    // an item of up to small_seqs[0], up to small_seqs[1] and more sequences, and of one of two kv-heads; an item beside
    // its tiles.
    int own_keys, own_ns, small_seqs[2], tile_ns[4], item_ns;
    // Nothing is shared unless that saves this much, or some group has this many shared tokens.
    int64_t least_ns;
    int long_prefix;
};

// A group's items: heads * parts of them, each of kt tiles of `keys` keys; the
// first blocks * width parts of a kv-head in the teams' stream, the `rest` in the
// plain one.
struct GroupItems {
    int pair, heads, parts, keys, kt, blocks, rest;
    int full, last;   // parts of seqs_per_item sequences, and the sequences of one with fewer (0: none)
};
__device__ __forceinline__ GroupItems group_items(int n, int C, int num_kv_heads, int seqs_per_item, int keys_per_tile,
                                                  int pair_seqs, int width) {
    GroupItems x;
    x.pair = n <= pair_seqs;
    x.heads = x.pair ? num_kv_heads >> 1 : num_kv_heads;
    x.parts = x.pair ? 1 : (n + seqs_per_item - 1) / seqs_per_item;
    x.keys = x.pair ? keys_per_tile >> 1 : keys_per_tile;
    x.kt = (C + x.keys - 1) / x.keys;
    x.full = x.pair ? 0 : n / seqs_per_item;
    x.last = n - x.full * seqs_per_item;
    x.blocks = width > 1 ? x.parts / width : 0;
    x.rest = x.parts - x.blocks * width;
    return x;
}

// Estimated work of a group's shared tokens.
__device__ __forceinline__ int64_t items_ns(const SharedGroups &g, const GroupItems &x) {
    auto tile = [&](int seqs) { return g.tile_ns[seqs <= g.small_seqs[0] ? 0 : seqs <= g.small_seqs[1] ? 1 : 2]; };
    const int64_t tiles = x.pair ? g.tile_ns[3] : (int64_t)x.full * tile(g.seqs_per_item) + (x.last > 0 ? tile(x.last) : 0);
    return (tiles * x.kt + (int64_t)x.parts * g.item_ns) * x.heads;
}

// The plan, in the workspace.
struct SharedPlan {
    int32_t *seq_group;    // [num_seqs]
    int32_t *own_len;      // [num_seqs]: tokens behind the shared ones; 0: context length out of range
    int32_t *shared_len;   // [num_groups]: C_g
    int64_t *tile_start;   // [num_groups + 1]: the plain stream's tiles of the groups before
    int64_t *team_start;   // [num_groups + 1]: the teams' stream's tiles of the groups before
    int32_t *width;        // of the teams
};
constexpr int kMaxTeam = 4;

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

// The same by a whole warp with the same arguments in every lane: a load for every factor of 32, not of 2.
template <typename V, typename X>
__device__ __forceinline__ int last_at_most_warp(const V *a, int n, X v) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
        lo += (31 - __clz(__ballot_sync(0xffffffffu, i < hi && a[i < hi ? i : lo] <= v))) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The prefix item at tile t of a stream (t < the stream's end), by a whole warp; lane: the CTA's place in its team, or
// -1: the plain stream.
struct PrefixItem {
    int g, C;              // group, its shared tokens
    int s0, n;             // the group's first sequence, its sequences
    int kvh, part;         // (first) kv-head; the item's place among the group's sequences
    int tile;              // t's tile of the item
    GroupItems of;
};
__device__ __forceinline__ PrefixItem prefix_item(const SharedPlan &plan, const int32_t *starts, int num_groups,
                                                  int num_kv_heads, int seqs_per_item, int keys_per_tile, int pair_seqs,
                                                  int width, int lane, int64_t t) {
    const int64_t *start = lane < 0 ? plan.tile_start : plan.team_start;
    PrefixItem it;
    it.g = last_at_most_warp(start, num_groups, t);   // (groups without tiles are passed over)
    it.C = plan.shared_len[it.g];
    it.s0 = __ldg(starts + it.g);
    it.n = __ldg(starts + it.g + 1) - it.s0;
    it.of = group_items(it.n, it.C, num_kv_heads, seqs_per_item, keys_per_tile, pair_seqs, width);
    const int64_t local = t - start[it.g];
    const int item = (int)(local / it.of.kt), per_head = lane < 0 ? it.of.rest : it.of.blocks;
    it.tile = (int)(local - (int64_t)item * it.of.kt);
    it.kvh = item / per_head;
    it.part = item - it.kvh * per_head;
    it.part = lane < 0 ? it.of.blocks * width + it.part : it.part * width + lane;
    if (it.of.pair) it.kvh *= 2;
    return it;
}

// Row of sequence s0 + i, q-head 0 of kv-head kvh, among the items' own rows.
__device__ __forceinline__ int64_t item_row(int s0, int n, int kvh, int i, int num_heads, int group) {
    return (int64_t)s0 * num_heads + ((int64_t)kvh * n + i) * group;
}

// Exclusive scans of N values over a CTA of kThreads threads, in place; total[k] their sums.  `tot` holds N * kThreads /
// 32 values that no thread reads or writes meanwhile.
template <int kThreads, int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (*tot)[kThreads / 32], int64_t (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        incl[k] = v[k];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl[k], off);
            if (lane >= off) incl[k] += y;
        }
        if (lane == 31) tot[k][warp] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int64_t before = 0;
        total[k] = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int64_t x = tot[k][w];
            if (w < warp) before += x;
            total[k] += x;
        }
        v[k] = before + incl[k] - v[k];
    }
    __syncthreads();
}

// C_g of every group into lens[num_groups], by a whole CTA of kThreads threads;
// `starts` receives a copy of the groups' starts when it is not the input
// itself.  Both may be shared or global memory.  False, and every C 0: the
// starts do not run from 0 to num_seqs in order.  `status` (nullable) receives
// what is out of range.
template <int kThreads>
__device__ bool shared_lens(const SharedGroups &g, int32_t *starts, int32_t *lens, int32_t *status) {
    const int tid = threadIdx.x, S = g.num_seqs, NG = g.num_groups;
    // the first round's loads all at once; later rounds (more groups or sequences than threads) load again
    int a = 0, b = 0, P = 0, ctx = 0;
    if (tid < NG) {
        a = __ldg(g.starts + tid);
        b = __ldg(g.starts + tid + 1);
        P = __ldg(g.prefix_lens + tid);
    }
    if (tid < S) ctx = __ldg(g.context_lens + tid);
    int wrong = 0;
    for (int i = tid; i < NG; i += kThreads) {
        const int x = i == tid ? a : __ldg(g.starts + i), y = i == tid ? b : __ldg(g.starts + i + 1);
        wrong |= x < 0 || y < x || y > S || (i == 0 && x != 0) || (i == NG - 1 && y != S);
        if (starts) starts[i] = x;
        lens[i] = INT_MAX;
    }
    const bool ok = !__syncthreads_or(wrong);
    if (!ok && tid == 0) set_status(status, PA_ERR_OUT_OF_RANGE);
    const int32_t *from = starts ? starts : g.starts;
    for (int s = tid; s < S; s += kThreads) {   // the smallest context of each group
        const int c = s == tid ? ctx : __ldg(g.context_lens + s);
        if (c <= 0 || c > g.max_tokens) set_status(status, PA_ERR_OUT_OF_RANGE);
        else if (ok) atomicMin(lens + last_at_most(from, NG, s), c);
    }
    __syncthreads();
    int64_t saved[2] = {}, all[2];   // and the groups with long prefixes
    for (int i = tid; i < NG; i += kThreads) {
        const int n = i == tid ? b - a : __ldg(g.starts + i + 1) - __ldg(g.starts + i);
        const int len = i == tid ? P : __ldg(g.prefix_lens + i);
        const int least = *const_cast<volatile int32_t *>(lens + i);   // (global atomics: not through L1)
        int C = 0;
        if (len < 0 || len > g.max_tokens) set_status(status, PA_ERR_OUT_OF_RANGE);
        else if (ok && n >= 2 && least != INT_MAX) C = min(len, least - 1) / g.block_size * g.block_size;
        // shared only where that is less work than every sequence reading these tokens for itself
        if (C > 0) {
            const int64_t less = (int64_t)n * ((C + g.own_keys - 1) / g.own_keys) * g.own_ns -
                                 items_ns(g, group_items(n, C, g.num_kv_heads, g.seqs_per_item, g.keys_per_tile, g.pair_seqs, 1));
            if (less > 0) {
                saved[0] += less;
                saved[1] += C >= g.long_prefix;
            } else {
                C = 0;
            }
        }
        lens[i] = C;
    }
    __shared__ int64_t tot[2][kThreads / 32];
    block_scan<kThreads, 2>(saved, tot, all);
    if (all[0] < g.least_ns && all[1] == 0) {
        for (int i = tid; i < NG; i += kThreads) lens[i] = 0;
        __syncthreads();
    }
    return ok;
}

// The plan's arrays from C_g, by a whole CTA.  Returns the estimated work of the own and of the shared parts, and the
// teams' width.
struct PlanSums {
    int64_t own, prefix;
    int width;
};
template <int kThreads>
__device__ __forceinline__ PlanSums shared_write_plan(const SharedGroups &g, const SharedPlan &plan, bool ok,
                                                      const int32_t *starts, const int32_t *lens) {
    __shared__ int64_t tot[5][kThreads / 32];
    const int tid = threadIdx.x;
    auto items_of = [&](int i, int width) {
        return group_items(__ldg(g.starts + i + 1) - __ldg(g.starts + i), lens[i], g.num_kv_heads, g.seqs_per_item,
                           g.keys_per_tile, g.pair_seqs, width);
    };
    // costs, and the tiles that teams of 2, 3 and 4 leave to be read once only
    int64_t sum[5] = {}, total[5];
    for (int s = tid; s < g.num_seqs; s += kThreads) {
        const int ctx = __ldg(g.context_lens + s);
        const int grp = ok ? last_at_most(starts, g.num_groups, s) : 0;
        const int own = ctx > 0 && ctx <= g.max_tokens ? ctx - lens[grp] : 0;
        plan.seq_group[s] = grp;
        plan.own_len[s] = own;
        sum[0] += (int64_t)((own + g.own_keys - 1) / g.own_keys) * g.own_ns;
    }
    for (int i = tid; i < g.num_groups; i += kThreads)
        if (lens[i] > 0) {
            const GroupItems x = items_of(i, 1);
            sum[1] += items_ns(g, x);
#pragma unroll
            for (int w = 2; w <= kMaxTeam; ++w)
                if (w <= g.max_width) sum[w] += (int64_t)(x.parts / w) * (w - 1) * x.heads * x.kt;
        }
    block_scan<kThreads, 5>(sum, tot, total);
    PlanSums r = {total[0], total[1], 1};
    int64_t best = 0;
#pragma unroll
    for (int w = 2; w <= kMaxTeam; ++w)
        if (total[w] > best) { best = total[w]; r.width = w; }
    // where each group's items begin
    int64_t before[2] = {};
    for (int base = 0; base < g.num_groups; base += kThreads) {
        const int i = base + tid;
        int64_t at[2] = {}, all[2];
        if (i < g.num_groups) {
            const int C = lens[i];
            if (C > 0) {
                const GroupItems x = items_of(i, r.width);
                at[0] = (int64_t)x.heads * x.rest * x.kt;
                at[1] = (int64_t)x.heads * x.blocks * x.kt;
            }
            plan.shared_len[i] = C;
        }
        block_scan<kThreads, 2>(at, tot, all);
        if (i < g.num_groups) {
            plan.tile_start[i] = before[0] + at[0];
            if (plan.team_start) plan.team_start[i] = before[1] + at[1];
        }
        before[0] += all[0];
        before[1] += all[1];
    }
    if (tid == 0) {
        plan.tile_start[g.num_groups] = before[0];
        if (plan.team_start) {
            plan.team_start[g.num_groups] = before[1];
            *plan.width = r.width;
        }
    }
    return r;
}

}  // namespace pa
