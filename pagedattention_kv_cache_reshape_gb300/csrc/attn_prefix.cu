// attn_prefix.cu -- the shared part of pa_decode_shared_prefix on the 5th-gen
// tensor cores: what all sequences of a group see, for all their query rows.
//
// For an item (group, kv-head, up to 2 * POS neighbouring sequences, POS =
// 128 / G) the rows (sequence, q-head of the kv-head) are the M of
//     S = Q K^T,  P = 2^(S * scale*log2e - m),  O += P V,  l += rows' sums of P
// over the group's shared keys, and the result stays (m, l, O) in fp32: the
// merge kernel joins it with the sequences' own parts.
//
// Work: the items' tiles, one after the other, are a stream (shared_plan.cuh).
// Each persistent CTA takes an equal contiguous share, so every CTA has the same
// number of tiles whatever the group sizes; a share holds a few pieces of items,
// usually one or two.  Items that read the same tiles go to teams of CTAs that
// read them together: 256 sequences (4 items a kv-head) over 32,768 tokens read
// 137 MB from HBM instead of 406 MB, and the call took 130 us instead of 149
// (teams of at most two: 136) when they were introduced; it takes 128-130 now.
//
// Bound: a 64 KB tile (K and V, 128 keys x 128 dims) takes an SM's share of
// HBM 1.5 us; the products of one M-tile of 128 rows take 0.5 us of the tensor
// pipe, of two 1 us.  So groups of up to 256 rows a kv-head are bound by HBM,
// larger ones (several items read the same tiles) by the tensor pipe and the
// softmax beside it.  Measured (32 / 8 heads x 128): 16 sequences over one prefix
// of 131,072 tokens 89 us, 6.0 TB/s; 256 over 32,768 104 us, the tensor pipe 75 %
// busy (a tile of two M-tiles takes about 2700 cycles, its products 2048); 24
// groups of 8 over up to 4096 tokens, 32 heads, 165 us beside the decode kernel,
// 5.2 TB/s: there an SM waits for its ring of tiles, 56-58 GB/s a SM.
//
// Roles (512 threads): warps 0-7 two softmax warpgroups (thread = row = TMEM
// lane of its M-tile), warp 8 TMA producer, warp 9 TMEM owner and MMA issuer,
// warps 12-15 output.  Schedule, layouts and waits as in attn_prefill.cu; no
// causal mask, and blocks past the shared tokens come in as zeros (TMA
// out-of-bounds fill) with their logits masked.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "shared_plan.cuh"

namespace pa {
namespace {

constexpr int BM = 128;               // rows per M-tile
constexpr int kMT = 2;                // M-tiles per item at most, one softmax warpgroup each
constexpr int BN = kPrefixKeys;       // keys per KV tile
static_assert(BN == 128, "P is released in two halves of 64 keys");
constexpr size_t kSmemLimit = 227 * 1024;
constexpr int kProducerWarp = 4 * kMT;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kOutWarp = kProducerWarp + 4;
constexpr int kThreads = 32 * (4 * kMT + 8);
// Register split: launched at 128 a thread; the softmax warpgroups' share comes from the others'.
constexpr int kRegsLaunch = 128;
constexpr int kRegsSide = 64;
constexpr int kRegsOut = 64;
constexpr int kRegsSoftmax = 192;
static_assert(128 * (kRegsSide + kRegsOut) + 128 * kMT * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr int kTmemCols = 512;

struct PrefixParams {
    SharedPlan plan;
    const int32_t *starts;
    const int32_t *block_tables;
    const int32_t *shares;     // CTAs that take a share
    float *o;                  // pieces: [rows][D]
    float2 *ml;                // [rows]
    int num_seqs;
    int num_groups;
    int num_heads;
    int num_kv_heads;
    int pair_seqs;    // groups of at most this many sequences: items of two kv-heads
    int group;        // q-heads per kv-head
    int pos;          // sequences per M-tile: 128 / group
    int item_rows;
    int max_blocks;
    int num_blocks;
    float scale_log2;
    int32_t *status;
    // bounded waits: their limit, and the test hook's stall (PA_STALL_*)
    uint64_t wait_ns;
    int stall;
    int stall_after;
    int32_t *wait_sites;
};

// Whether the phase has completed already, in a register that may be used later: the answer travels while products are
// issued, and a wait is left out where it is yes.
__device__ __forceinline__ uint32_t peek(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done;
}
__device__ __forceinline__ bool wait_unless(uint32_t done, uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, done != 0) || mbar_wait_warp(bar, parity, limit_ns);
}

template <int D> struct Shape {
    static constexpr int kDH = D / 64;                 // 64-column planes of a head
    static constexpr int kQBytes = BM * D * 2;         // one M-tile of Q
    static constexpr int kSlotBytes = BN * D * 2;      // K or V of one KV tile
    static constexpr int kPlaneQ = BM * 128;           // one 64-column plane of Q
    static constexpr int kBarBytes = 2816;             // barriers, TMEM address, item slots, (m, l) of the rows
    static constexpr int kFit = (int)((kSmemLimit - kMT * kQBytes - kBarBytes) / kSlotBytes);
    static constexpr int kSlots = kFit < 8 ? kFit : 8;  // K/V ring depth
    static constexpr size_t kSmem = (size_t)kMT * kQBytes + (size_t)kSlots * kSlotBytes + kBarBytes;
    // kPair's softmax looks at the phase of V's entry of tile j - 1 until its own weights of tile j are out.  The same slot
    // must not be released again before that: with three slots it would be by tile j + 1's K, whose product waits for no
    // weights; with four it is by tile j + 1's V, whose product waits for them.
    static_assert(kSlots >= 4, "the K/V ring needs at least four slots");
    static_assert(kSmem <= kSmemLimit, "shared memory");
};

// A piece: tiles tile0 .. tile0 + nkv - 1 of an item.  Three kinds:
//  kWide  more than `pos` sequences: M-tile t holds the t-th `pos` of them; both
//         take every KV tile of 128 keys
//  kPair  a small group and two kv-heads: M-tile t holds the rows of kv-head
//         kvh + t; a KV tile is 64 keys of both, so a TMA box carries both heads
//         (half the boxes a byte, rows of memory twice as long: the 24 groups of 8
//         222 us against 237 one head at a time, one of 16 over 131,072 tokens 110
//         against 114, the whole call with a flushed L2)
//  kTurns up to `pos` sequences of one kv-head (an odd number of kv-heads, or the last
//         few of a larger group): both M-tiles hold the same rows, t takes KV tiles t,
//         t + 2, ..., and the output warpgroup joins them
// live = 0 marks the end.
constexpr int kTurns = 0, kWide = 1, kPair = 2;
struct Piece {
    int table_seq, kvh, seq0, nseq, kind, tile0, nkv, C, live, second;
    int64_t row;      // row of (sequence seq0, q-head 0 of kvh) in o and ml; M-tile 1's rows begin `second` sequences on
    __device__ __forceinline__ int tiles(int t) const { return kind != kTurns ? nkv : (nkv + 1 - t) >> 1; }
};
constexpr int kItemSlots = 4;                 // pieces published ahead of their use

template <int D, int kB>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_k2,
                  const __grid_constant__ CUtensorMap tmap_v2, const PrefixParams p) {
    constexpr int kBlocksPerTile = BN / kB;          // cache blocks per KV tile
    static_assert(kBlocksPerTile <= 32, "one TMA box per producer lane");
    using SH = Shape<D>;
    constexpr int kDH = SH::kDH, kQBytes = SH::kQBytes, kSlotBytes = SH::kSlotBytes;
    constexpr int kPlaneQ = SH::kPlaneQ, kSlots = SH::kSlots;
    // V: [block][D/64 plane][B rows][64]; 16-key MMA steps 0..3 of 64 keys start
    // at 0, kVS1, kVS2 and kVS2 + kVS1
    constexpr int kVBlockBytes = kDH * kB * 128;                       // one block, all planes
    constexpr int kVS1 = (16 / kB) * kVBlockBytes + (16 % kB) * 128;
    constexpr int kVS2 = (32 / kB) * kVBlockBytes + (32 % kB) * 128;
    static_assert(((48 / kB) * kVBlockBytes + (48 % kB) * 128) == kVS1 + kVS2, "step 3 = s2 + s1");
    constexpr int kVChunk = 64 / kB * kVBlockBytes;                    // 64 keys
    constexpr int kVLbo = kB * 128;
    constexpr int kVSbo = kB < 16 ? kVBlockBytes : 1024;
    // K: [8-row group][D/64 plane][8 rows][64]
    constexpr int kKSbo = kDH * 1024;
    constexpr int kKPlane = 1024;
    // tiles of two kv-heads: a block's share is twice as long, [..][kv-head][plane][..], the heads kDH planes apart
    constexpr int kBlock2 = 2 * kVBlockBytes;
    constexpr int kVS1p = (16 / kB) * kBlock2 + (16 % kB) * 128, kVS2p = (32 / kB) * kBlock2 + (32 % kB) * 128;
    static_assert(((48 / kB) * kBlock2 + (48 % kB) * 128) == kVS1p + kVS2p, "step 3 = s2 + s1");
    constexpr int kVSboP = kB < 16 ? kBlock2 : 1024;
    constexpr int kKSboP = 2 * kDH * 1024;
    constexpr uint32_t kIdescQK2 = umma_idesc_bf16(BM, BN / 2, 0);
    constexpr uint32_t kIdescQK = umma_idesc_bf16(BM, BN, 0);
    constexpr uint32_t kIdescPV = umma_idesc_bf16(BM, D, 1);
    constexpr uint32_t kAll = 0xffffffffu;

    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_s = smem;
    uint8_t *kv_s = smem + kMT * kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(kv_s + kSlots * kSlotBytes);
    uint64_t *q_full = bars;                       // Q of the piece landed
    uint64_t *q_empty = q_full + 1;                // every QK product of the piece done
    uint64_t *kv_full = q_empty + 1;               // [kSlots]: slot landed
    uint64_t *kv_empty = kv_full + kSlots;         // [kSlots]: slot read by its products
    uint64_t *s_full = kv_empty + kSlots;          // [tile]: S_t written
    uint64_t *p_full = s_full + kMT;               // [tile]: P_t written (and O_t rescaled)
    uint64_t *o_full = p_full + kMT;               // [tile]: last product of the piece into O_t done
    uint64_t *p_half = o_full + kMT;               // [tile]: P_t's first 64 keys written
    uint64_t *o_empty = p_half + kMT;              // [tile]: O_t read by the output warpgroup
    uint64_t *l_full = o_empty + kMT;              // [tile]: the rows' (m, l) written
    // kPair, [place][tile]: S_t written in its first (even KV tiles) or second place, P_t written there.  The softmax
    // warpgroups may be a tile ahead of the products, so each place has barriers of its own: the next use of a place
    // comes after the products that read it, and no barrier gets two phases ahead of who waits for it.
    uint64_t *s2_full = l_full + kMT;
    uint64_t *p2_full = s2_full + 2 * kMT;
    uint64_t *item_full = p2_full + 2 * kMT;       // [kItemSlots]: piece published
    uint64_t *item_empty = item_full + kItemSlots; // [kItemSlots]: piece read by every consumer
    uint64_t *drained = item_empty + kItemSlots;   // every product issued has completed
    uint32_t &tmem_base_s = *reinterpret_cast<uint32_t *>(drained + 1);
    Piece *items = reinterpret_cast<Piece *>(drained + 2);           // [kItemSlots]
    int64_t *range_s = reinterpret_cast<int64_t *>(items + kItemSlots);   // this CTA's shares: begin and end, team's and plain
    float2 *ml_s = reinterpret_cast<float2 *>(range_s + 4);          // [tile][row]
    static_assert((3 + 2 * kSlots + 10 * kMT + 2 * kItemSlots + 2) * 8 + kItemSlots * sizeof(Piece) + 32 +
                          kMT * BM * sizeof(float2) <= SH::kBarBytes,
                  "barrier area");

    // the warp index broadcast from lane 0 is provably warp-uniform
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need 1024-byte alignment
        if (tid == 0) set_status(p.status, PA_ERR_CUDA);
        grid_dependency_wait();
        return;
    }
    // This grid starts once every decode CTA has passed its wait for the plan, so
    // the plan is complete.  Shares for fewer CTAs than the grid has: the others
    // leave their SMs (but not before the decode grid is done: what waits for
    // this grid relies on both).
    // Plain loads: written by the plan grid.  Teams of `width` CTAs (as many as there are tiles at most, so that no
    // share is empty) and their place in one; then every CTA by itself.
    const int cta = blockIdx.x, width = *p.plan.width, shares = p.shares[0];
    const int64_t T1 = p.plan.team_start[p.num_groups], P1 = min((int64_t)(shares / width), T1);
    const int64_t T0 = p.plan.tile_start[p.num_groups], P0 = min((int64_t)shares, T0);
    const bool in_team = cta / width < P1, alone = cta < P0;
    const int64_t a1 = in_team ? share_begin(cta / width, T1, P1) : 0, b1 = in_team ? share_begin(cta / width + 1, T1, P1) : 0;
    const int64_t a0 = alone ? share_begin(cta, T0, P0) : 0, b0 = alone ? share_begin(cta + 1, T0, P0) : 0;
    grid_dependents_launch();    // every decode and prefix CTA runs before the merge's take up room

    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(kv_full + i, 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int t = 0; t < kMT; ++t) {
            mbar_init(s_full + t, 1);
            mbar_init(p_full + t, BM);
            mbar_init(o_full + t, 1);
            mbar_init(p_half + t, BM);
            mbar_init(o_empty + t, BM);
            mbar_init(l_full + t, BM);
            for (int b = 0; b < 2; ++b) {
                mbar_init(s2_full + b * kMT + t, 1);
                mbar_init(p2_full + b * kMT + t, BM);
            }
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(item_full + i, 1);
            mbar_init(item_empty + i, 1 + 4 * kMT + 4);  // the MMA warp, every softmax and output warp
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (cta >= shares) {         // (the same in every thread)
        grid_dependency_wait();
        return;
    }
    if (warp == kMmaWarp) tmem_alloc(&tmem_base_s, kTmemCols);
    if (warp == kProducerWarp && lane == 0) {
        range_s[0] = a1;
        range_s[1] = b1;
        range_s[2] = a0;
        range_s[3] = b0;
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    // TMEM columns: S_t at t*BN (fp32); P_t, bf16 pairs, over the first BN/2 columns of S_t; O_t at kMT*BN + t*D.
    // kPair: S_t of 64 columns has two places, for even and odd KV tiles
    auto s_col = [](int t) { return (uint32_t)(t * BN); };
    auto o_col = [](int t) { return (uint32_t)(kMT * BN + t * D); };
    auto slot_of = [](int n) { return n % kSlots; };
    auto phase_of = [](int n) { return (uint32_t)((n / kSlots) & 1); };
    // a place in the K/V ring
    struct Ring {
        int slot;
        uint32_t phase;
        __device__ __forceinline__ Ring next() const {
            Ring r;
            r.slot = slot + 1 == kSlots ? 0 : slot + 1;
            r.phase = slot + 1 == kSlots ? phase ^ 1u : phase;
            return r;
        }
    };
    auto take_item = [&](int it, Piece &I) -> bool {
        if (!mbar_wait_warp(item_full + it % kItemSlots, (uint32_t)((it / kItemSlots) & 1), p.wait_ns)) return false;
        I = items[it % kItemSlots];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + it % kItemSlots);
        return true;
    };

    if (warp >= kOutWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
        // ================= output warpgroup: thread r writes (m, l, O) of row r of M-tile t after the piece's last
        // product into O_t; the MMA warp waits for its o_empty before the next piece's first product into O_t
        const int r = tid & (BM - 1);
        const int head = r / p.pos, i_pos = r - head * p.pos;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        bool ok = true;
        int no[kMT] = {};
        for (int it = 0; ok; ++it) {
            Piece I;
            if (!take_item(it, I)) { ok = false; break; }
            if (!I.live) break;
            if (I.kind == kTurns && I.nkv > 1) {
                // both M-tiles hold this row: joined on the way out
#pragma unroll
                for (int t = 0; t < kMT; ++t)
                    ok = ok && mbar_wait_warp(o_full + t, (uint32_t)(no[t] & 1), p.wait_ns) &&
                         mbar_wait_warp(l_full + t, (uint32_t)(no[t] & 1), p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const float2 a = ml_s[r], b = ml_s[BM + r];
                const float M = fmaxf(a.x, b.x), ref = M == -INFINITY ? 0.f : M;   // (-inf: only logits of -inf)
                const float fa = fast_exp2(a.x - ref), fb = fast_exp2(b.x - ref);
                const bool row_valid = head < p.group && i_pos < I.nseq;
                const int64_t row = I.row + (row_valid ? (int64_t)i_pos * p.group + head : 0);
                float *dst = p.o + row * D;
                if (row_valid) p.ml[row] = make_float2(M, a.y * fa + b.y * fb);
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o0[16], o1[16];
                    tmem_ld16(lane_addr + o_col(0) + 16 * c, o0);
                    tmem_ld16(lane_addr + o_col(1) + 16 * c, o1);
                    tmem_wait_ld();
                    if (c == D / 16 - 1) {
                        tc_fence_before();
                        mbar_arrive(o_empty);
                        mbar_arrive(o_empty + 1);
                    }
                    if (row_valid) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                x[e] = __float_as_uint(__uint_as_float(o0[8 * h + e]) * fa + __uint_as_float(o1[8 * h + e]) * fb);
                            st_global_v8(dst + 16 * c + 8 * h, x);
                        }
                    }
                }
                ++no[0];
                ++no[1];
                continue;
            }
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
                if ((t > 0 && I.kind == kTurns) || !ok) continue;
                if (!mbar_wait_warp(o_full + t, (uint32_t)(no[t] & 1), p.wait_ns) ||
                    !mbar_wait_warp(l_full + t, (uint32_t)(no[t] & 1), p.wait_ns)) {
                    ok = false;
                    continue;
                }
                tc_fence_after();
                const float2 ml = ml_s[t * BM + r];
                const int i = t * I.second + i_pos;         // sequence within the item (kPair: and kv-head)
                const bool row_valid = head < p.group && (I.kind == kPair ? i_pos : i) < I.nseq;
                const int64_t row = I.row + (row_valid ? (int64_t)i * p.group + head : 0);
                float *dst = p.o + row * D;
                if (row_valid) p.ml[row] = ml;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o0[16], o1[16];
                    tmem_ld16(lane_addr + o_col(t) + 32 * c, o0);
                    tmem_ld16(lane_addr + o_col(t) + 32 * c + 16, o1);
                    tmem_wait_ld();
                    if (c == D / 32 - 1) {       // O_t read: the next piece's products may overwrite it
                        tc_fence_before();
                        mbar_arrive(o_empty + t);
                    }
                    if (row_valid) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a[8], b[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                a[e] = (h ? o1 : o0)[e];
                                b[e] = (h ? o1 : o0)[8 + e];
                            }
                            st_global_v8(dst + 32 * c + 16 * h, a);      // whole 32-byte sectors
                            st_global_v8(dst + 32 * c + 16 * h + 8, b);
                        }
                    }
                }
                ++no[t];
            }
        }
        if (!ok && r == 0) {
            set_status(p.status, PA_ERR_TIMEOUT);
            note_wait_site(p.wait_sites, PA_WAIT_PREFILL_SOFTMAX);
        }
    } else if (warp >= kProducerWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSide));
    if (warp == kProducerWarp) {
        // ================= TMA producer
        bool ok = true, stopped = false;
        int n = 0, nq = 0, issued_end = 0;   // issued_end: ring entries issued so far
        Ring at = {0, 0};
        int64_t t_next = range_s[0];
        int place = (int)blockIdx.x % *p.plan.width;      // in the team, whose share comes first; -1: on its own
        // the next piece of this CTA's share, published one piece ahead of its use
        auto publish = [&](int it, Piece &I) -> bool {
            bool okp = true;
            if (lane == 0 && it >= kItemSlots &&
                !mbar_wait(item_empty + it % kItemSlots, (uint32_t)(((it / kItemSlots) - 1) & 1), p.wait_ns))
                okp = false;
            okp = __shfl_sync(kAll, okp ? 1 : 0, 0) != 0;
            I = Piece{};
            if (place >= 0 && t_next >= range_s[1]) {
                place = -1;
                t_next = range_s[2];
            }
            const int64_t t_end = range_s[place >= 0 ? 1 : 3];
            if (t_next < t_end) {
                const int spi = kMT * p.pos;
                const PrefixItem x = prefix_item(p.plan, p.starts, p.num_groups, p.num_kv_heads, spi, BN, p.pair_seqs,
                                                 *p.plan.width, place, t_next);
                const int i0 = x.part * spi;
                I.table_seq = x.s0;
                I.kvh = x.kvh;
                I.seq0 = x.s0 + i0;
                I.nseq = min(spi, x.n - i0);
                I.kind = x.of.pair ? kPair : I.nseq > p.pos ? kWide : kTurns;
                I.second = x.of.pair ? x.n : p.pos;
                I.tile0 = x.tile;
                I.nkv = (int)min((int64_t)(x.of.kt - x.tile), t_end - t_next);
                I.C = x.C;
                I.live = 1;
                I.row = x.tile == 0 ? item_row(x.s0, x.n, x.kvh, i0, p.num_heads, p.group)
                                    : (int64_t)p.num_seqs * p.num_heads + (2 * (int)blockIdx.x + (place >= 0 ? 1 : 0)) * (int64_t)p.item_rows;
                t_next += I.nkv;
            }
            if (lane == 0 && okp) {
                items[it % kItemSlots] = I;
                mbar_arrive(item_full + it % kItemSlots);
            }
            return okp;
        };
        // block ids of piece X, 32 per chunk (lane l holds block 32*chunk + l of the piece); past the shared tokens (or
        // invalid) the coordinate num_blocks is out of bounds and TMA fills zeros
        auto load_ids = [&](const Piece &X, int chunk) {
            const int per = X.kind == kPair ? kBlocksPerTile / 2 : kBlocksPerTile, lb = X.tile0 * per + chunk * 32 + lane;
            int coord = p.num_blocks;
            if (X.live && chunk * 32 + lane < X.nkv * per && lb < X.C / kB) {
                const int32_t blk = __ldg(p.block_tables + (int64_t)X.table_seq * p.max_blocks + lb);
                if (blk >= 0 && blk < p.num_blocks) coord = blk;
                else set_status(p.status, PA_ERR_OUT_OF_RANGE);
            }
            return coord;
        };
        Piece I, I_next;
        ok = publish(0, I);
        int pre_cur = load_ids(I, 0), pre_next = load_ids(I, 1);
        for (int it = 0; ok && I.live; ++it, I = I_next) {
            if (!publish(it + 1, I_next)) { ok = false; break; }
            int ids_cur = pre_cur, ids_next = pre_next, chunk_cur = 0;
            pre_cur = load_ids(I_next, 0);
            pre_next = load_ids(I_next, 1);
            // Q: its buffer is free once every QK product of the previous piece completed
            if (lane == 0) {
                if (nq >= 1 && !mbar_wait(q_empty, (uint32_t)((nq - 1) & 1), p.wait_ns)) ok = false;
                if (ok) {
                    const int mt = I.kind == kTurns ? 1 : kMT;
                    mbar_arrive_expect_tx(q_full, (uint32_t)(mt * kDH * p.pos * p.group * 128));
                    for (int t = 0; t < mt; ++t)
                        for (int pl = 0; pl < kDH; ++pl)
                            tma_load_4d(q_s + t * kQBytes + pl * kPlaneQ, &tmap_q, 0, I.seq0 + (I.kind == kWide ? t * p.pos : 0),
                                        (I.kvh + (I.kind == kPair ? t : 0)) * p.group, pl, q_full);
                }
            }
            ok = __shfl_sync(kAll, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            ++nq;
            const bool pair = I.kind == kPair;
            const int per = pair ? kBlocksPerTile / 2 : kBlocksPerTile;
            for (int j = 0; ok && j < I.nkv; ++j) {
                if ((j * per) / 32 != chunk_cur) {
                    ids_cur = ids_next;
                    ++chunk_cur;
                    ids_next = load_ids(I, chunk_cur + 1);
                }
                const int id0 = (j * per) & 31;
                const int cbv = __shfl_sync(kAll, ids_cur, id0 + (lane & (per - 1)));
                for (int kv = 0; kv < 2; ++kv) {
                    const int m = n + 2 * j + kv;
                    if (p.stall == PA_STALL_PRODUCER && m >= p.stall_after) {
                        stopped = true;   // test hook: entry m and later are never filled
                        ok = false;
                        break;
                    }
                    if (lane == 0 && m >= kSlots && !mbar_wait(kv_empty + at.slot, at.phase ^ 1u, p.wait_ns))
                        ok = false;
                    ok = __shfl_sync(kAll, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(kv_full + at.slot, kSlotBytes);
                    __syncwarp();
                    // lane b < per copies block b of K or V
                    if (lane < per) {
                        uint8_t *dst = kv_s + at.slot * kSlotBytes + lane * (pair ? kBlock2 : kVBlockBytes);
                        const CUtensorMap *map = kv ? (pair ? &tmap_v2 : &tmap_v) : (pair ? &tmap_k2 : &tmap_k);
                        if (kv || kB == 8) tma_load_5d(dst, map, 0, 0, 0, I.kvh, cbv, kv_full + at.slot);
                        else tma_load_5d(dst, map, 0, 0, I.kvh * kDH, 0, cbv, kv_full + at.slot);
                    }
                    issued_end = m + 1;
                    at = at.next();
                }
            }
            n += 2 * I.nkv;
        }
        if (!ok && !stopped && lane == 0) {
            set_status(p.status, PA_ERR_TIMEOUT);
            note_wait_site(p.wait_sites, PA_WAIT_PREFILL_PRODUCER);
        }
        // every copy this CTA issued has landed before the CTA may exit (default limit)
        if (lane == 0) {
            if (nq >= 1) mbar_wait(q_full, (uint32_t)((nq - 1) & 1));
            for (int m = issued_end > kSlots ? issued_end - kSlots : 0; m < issued_end; ++m)
                mbar_wait(kv_full + slot_of(m), phase_of(m));
        }
    } else if (warp == kMmaWarp) {
        // ================= MMA issuer: all lanes follow the schedule, one elected lane issues.  Tensor-pipe order, per
        // KV tile j: PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1), so one M-tile's products run while the other's softmax
        // turns S into P.  QK_t(j+1) overwrites the TMEM columns that PV_t(j) reads P_t from; the pipe runs one
        // thread's MMAs in issue order, so the read precedes the overwrite.
        const uint32_t q_addr = smem_u32(q_s), kv_addr = smem_u32(kv_s);
        const uint64_t dq = umma_desc_sw128(q_addr, 16, 1024);
        const uint64_t dk = umma_desc_sw128(kv_addr, 16, kKSbo);
        const uint64_t dv = umma_desc_sw128(kv_addr, kVLbo, kVSbo);
        // S_t = Q_tq K^T, K in ring entry nk
        auto issue_qk = [&](int t, int tq, int slot) {
            const uint32_t ko = (uint32_t)slot * kSlotBytes;
#pragma unroll
            for (int pl = 0; pl < D / 64; ++pl)
                umma_bf16_k64(tmem + s_col(t), dq + ((uint32_t)(tq * kQBytes + pl * kPlaneQ) >> 4),
                              dk + ((ko + pl * kKPlane) >> 4), kIdescQK, pl > 0 ? 1u : 0u);
        };
        // O_t (+)= P_t V over keys 64 kq .. 64 kq + 63 (4 MMAs of 16), V in ring entry nv
        auto issue_pv = [&](int t, int slot, int kq, bool first) {
            const uint32_t vo = (uint32_t)slot * kSlotBytes;
            umma_bf16_tmem_a_k64(tmem + o_col(t), tmem + s_col(t) + kq * 32, dv + ((vo + kq * kVChunk) >> 4), kIdescPV,
                                 kVS1 >> 4, kVS2 >> 4, (!first || kq > 0) ? 1u : 0u);
        };
        // tiles of two kv-heads: S_t = Q_t K_t^T and O_t (+)= P_t V_t over 64 keys, head t of ring entry nk / nv; b: S's place
        const uint64_t dk2 = umma_desc_sw128(kv_addr, 16, kKSboP), dv2 = umma_desc_sw128(kv_addr, kVLbo, kVSboP);
        auto issue_qk2 = [&](int t, int b, int slot) {
            const uint32_t ko = (uint32_t)slot * kSlotBytes + t * (kDH * 1024);
#pragma unroll
            for (int pl = 0; pl < D / 64; ++pl)
                umma_bf16_k64(tmem + s_col(t) + b * 64, dq + ((uint32_t)(t * kQBytes + pl * kPlaneQ) >> 4),
                              dk2 + ((ko + pl * kKPlane) >> 4), kIdescQK2, pl > 0 ? 1u : 0u);
        };
        auto issue_pv2 = [&](int t, int b, int slot, bool first) {
            const uint32_t vo = (uint32_t)slot * kSlotBytes + t * kVBlockBytes;
            umma_bf16_tmem_a_k64(tmem + o_col(t), tmem + s_col(t) + b * 64, dv2 + (vo >> 4), kIdescPV, kVS1p >> 4, kVS2p >> 4,
                                 first ? 0u : 1u);
        };
        bool ok = true, stopped = false;
        int n = 0, nq = 0;
        int J0 = 0, J1 = 0, no0 = 0, no1 = 0;   // per M-tile: tiles (other than kPair's) and pieces so far
        int U0 = 0, U1 = 0;                     // kPair: uses of S's places so far
        for (int it = 0; ok; ++it) {
            Piece I;
            if (!take_item(it, I)) { ok = false; break; }
            if (!I.live) break;
            const int nkv = __shfl_sync(kAll, I.nkv, 0);
            const int kind = __shfl_sync(kAll, I.kind, 0);
            if (p.stall == PA_STALL_CONSUMER && n >= p.stall_after) { stopped = true; ok = false; break; }
            if (!mbar_wait_warp(q_full, (uint32_t)(nq & 1), p.wait_ns) ||
                !mbar_wait_warp(kv_full + slot_of(n), phase_of(n), p.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // the piece's first product into O_t overwrites it: the output warpgroup has read the last piece's
            auto o_free = [&](int t) -> bool {
                const int no = t ? no1 : no0;
                return no == 0 || mbar_wait_warp(o_empty + t, (uint32_t)((no - 1) & 1), p.wait_ns);
            };
            // O_t's half products with V in the ring's `slot`, as P_t comes; x: M-tile t's tiles so far in this piece; half:
            // whether its first half was seen to be there
            auto pv = [&](int t, int slot, int x, uint32_t half) -> bool {
                const uint32_t ph = (uint32_t)(((t ? J1 : J0) + x) & 1);
                if (x == 0 && !o_free(t)) return false;
                if (!wait_unless(half, p_half + t, ph, p.wait_ns)) return false;
                tc_fence_after();
                const uint32_t rest = peek(p_full + t, ph);
                issue_pv(t, slot, 0, x == 0);
                if (!wait_unless(rest, p_full + t, ph, p.wait_ns)) return false;
                tc_fence_after();
                issue_pv(t, slot, 1, x == 0);
                return true;
            };
            auto peek_half = [&](int t, int x) { return peek(p_half + t, (uint32_t)(((t ? J1 : J0) + x) & 1)); };
            Ring rk = {slot_of(n), phase_of(n)};     // K of the tile at hand
            if (kind == kPair) {
                // QK_0(j+1) QK_1(j+1) PV_0(j) PV_1(j): the next tile's logits are under way while the softmax
                // warpgroups turn this one's into weights
#pragma unroll
                for (int t = 0; t < kMT; ++t) {
                    issue_qk2(t, 0, rk.slot);
                    umma_commit(s2_full + t);
                }
                if (nkv == 1) umma_commit(q_empty);
                umma_commit(kv_empty + rk.slot);
                for (int j = 0; j < nkv; ++j) {
                    const int nv = n + 2 * j + 1, b = j & 1;
                    const Ring rv = rk.next();
                    rk = rv.next();
                    // test hook: stop, leaving ring entries unreleased, so the producer's wait runs out
                    if (p.stall == PA_STALL_CONSUMER && nv >= p.stall_after) { stopped = true; ok = false; break; }
                    if (!mbar_wait_warp(kv_full + rv.slot, rv.phase, p.wait_ns)) { ok = false; break; }
                    if (j + 1 < nkv) {
                        if (!mbar_wait_warp(kv_full + rk.slot, rk.phase, p.wait_ns)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll
                        for (int t = 0; t < kMT; ++t) {
                            issue_qk2(t, b ^ 1, rk.slot);
                            umma_commit(s2_full + (b ^ 1) * kMT + t);
                        }
                        umma_commit(kv_empty + rk.slot);
                        if (j + 2 == nkv) umma_commit(q_empty);    // the piece's last QK products
                    }
#pragma unroll
                    for (int t = 0; t < kMT; ++t) {
                        if (!ok || (j == 0 && !o_free(t)) ||
                            !mbar_wait_warp(p2_full + b * kMT + t, (uint32_t)(((b ? U1 : U0) + (j >> 1)) & 1), p.wait_ns)) {
                            ok = false;
                            continue;
                        }
                        tc_fence_after();
                        issue_pv2(t, b, rv.slot, j == 0);
                        if (j + 1 == nkv) umma_commit(o_full + t);
                    }
                    if (!ok) break;
                    umma_commit(kv_empty + rv.slot);
                }
            } else if (kind == kWide) {
#pragma unroll
                for (int t = 0; t < kMT; ++t) {
                    issue_qk(t, t, rk.slot);
                    umma_commit(s_full + t);
                }
                if (nkv == 1) umma_commit(q_empty);
                umma_commit(kv_empty + rk.slot);
                uint32_t half = 0, v_in = 0, k_in = 0;
                for (int j = 0; j < nkv; ++j) {
                    const bool next = j + 1 < nkv;
                    const int nv = n + 2 * j + 1;
                    const Ring rv = rk.next();
                    rk = rv.next();
                    if (p.stall == PA_STALL_CONSUMER && nv >= p.stall_after) { stopped = true; ok = false; break; }
                    if (!wait_unless(v_in, kv_full + rv.slot, rv.phase, p.wait_ns)) { ok = false; break; }
#pragma unroll
                    for (int t = 0; t < kMT; ++t) {
                        if (t == 0) k_in = peek(kv_full + rk.slot, rk.phase);
                        if (!ok || !pv(t, rv.slot, j, half)) { ok = false; continue; }
                        if (next) {
                            if (t == 0 && !wait_unless(k_in, kv_full + rk.slot, rk.phase, p.wait_ns)) { ok = false; continue; }
                            tc_fence_after();
                            if (t == 1) v_in = peek(kv_full + rk.next().slot, rk.next().phase);
                            half = peek_half(t ^ 1, j + t);
                            issue_qk(t, t, rk.slot);
                            umma_commit(s_full + t);
                        } else {
                            half = peek_half(1, j);
                            umma_commit(o_full + t);
                        }
                    }
                    if (!ok) break;
                    umma_commit(kv_empty + rv.slot);
                    if (next) {
                        umma_commit(kv_empty + rk.slot);
                        if (j + 2 == nkv) umma_commit(q_empty);    // the piece's last QK products
                    }
                }
            } else {
                // M-tile t takes KV tiles t, t + 2, ...: PV_t(x) QK_t(x + 2), t = x & 1
                for (int x = 0; x < 2 && x < nkv; ++x) {
                    const int nk = n + 2 * x;
                    if (x > 0 && p.stall == PA_STALL_CONSUMER && nk >= p.stall_after) { stopped = true; ok = false; break; }
                    if (x > 0 && !mbar_wait_warp(kv_full + slot_of(nk), phase_of(nk), p.wait_ns)) { ok = false; break; }
                    tc_fence_after();
                    issue_qk(x, 0, slot_of(nk));
                    umma_commit(s_full + x);
                    umma_commit(kv_empty + slot_of(nk));
                }
                if (ok && nkv <= 2) umma_commit(q_empty);
                for (int x = 0; ok && x < nkv; ++x) {
                    const int t = x & 1, nv = n + 2 * x + 1, nk = n + 2 * x + 4;
                    if (p.stall == PA_STALL_CONSUMER && nv >= p.stall_after) { stopped = true; ok = false; break; }
                    if (!mbar_wait_warp(kv_full + slot_of(nv), phase_of(nv), p.wait_ns) || !pv(t, slot_of(nv), x >> 1, 0)) { ok = false; break; }
                    umma_commit(kv_empty + slot_of(nv));
                    if (x + 2 < nkv) {
                        if (!mbar_wait_warp(kv_full + slot_of(nk), phase_of(nk), p.wait_ns)) { ok = false; break; }
                        tc_fence_after();
                        issue_qk(t, 0, slot_of(nk));
                        umma_commit(s_full + t);
                        umma_commit(kv_empty + slot_of(nk));
                        if (x + 3 == nkv) umma_commit(q_empty);
                    } else {
                        umma_commit(o_full + t);
                    }
                }
            }
            n += 2 * nkv;
            ++nq;
            if (kind == kPair) {
                U0 += (nkv + 1) >> 1;
                U1 += nkv >> 1;
            } else {
                J0 += kind == kWide ? nkv : (nkv + 1) >> 1;
                J1 += kind == kWide ? nkv : nkv >> 1;
            }
            ++no0;
            no1 += kind != kTurns || nkv > 1 ? 1 : 0;
        }
        if (!ok && !stopped && lane == 0) {
            set_status(p.status, PA_ERR_TIMEOUT);
            note_wait_site(p.wait_sites, PA_WAIT_PREFILL_MMA);
        }
        // drain (default limit): everything issued must finish before TMEM is released
        umma_commit(drained);
        mbar_wait_warp(drained, 0);
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ================= softmax warpgroup t: thread r owns row r of M-tile t
        const int t = warp >> 2;
        const int r = tid & (BM - 1);
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl2 = p.scale_log2;
        bool ok = true;
        int no = 0, n_next = 0, J = 0, U0 = 0, U1 = 0;    // pieces, ring entries, tiles (kPair: by S_t's place) so far
        for (int it = 0; ok; ++it) {
            Piece I;
            if (!take_item(it, I)) { ok = false; break; }
            if (!I.live) break;
            const int mine = I.tiles(t), n = n_next;
            n_next += 2 * I.nkv;
            if (mine == 0) continue;
            float m = -INFINITY, l = 0.f;
            // One tile: S to P.  S is read whole and its max taken first; 128 keys of P then go out in two halves (the
            // tensor pipe takes the first while the second is computed).  The piece's first tile takes its own max;
            // later ones run with the running max m: P stays <= 2^8 unless the tile's max exceeds it by more than 8,
            // and then (rarely) the row moves its max and rescales O first.  While all logits were -inf the max stays
            // -inf, the weights 0 (taken against 0), and the first finite tile moves it, however low it lies.  lim: shared
            // keys from the tile's first on; nv: ring entry of the last tile's values.  bar, out: S written, P's first
            // half (all 64 keys) written.
            auto tile = [&](auto keys, uint32_t col, uint64_t *bar, uint64_t *out, uint32_t phase, int lim, bool first,
                            int nv) -> bool {
                constexpr int kN = decltype(keys)::value;
                if (!mbar_wait_warp(bar, phase, p.wait_ns)) return false;
                tc_fence_after();
                uint32_t sr[kN / 32][32];
                auto mask = [&](int c) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e >= lim) sr[c][e] = __float_as_uint(-INFINITY);
                };
                float a0 = -INFINITY, a1 = -INFINITY;
                auto max_of = [&](int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        a0 = fmax3(a0, __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
                        a1 = fmax3(a1, __uint_as_float(sr[c][e + 2]), __uint_as_float(sr[c][e + 3]));
                    }
                };
                tmem_ld32(col, sr[0]);
                tmem_ld32(col + 32, sr[1]);
                tmem_wait_ld_regs(sr[0], sr[1]);
                if constexpr (kN == BN) {
                    tmem_ld32(col + 64, sr[2]);
                    tmem_ld32(col + 96, sr[3]);
                }
                if (lim < kN) { mask(0); mask(1); }
                max_of(0);
                max_of(1);
                if constexpr (kN == BN) {
                    tmem_wait_ld_regs(sr[2], sr[3]);
                    if (lim < kN) { mask(2); mask(3); }
                    max_of(2);
                    max_of(3);
                }
                const float m_tile = fmaxf(a0, a1) * sl2;
                if (first) {
                    m = m_tile;
                } else {
                    const bool need = m_tile > m + 8.f;
                    if (__any_sync(kAll, need)) {
                        const float alpha = need ? fast_exp2(m - m_tile) : 1.f;
                        l *= alpha;
                        // O_t's earlier products are done: with 128 keys they completed before this S was committed;
                        // with 64, whose S comes a tile early, their values' ring entry must have been released (it
                        // is not used and released again before this tile's P is out)
                        if (kN != BN && !mbar_wait_warp(kv_empty + slot_of(nv), phase_of(nv), p.wait_ns)) return false;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(lane_addr + o_col(t) + 32 * c, o);
                            tmem_wait_ld();
                            reg_fence32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(lane_addr + o_col(t) + 32 * c, o);
                        }
                        if (need) m = m_tile;
                    }
                }
                // P for 32 key pairs into pk, rounded to bf16 (the products' operand type): independent roundings of
                // half a step, beside a result rounded to bf16 itself; l sums the unrounded values
                const float neg = m == -INFINITY ? 0.f : -m;
                const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(neg, neg);
                float2 ls = make_float2(0.f, 0.f);
                uint32_t pk[32];
                auto pass = [&](auto u0c) {
                    constexpr int u0 = decltype(u0c)::value;
#pragma unroll
                    for (int u = u0; u < u0 + 32; ++u) {
                        const float s0 = __uint_as_float(sr[u >> 4][(2 * u) & 31]);
                        const float s1 = __uint_as_float(sr[u >> 4][(2 * u + 1) & 31]);
                        const float2 x = fma_f32x2(make_float2(s0, s1), sl2x2, negm);
                        const float p0 = fast_exp2(x.x);
                        const float p1 = fast_exp2(x.y);
                        ls = add_f32x2(ls, make_float2(p0, p1));
                        pk[u - u0] = pack_bf16x2(p0, p1);
                    }
                };
                pass(std::integral_constant<int, 0>{});
                tmem_st32(col, pk);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(out);
                if constexpr (kN == BN) {
                    pass(std::integral_constant<int, 32>{});
                    tmem_st32(col + 32, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full + t);
                }
                l += ls.x + ls.y;
                return true;
            };
            const uint32_t col = lane_addr + s_col(t);
            for (int j = 0; j < mine; ++j) {
                if (I.kind == kPair) {
                    const int b = j & 1;
                    ok = tile(std::integral_constant<int, BN / 2>{}, col + b * 64, s2_full + b * kMT + t, p2_full + b * kMT + t,
                              (uint32_t)((b ? U1++ : U0++) & 1), I.C - (I.tile0 + j) * (BN / 2), j == 0, n + 2 * j - 1);
                } else {
                    ok = tile(std::integral_constant<int, BN>{}, col, s_full + t, p_half + t, (uint32_t)(J++ & 1),
                              I.C - (I.tile0 + (I.kind == kWide ? j : 2 * j + t)) * BN, j == 0, 0);
                }
                if (!ok) break;
            }
            if (!ok) break;
            // (m, l) for the output warpgroup, which read the last piece's before it released O_t
            if (no > 0 && !mbar_wait_warp(o_empty + t, (uint32_t)((no - 1) & 1), p.wait_ns)) { ok = false; break; }
            ml_s[t * BM + r] = make_float2(m, l);
            mbar_arrive(l_full + t);
            ++no;
        }
        if (!ok && r == 0) {
            set_status(p.status, PA_ERR_TIMEOUT);
            note_wait_site(p.wait_sites, PA_WAIT_PREFILL_SOFTMAX);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    grid_dependency_wait();
}

CUresult encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                const cuuint32_t *box) {
    auto fn = tensor_map_encoder();
    if (!fn) return CUDA_ERROR_NOT_FOUND;
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// q [num_seqs][num_heads][D]: one plane of `pos` sequences x `group` heads lands as [head][sequence][64]
CUresult make_q_map(CUtensorMap *map, const void *q, int num_seqs, int num_heads, int D, int pos, int group) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)num_seqs, (cuuint64_t)num_heads, (cuuint64_t)(D / 64)};
    const cuuint64_t strides[3] = {(cuuint64_t)num_heads * D * 2, (cuuint64_t)D * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)pos, (cuuint32_t)group, 1};
    return encode(map, q, 4, dims, strides, box);
}

// One block of `heads` kv-heads: [kv-head][plane][B rows][64]
CUresult make_v_map(CUtensorMap *map, const void *pool, int num_blocks, int kB, int hkv, int D, int heads) {
    const cuuint64_t dims[5] = {64, (cuuint64_t)kB, (cuuint64_t)(D / 64), (cuuint64_t)hkv, (cuuint64_t)num_blocks};
    const cuuint64_t strides[4] = {(cuuint64_t)hkv * D * 2, 128, (cuuint64_t)D * 2, (cuuint64_t)kB * hkv * D * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)kB, (cuuint32_t)(D / 64), (cuuint32_t)heads, 1};
    return encode(map, pool, 5, dims, strides, box);
}

// One block of `heads` kv-heads: [8-row group][kv-head][plane][8 rows][64] (at B = 8 the map above gives the same)
CUresult make_k_map(CUtensorMap *map, const void *pool, int num_blocks, int kB, int hkv, int D, int heads) {
    if (kB == 8) return make_v_map(map, pool, num_blocks, kB, hkv, D, heads);
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)hkv * (D / 64), (cuuint64_t)(kB / 8), (cuuint64_t)num_blocks};
    const cuuint64_t strides[4] = {(cuuint64_t)hkv * D * 2, 128, (cuuint64_t)8 * hkv * D * 2, (cuuint64_t)kB * hkv * D * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)(heads * (D / 64)), (cuuint32_t)(kB / 8), 1};
    return encode(map, pool, 5, dims, strides, box);
}

template <int D, int B>
cudaError_t launch_main(const CUtensorMap (&m)[5], const PrefixParams &prm, int grid, cudaStream_t stream) {
    const size_t smem = Shape<D>::kSmem;
    auto kern = prefix_kernel<D, B>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(grid), dim3(kThreads), smem, stream, m[0], m[1], m[2], m[3], m[4], prm);
}

}  // namespace

int prefix_seqs_per_item(int group) { return kMT * (BM / group); }

cudaError_t launch_prefix(const AttnArgs &a, const SharedJob &job, cudaStream_t stream) {
    const int G = a.num_heads / a.num_kv_heads;
    CUtensorMap m[5];   // q, then K and V of one kv-head, of two
    const int two = a.num_kv_heads > 1 ? 2 : 1;
    if (make_q_map(&m[0], a.q, a.num_seqs, a.num_heads, a.head_dim, BM / G, G) != CUDA_SUCCESS) return cudaErrorNotSupported;
    for (int i = 0; i < 2; ++i)
        if (make_k_map(&m[1 + 2 * i], a.k_cache, a.num_blocks, a.block_size, a.num_kv_heads, a.head_dim, i ? two : 1) != CUDA_SUCCESS ||
            make_v_map(&m[2 + 2 * i], a.v_cache, a.num_blocks, a.block_size, a.num_kv_heads, a.head_dim, i ? two : 1) != CUDA_SUCCESS)
            return cudaErrorNotSupported;
    PrefixParams prm;
    prm.plan = job.plan;
    prm.starts = job.groups.starts;
    prm.block_tables = a.block_tables;
    prm.shares = job.shares;
    prm.o = job.pre_o;
    prm.ml = job.pre_ml;
    prm.num_seqs = a.num_seqs;
    prm.num_groups = job.groups.num_groups;
    prm.num_heads = a.num_heads;
    prm.num_kv_heads = a.num_kv_heads;
    prm.pair_seqs = job.groups.pair_seqs;
    prm.group = G;
    prm.pos = BM / G;
    prm.item_rows = job.item_rows;
    prm.max_blocks = a.max_blocks;
    prm.num_blocks = a.num_blocks;
    prm.scale_log2 = a.scale * 1.4426950408889634f;
    prm.status = a.status;
    const WaitTest &wt = wait_test();
    prm.wait_ns = wt.limit_ns;
    prm.stall = wt.stall;
    prm.stall_after = wt.after;
    prm.wait_sites = wt.sites;
    const int grid = prefix_grid();
    switch (a.head_dim * 100 + a.block_size) {
        case 6408: return launch_main<64, 8>(m, prm, grid, stream);
        case 6416: return launch_main<64, 16>(m, prm, grid, stream);
        case 6432: return launch_main<64, 32>(m, prm, grid, stream);
        case 12808: return launch_main<128, 8>(m, prm, grid, stream);
        case 12816: return launch_main<128, 16>(m, prm, grid, stream);
        case 12832: return launch_main<128, 32>(m, prm, grid, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa
