// attn_decode_q4.cu -- paged decode attention over 4-bit pools (q4_format.cuh):
//     out[s][h] = sum_j softmax_j(scale <q[s][h], K_s[j][g]>) V_s[j][g]
// with K and V the values their codes and scales stand for.
//
// What it has to move is 4.5 bits a cached value, 3.6 times less than a bf16
// cache; the bound that comes up before HBM is the instruction issue of turning
// nibbles into matrix operands, so the kernel is built to spend little there
// (bf16 queries; fp32 below):
//  * A nibble is an operand as it stands: in the low 4 bits of an fp16 it is
//    the number n 2^-24, in the next 4 bits n 2^-20 (subnormals, which the
//    matrix instructions take exactly), so an AND makes two of them and one
//    shift serves four.  Scales are never multiplied into elements, and the 8
//    in n - 8 is taken off sums, not off elements.  (e4m3 operands would take
//    a nibble as well, but that mma.sync is itself made of conversions and
//    fp16 products: 16 x 32768 tokens took 187 us with it, 151 us with fp16.)
//  * S = K Q^T (tokens in M, q-heads in N, m16n8k16): q in fp16 times a power of
//    two per head that brings its largest element into [2^14, 2^15), in the
//    dims of the upper nibbles (1, 3, 5, 7 mod 8) divided by the 16 that those
//    carry: elements are exact down to 2^-31 of the head's largest in the even
//    dims, to 2^-27 in the odd ones.  The group's scale is applied to the 4 sums
//    of a lane, and the -8 sum(q) scale of all groups is one more product, of
//    the scales with -8 sum(q) in three bf16 parts.
//  * O^T += V^T P^T (dims in M, tokens in K): the token's scale of V goes into
//    the weight, once per group, and the product is rounded to fp16 (2^-11).
//    The scales are first brought up by a power of two of their group (packed
//    products, two scales each), which took the group's largest scale into
//    [2^6, 2^7) when it was set and is set anew when one passes 2^8: with
//    weights up to 2^7 nothing overflows, a product 2^-20 of the group's
//    largest still has its 11 bits, and no group loses to another, as it did
//    under one power for all four (16 x 32768 tokens 115.8 us with one, 117.4
//    with four; groups told apart only where they differ, by a check or a form
//    of their own, took 119.5 to 125).  The 8 is taken off by a product of the
//    same weights with -8 right after: a sum over many tokens would otherwise
//    lose a small result under 8 times its weights.
//  * The softmax reference of a head moves only when a logit passes it by 7
//    (base 2), found by one warp vote a step: weights stay below 2^7 and sums
//    are rescaled a few times a sequence instead of every step.
//  * A warp takes units of 16 tokens of one sequence and kv-head through a ring
//    of its own in shared memory (16-byte asynchronous copies), two a step
//    where it can: nothing is shared between warps until their pieces are
//    merged.  12 warps of 168 registers an SM; 16 of 128 spilled (151 us
//    against 134 at that stage, 16 x 32768 tokens), 10 took 155 against 126.
//
// The batch is one stream of units, (sequence, kv-head, 16 tokens); every CTA
// takes an equal contiguous share and every warp of it an equal part, whatever
// the mix of lengths.  What a new (sequence, kv-head) costs a warp beside its
// units (queries, first block ids, normalising or leaving a piece) counts as
// kHeadCost units of the stream in front of it (256 power-law sequences: 42.5 us
// with 2, 40.3 with 3, 41.6 with 5, and 90 against 60 at an early stage with
// none).  A (sequence, kv-head) inside one warp is normalised and stored; cut
// ones leave (m, l, o) pieces, merged first between the warps of a CTA (shared
// memory), then, where a CTA boundary cuts a head, by a second small kernel
// (workspace), always in stream order, so results do not depend on timing.
// Every CTA finds its share by itself, from a prefix sum over the lengths in
// shared memory; only batches of more than kScanSeqs sequences have it made by
// a kernel of its own.  Over short tables a CTA takes whole heads, one or
// several, and there is no second kernel.
//
// Measured (32 / 8 heads of 128, blocks of 16): 256 power-law sequences, 151 MB,
// 40.8 us; 16 x 32768 tokens, 604 MB, 116.5 us = 5.2 TB/s, 0.76 of the copy
// peak, at 62 % of the issue slots and 55 % of the ALU pipe, 310 instructions a
// unit and warp; with the products left out its copies take 96 us.  A short
// request takes 5.6 us.
//
// fp32 queries: q and the weights are split into three bf16 parts each (24
// bits), and the codes are brought to n - 8 one by one (0x4300 | n is 128 + n
// in bf16), so that no sum carries a surplus.
#include <math.h>

#include <atomic>
#include <type_traits>

#include <cuda_fp16.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kU = 16;              // tokens a unit: the M of the first product, the K of the second
constexpr int kStages = 4;
constexpr int kPlanThreads = 1024;
constexpr int kMaxCtas = 512;
constexpr int kScanSeqs = 4096;     // sequences whose prefix a CTA makes itself (48 KB of shared memory)
constexpr int kHeadCost = 3;
constexpr float kMoveAt = 7.0f;     // a logit this far (base 2) over the reference moves it

// A head cut at the end of CTA c (seq < 0: none): its pieces are c's second, then the first of c + 1 .. last.
struct Cut { int seq, vh, last, pad; };

struct Q4Params {
    const void *q;
    void *out;
    const uint8_t *k, *v;
    const int32_t *block_tables, *context_lens;
    int64_t *prefix;           // [num_seqs + 1] stream length of one head before each sequence (not `scan`)
    struct Cut *cuts;          // [CTAs] the head cut at each CTA's end
    float *part;               // [CTAs][2][heads][D + 2]
    int scan;                  // the CTAs make the prefix themselves
    int by_head;               // CTA i takes head i
    int whole;                 // the CTAs' shares end between heads
    int num_seqs, num_heads, num_kv_heads;
    int group;                 // q-heads per kv-head
    int split;                 // parts a group is split into
    int hw;                    // q-heads of a part
    int log2b, max_blocks, num_blocks;
    uint32_t slab, block_bytes;
    float scale_log2;
    int vec;                   // q rows and out rows take wide loads and stores
    int32_t *status;
};

__device__ __forceinline__ int units_of(int ctx, int max_tokens) {
    return ctx <= 0 || ctx > max_tokens ? 0 : (ctx - 1) / kU + 1;
}

// A head of a sequence in the stream: its units and what it costs beside them.
__device__ __forceinline__ int length_of(int nu) { return nu ? nu + kHeadCost : 0; }

// Exclusive prefix of the sequences' stream lengths, by a CTA of kT threads.  `ctxs`, if set, receives the lengths.
template <int kT>
__device__ __forceinline__ void prefix_of(const int32_t *__restrict__ context_lens, int num_seqs, int max_tokens,
                                          int64_t *prefix, int32_t *ctxs, int64_t *warp_tot, int32_t *status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t running = 0;
    for (int base = 0; base < num_seqs; base += kT) {
        const int s = base + tid;
        int len = 0;
        if (s < num_seqs) {
            const int ctx = __ldg(context_lens + s);
            len = length_of(units_of(ctx, max_tokens));
            if (len == 0) set_status(status, PA_ERR_OUT_OF_RANGE);
            if (ctxs) ctxs[s] = ctx;
        }
        int64_t incl = len;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        int64_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kT / 32; ++w) {
            const int64_t t = warp_tot[w];
            before += w < warp ? t : 0;
            all += t;
        }
        if (s < num_seqs) prefix[s] = running + before + incl - len;
        running += all;
        __syncthreads();
    }
    if (tid == 0) prefix[num_seqs] = running;
}

__global__ void __launch_bounds__(kPlanThreads)
    q4_plan_kernel(const int32_t *__restrict__ context_lens, int num_seqs, int max_tokens, int64_t *prefix,
                   int32_t *status) {
    __shared__ int64_t warp_tot[kPlanThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    prefix_of<kPlanThreads>(context_lens, num_seqs, max_tokens, prefix, nullptr, warp_tot, status);
}

__device__ __forceinline__ uint32_t nibbles_128(uint32_t w) {   // 128 + nibble 0 | 128 + nibble 4 << 16, bf16
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(r) : "r"(w), "r"(0x43004300u));
    return r;
}
__device__ __forceinline__ uint32_t minus_136(uint32_t a) {     // exact: 128 + n -> n - 8
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x43084308u));
    return r;
}
// D = A(16x16, row) * B(16x8, col) + D, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a chain: D = A B.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// Nibbles i and i + 4 of w (i = 0..3) as an fp16 pair: n 2^-24 (i even) or n 2^-20 (i odd).
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t w, int i) {
    return (i < 2 ? w : w >> 8) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The largest scales that powers of two `up` take to less than 2^8 (bf16 pairs): exponent fields 261 - up's.
__device__ __forceinline__ uint32_t cap_of(uint32_t up) { return 0x82ff82ffu - up; }
__device__ __forceinline__ void cp_async16(uint32_t smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The NG bf16 scales of a row in shared memory, and one of them.
template <int NG> __device__ __forceinline__ void load_scales(uint32_t (&w)[NG / 2], const uint8_t *at) {
    if constexpr (NG == 4) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(at);
    else w[0] = *reinterpret_cast<const uint32_t *>(at);
}
template <int N> __device__ __forceinline__ float scale_of(const uint32_t (&w)[N], int g) {
    return __uint_as_float(g & 1 ? w[g / 2] & 0xffff0000u : w[g / 2] << 16);
}
__device__ __forceinline__ float bf16_part(float &x) {          // the leading bf16 of x, taken off it
    const float h = __bfloat162float(__float2bfloat16_rn(x));
    x -= h;
    return h;
}

// A value that is the same in all lanes, marked as such: code that depends on it alone then runs on the warp's
// uniform registers and branches, beside the lanes' arithmetic.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// a / b of non-negative values, with 32-bit division where a allows it (a tenth of the instructions)
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The last sequence s with prefix[s] <= t, by the warp, 33 ways a step.
__device__ __forceinline__ int find_seq(const int64_t *prefix, int num_seqs, int64_t t, int lane) {
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int64_t n = hi - lo;
        const bool le = prefix[lo + (int)(n * (lane + 1) / 33)] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        hi = c < 32 ? lo + (int)(n * (c + 1) / 33) : hi;
        lo = c > 0 ? lo + (int)(n * c / 33) : lo;
    }
    return lo;
}

template <typename T, int D, int NT>
struct Q4Shape {
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int kWarps = NT == 1 && !kF32 ? 12 : 8;   // one CTA per SM
    static constexpr int NS = kF32 ? 3 : 1;           // bf16 parts of q and of a weight
    static constexpr int NG = D / kQ4Group;
    static constexpr int HW = 8 * NT;                 // q-heads a warp has room for
    static constexpr int kCodes = kU * D / 2;         // bytes of a unit's codes, K or V
    static constexpr int kScales = kU * NG * 2;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kRing = kStages * kStage;
    static constexpr int kPiece = HW * (D + 2);       // floats: o [HW][D], (m, l) [HW][2]
    static constexpr int kSmem = kWarps * (kRing + kPiece * 4);
    static constexpr int kSmemMost = kSmem + (kScanSeqs + 2) * 12;
    static_assert(kSmemMost <= 226 * 1024, "fits an SM");
    static_assert(kRing >= kPiece * 4, "a drained ring holds a piece");
};

struct PieceMeta { int seq, vh, u0, u1, nu; };   // units [u0, u1) of nu; seq < 0: none

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Q4Shape<T, D, NT>::kWarps * 32, 1) q4_decode_kernel(const Q4Params p) {
    using S = Q4Shape<T, D, NT>;
    constexpr int NG = S::NG, NS = S::NS, HW = S::HW, kWarps = S::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PieceMeta meta[2 * kWarps];
    __shared__ int64_t warp_tot[kWarps];
    __shared__ int64_t share_s[3];   // of the stream: from, to, and a CTA's usual length
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), r = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + warp * S::kRing;
    float *first_piece = reinterpret_cast<float *>(smem + kWarps * S::kRing) + warp * S::kPiece;
    const int VH = p.num_kv_heads * p.split, B = 1 << p.log2b, max_tokens = p.max_blocks << p.log2b;
    if (lane == 0) meta[2 * warp].seq = meta[2 * warp + 1].seq = -1;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t *prefix = p.prefix;
    const int32_t *ctxs = p.context_lens;
    if (p.scan) {
        int64_t *pre = reinterpret_cast<int64_t *>(smem + S::kSmem);
        int32_t *cx = reinterpret_cast<int32_t *>(pre + p.num_seqs + 1);
        prefix_of<kWarps * 32>(p.context_lens, p.num_seqs, max_tokens, pre, cx, warp_tot,
                               blockIdx.x == 0 ? p.status : nullptr);
        __syncthreads();
        prefix = pre;
        ctxs = cx;
    }
    if (warp == 0) {   // the CTA's share of the stream
        const int64_t total = prefix[p.num_seqs] * VH;
        // at least a unit a warp: small batches use fewer CTAs and merge in shared memory
        const int64_t share = max((int64_t)kWarps, quotient(total + gridDim.x - 1, gridDim.x));
        int64_t from = min(total, share * blockIdx.x), to = min(total, from + share);
        if (p.by_head) {
            const int s = blockIdx.x / VH, len = (int)(prefix[s + 1] - prefix[s]);
            from = prefix[s] * VH + (int64_t)(blockIdx.x - s * VH) * len;
            to = from + len;
        } else if (p.whole) {   // up to the next head's beginning
#pragma unroll 1
            for (int end = 0; end < 2; ++end) {
                int64_t x = end ? to : from;
                if (x < total) {
                    const int s = find_seq(prefix, p.num_seqs, quotient(x, VH), lane);
                    const int len = (int)(prefix[s + 1] - prefix[s]);
                    x = prefix[s] * VH + quotient(x - prefix[s] * VH + len - 1, len) * len;
                }
                (end ? to : from) = x;
            }
        } else if (lane == 0) {
            p.cuts[blockIdx.x].seq = -1;
        }
        if (lane == 0) {
            share_s[0] = from;
            share_s[1] = to;
            share_s[2] = share;
        }
    }
    __syncthreads();
    const int64_t cta0 = share_s[0], cta1 = share_s[1];
    if (cta0 == cta1) return;
    const int64_t w0 = cta0 + quotient((cta1 - cta0) * warp, kWarps), w1 = cta0 + quotient((cta1 - cta0) * (warp + 1), kWarps);

    if (w1 > w0) {
        // ---- where the warp's part begins
        int s = uniform(find_seq(prefix, p.num_seqs, quotient(w0, VH), lane));
        int ctx = uniform(ctxs[s]), nu = units_of(ctx, max_tokens);
        const int64_t in_seq = w0 - prefix[s] * VH;
        int vh = uniform((int)quotient(in_seq, length_of(nu)));
        const int into = uniform((int)(in_seq - (int64_t)vh * length_of(nu)));
        int u = max(0, into - kHeadCost);
        int left = uniform((int)(w1 - w0)) - max(0, kHeadCost - into);   // of the part, in stream units
        // ---- the copies' own place in the stream, kStages units ahead: a stretch is the units whose block ids the
        // lanes hold (id i of the stretch in lane i); the next stretch's ids are requested one stretch early
        int cs = s, cctx = ctx, cnu = nu, cvh = vh, cu = u, cleft = left;   // the next stretch
        int next_len = 0, next_ids = 0, ids_seq = -1, ids_base = 0;
        int stretch = 0, id_at = 0, half = 0, ids = 0;
        const uint32_t ring_a = smem_u32(ring);
        uint32_t wr = ring_a;
        const int v_sw = lane ^ (2 * ((lane / NG >> 2) & 3));      // swizzled place of V's chunk `lane`
        const int k_sw = D == 64 ? lane ^ (4 * ((lane / NG >> 2) & 1)) : lane;
        const int chunk = D == 128 ? lane : lane & 15;
        const uint8_t *k_src, *v_src, *sc_src;
        auto request = [&]() {
            if (cu == cnu) {
                cu = 0;
                cleft -= kHeadCost;
                if (++cvh == VH && cleft > 0) {
                    cvh = 0;
                    do {
                        cctx = uniform(ctxs[++cs]);
                        cnu = units_of(cctx, max_tokens);
                    } while (cnu == 0);
                }
            }
            next_len = 0;
            if (cleft <= 0) return;
            const int b = (int)(((unsigned)cu * kU) >> p.log2b);
            if (cs != ids_seq || b != ids_base) {
                ids_seq = cs;
                ids_base = b;
                const int64_t e = (int64_t)b + lane;
                next_ids = 0;   // behind the sequence or out of range: block 0 is read and not used
                if ((e << p.log2b) < cctx) next_ids = __ldg(p.block_tables + (int64_t)cs * p.max_blocks + e);
            }
            const int held = p.log2b == 4 ? 32 : p.log2b == 3 ? 16 : 64 - (cu & 1);
            next_len = min(min(cnu - cu, held), cleft);
            cleft -= next_len;
        };
        auto next_stretch = [&]() {
            stretch = next_len;
            if (stretch == 0) return;
            if (next_ids < 0 || next_ids >= p.num_blocks) {
                set_status(p.status, PA_ERR_OUT_OF_RANGE);
                next_ids = 0;
            }
            ids = next_ids;
            id_at = 0;
            half = p.log2b == 5 ? cu & 1 : 0;
            const uint64_t at = (uint64_t)(uint32_t)(cvh / p.split) * p.slab;
            k_src = p.k + at + chunk * 16;
            v_src = p.v + at + chunk * 16;
            sc_src = (lane < 2 * NG ? p.k : p.v) + at + B * (D / 2) + (lane % NG) * 16;
            if (p.log2b != 3 && lane & NG) sc_src += 8 * (NG * 2);   // the rows 8..15 of a unit
            cu += stretch;
            request();
        };
        auto copy = [&](const uint8_t *k0, const uint8_t *v0, const uint8_t *k1, const uint8_t *v1, const uint8_t *sc) {
            if constexpr (D == 128) {   // chunks 0..31: rows 0..7, 32..63: rows 8..15
                cp_async16(wr + lane * 16, k0);
                cp_async16(wr + lane * 16 + 512, k1);
                cp_async16(wr + S::kCodes + v_sw * 16, v0);
                cp_async16(wr + S::kCodes + 512 + (v_sw ^ 4) * 16, v1);
            } else {
                cp_async16(wr + k_sw * 16, lane < 16 ? k0 : k1);
                cp_async16(wr + S::kCodes + v_sw * 16, lane < 16 ? v0 : v1);
            }
            if (lane < 4 * NG) cp_async16(wr + 2 * S::kCodes + lane * 16, sc);
        };
        auto issue = [&]() {
            if (stretch > 0) {
                // tokens 0..7 and 8..15 of the unit: neighbouring rows of one block, or two blocks of 8
                constexpr int kHalf = 8 * (D / 2);
                const uint32_t id = __shfl_sync(0xffffffffu, ids, id_at);
                const uint64_t at = (uint64_t)id * p.block_bytes;
                if (p.log2b == 4) {
                    ++id_at;
                    copy(k_src + at, v_src + at, k_src + at + kHalf, v_src + at + kHalf, sc_src + at);
                } else if (p.log2b == 3) {
                    const uint64_t at1 = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, ids, id_at + 1) * p.block_bytes;
                    id_at += 2;
                    copy(k_src + at, v_src + at, k_src + at1, v_src + at1, sc_src + (lane & NG ? at1 : at));
                } else {
                    const uint64_t rows = at + half * (2 * kHalf);
                    copy(k_src + rows, v_src + rows, k_src + rows + kHalf, v_src + rows + kHalf,
                         sc_src + at + half * (kU * NG * 2));
                    id_at += half;
                    half ^= 1;
                }
                wr = wr + S::kStage == ring_a + S::kRing ? ring_a : wr + S::kStage;
                if (--stretch == 0) next_stretch();
            }
            cp_async_commit();
        };
        request();
        // a head's queries as they lie in memory; requested while the head before it is finished (one tile of bf16
        // queries: the larger forms have no registers for that)
        constexpr bool kEarly = NT == 1 && !S::kF32;
        Raw8<T> q_raw[NT][NG];
        auto request_q = [&](int seq, int head) {
            const int part = head % p.split, h0 = (head / p.split) * p.group + part * p.hw;
            const int heads = min(p.hw, p.group - part * p.hw);
            const T *qrow = static_cast<const T *>(p.q) + ((int64_t)seq * p.num_heads + h0) * D;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int h = 8 * nt + r;
                    const T *src = qrow + (int64_t)h * D + 32 * g + 8 * c;
                    q_raw[nt][g] = {};
                    if (h < heads) {
                        if (p.vec) {
                            q_raw[nt][g] = load_raw8(src);
                        } else {
#pragma unroll
                            for (int d = 0; d < 8; ++d) reinterpret_cast<T *>(&q_raw[nt][g])[d] = src[d];
                        }
                    }
                }
        };
        if (kEarly && left > 0) request_q(s, vh);
        next_stretch();

        // q as B operands of the first product, pair i the dims (i, i + 4) of the lane's 8 (bf16 calls: in fp16, odd
        // pairs divided by the 16 that their codes carry); q8: three bf16 parts of -8 sum(q) of the groups
        uint32_t qf[NT][NS][NG][4], q8[NT][2];
        float o[NT][2 * NG][4], m[NT][2], l[NT][2], sl[NT][2];   // sl: what brings the lane's columns to base-2 logits
        uint32_t far[NT];                                         // q-heads that leave 2^24 of it to the logits
        uint32_t up[NG / 2];                                      // the groups' powers of two for V's scales, bf16 pairs
        uint32_t cap[NG / 2];                                     // the largest scales that `up` takes to less than 2^8
        // What the compiler makes of the registers differs by form: with the units of a step taken downwards and the
        // caps made from `up` each time, 16 x 32768 tokens (D = 128, groups up to 8) take 117.4 us, upwards with caps
        // kept 122.0; for groups of 16 and 32 64 x 18750 tokens take 127 us that way and 121 this, fp32 147 and 141.
        constexpr bool kDown = !S::kF32 && NT == 1 && D == 128, kKeepCaps = NT == 2;
        bool fresh = true, at_start = true;
        int u_first = 0;
        const uint8_t *st = ring;
        // row m of the first product is token t(m): its rows (2c, 2c+1) and (2c+8, 2c+9) are the tokens
        // 4c .. 4c+3 that the lane holds of V; its own rows r and r + 8 are the tokens t0 and t0 + 2
        const int t0 = 4 * (r >> 1) + (r & 1), t1 = t0 + 2;
        const int k_at = D == 128 ? (t0 * 4 + c) * 16 : ((t0 * 2 + (c >> 1)) ^ (4 * ((t0 >> 2) & 1))) * 16 + (c & 1) * 8;
        // rows 4c and 4c + 1 of V; 4c + 2 and 4c + 3 lie two rows on
        const int v_at0 = D == 128 ? ((16 * c + (r >> 1)) ^ (2 * c)) * 16 + (r & 1) * 8 : ((8 * c + (r >> 2)) ^ (2 * c)) * 16 + (r & 3) * 4;
        const int v_at1 = D == 128 ? ((16 * c + 4 + (r >> 1)) ^ (2 * c)) * 16 + (r & 1) * 8 : ((8 * c + 2 + (r >> 2)) ^ (2 * c)) * 16 + (r & 3) * 4;
        // a tile's bytes two rows on (head_dim 64: the swizzle turns the step round)
        const int two_rows_k = D == 128 || !((t0 >> 2) & 1) ? D : -D, two_rows_v = D == 128 || c < 2 ? D : -D;
        // One or two units of the current head.
        auto step = [&](auto units) {
            constexpr int NU = decltype(units)::value;
            // the oldest units' copies are in (kStages are on their way at all times), for every lane
            cp_async_wait<kStages - NU>();
            __syncwarp();
            const uint8_t *at[NU];
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                at[j] = st;
                st = st + S::kStage == ring + S::kRing ? ring : st + S::kStage;
            }
            const int valid = ctx - u * kU - (NU - 1) * kU;   // tokens of the last unit that exist
            constexpr int L = NU - 1;

            // ---- S = K Q^T
            float x[NU][NT][4];
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int j = kDown ? NU - 1 - i : i;
                uint32_t k0[NG], k1[NG], z0[NG / 2], z1[NG / 2];
                if constexpr (D == 128) {
                    *reinterpret_cast<uint4 *>(k0) = *reinterpret_cast<const uint4 *>(at[j] + k_at);
                    *reinterpret_cast<uint4 *>(k1) = *reinterpret_cast<const uint4 *>(at[j] + k_at + 128);
                } else {
                    *reinterpret_cast<uint2 *>(k0) = *reinterpret_cast<const uint2 *>(at[j] + k_at);
                    *reinterpret_cast<uint2 *>(k1) = *reinterpret_cast<const uint2 *>(at[j] + k_at + two_rows_k);
                }
                load_scales<NG>(z0, at[j] + 2 * S::kCodes + t0 * (NG * 2));
                load_scales<NG>(z1, at[j] + 2 * S::kCodes + t0 * (NG * 2) + NG * 4);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    x[j][nt][0] = x[j][nt][1] = x[j][nt][2] = x[j][nt][3] = 0.0f;
                    if (!S::kF32) {   // K index i of this product: the scale of group i % NG
                        const uint32_t a0 = NG == 4 && c & 1 ? z0[NG / 2 - 1] : z0[0];
                        const uint32_t a1 = NG == 4 && c & 1 ? z1[NG / 2 - 1] : z1[0];
                        mma_bf16_16816(x[j][nt], a0, a1, a0, a1, q8[nt][0], q8[nt][1]);
                    }
                }
#pragma unroll
                for (int g = NG - 1; g >= 0; --g) {   // (upwards the compiled order is 1 % slower)
                    const float s0 = scale_of(z0, g), s1 = scale_of(z1, g);
                    uint32_t a[4][2];
                    if constexpr (S::kF32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e][0] = minus_136(nibbles_128(k0[g] >> (4 * e)));
                            a[e][1] = minus_136(nibbles_128(k1[g] >> (4 * e)));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e][0] = nibbles_f16(k0[g], e);
                            a[e][1] = nibbles_f16(k1[g], e);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float acc[4];
                        if constexpr (S::kF32) {
                            acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
#pragma unroll
                            for (int k = 0; k < NS; ++k) {
                                mma_bf16_16816(acc, a[0][0], a[0][1], a[1][0], a[1][1], qf[nt][k][g][0], qf[nt][k][g][1]);
                                mma_bf16_16816(acc, a[2][0], a[2][1], a[3][0], a[3][1], qf[nt][k][g][2], qf[nt][k][g][3]);
                            }
                        } else {
                            mma_f16_16816_first(acc, a[0][0], a[0][1], a[1][0], a[1][1], qf[nt][0][g][0], qf[nt][0][g][1]);
                            mma_f16_16816(acc, a[2][0], a[2][1], a[3][0], a[3][1], qf[nt][0][g][2], qf[nt][0][g][3]);
                        }
                        x[j][nt][0] = fmaf(s0, acc[0], x[j][nt][0]);
                        x[j][nt][1] = fmaf(s0, acc[1], x[j][nt][1]);
                        x[j][nt][2] = fmaf(s1, acc[2], x[j][nt][2]);
                        x[j][nt][3] = fmaf(s1, acc[3], x[j][nt][3]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (far[nt]) {   // (the same for the warp)
#pragma unroll
                    for (int j = 0; j < NU; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (far[nt] >> (8 * c + 4 * (e & 1)) & 1) x[j][nt][e] *= 0x1p24f;
                }
            // ---- softmax weights (base 2).  Rows behind the sequence may hold anything, NaN scales too: they are
            // selected away, not multiplied
            uint32_t vz0[NU][NG / 2], vz1[NU][NG / 2];   // V's scales
            auto load_v_scales = [&]() {
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    load_scales<NG>(vz0[j], at[j] + 2 * S::kCodes + S::kScales + t0 * (NG * 2));
                    load_scales<NG>(vz1[j], at[j] + 2 * S::kCodes + S::kScales + t0 * (NG * 2) + NG * 4);
                }
            };
            load_v_scales();
            if (valid < kU) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((e < 2 ? t0 : t1) >= valid) x[L][nt][e] = -INFINITY * sl[nt][e & 1];   // times sl: -inf
#pragma unroll
                for (int g = 0; g < NG / 2; ++g) {
                    if (t0 >= valid) vz0[L][g] = 0;
                    if (t1 >= valid) vz1[L][g] = 0;
                }
            }
            float w[NU][NT][4];
            bool move = false;
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[j][nt][e] = fmaf(x[j][nt][e], sl[nt][e & 1], -m[nt][e & 1]);
                        move |= w[j][nt][e] > kMoveAt;
                    }
            if (!S::kF32) {
#pragma unroll
                for (int g = 0; g < NG / 2; ++g) {
                    uint32_t top = 0;   // (a NaN scale is no size)
#pragma unroll
                    for (int j = 0; j < NU; ++j) top = max_bf16x2(top, max_bf16x2(vz0[j][g], vz1[j][g]));
                    const uint32_t most = kKeepCaps ? cap[g] : cap_of(up[g]);
                    move |= !__hble2(*reinterpret_cast<const __nv_bfloat162 *>(&top),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&most));
                }
            }
            if (__any_sync(0xffffffffu, move)) {
                float beta[NG];   // what the sums of a group are brought down by
                if (!S::kF32) {
#pragma unroll
                    for (int g = 0; g < NG / 2; ++g) {
                        uint32_t t = 0;
#pragma unroll
                        for (int j = 0; j < NU; ++j) t = max_bf16x2(t, max_bf16x2(vz0[j][g], vz1[j][g]));
                        t = max_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, 4));
                        t = max_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, 8));
                        t = max_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, 16));
                        // exponent fields: of a largest scale e, the power 260 - e takes it to 133 (2^6)
                        const int old0 = up[g] >> 7 & 0xff, old1 = up[g] >> 23;
                        const int new0 = min(old0, 260 - (int)(t >> 7 & 0xff)), new1 = min(old1, 260 - (int)(t >> 23 & 0xff));
                        beta[2 * g] = __uint_as_float((uint32_t)max(1, 127 + new0 - old0) << 23);
                        beta[2 * g + 1] = __uint_as_float((uint32_t)max(1, 127 + new1 - old1) << 23);
                        up[g] = (uint32_t)new0 << 7 | (uint32_t)new1 << 23;
                        cap[g] = cap_of(up[g]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = m[nt][e];
#pragma unroll
                        for (int j = 0; j < NU; ++j)
                            y = fmaxf(y, fmaxf(x[j][nt][e] * sl[nt][e], x[j][nt][e + 2] * sl[nt][e]));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                        const float alpha = y == m[nt][e] ? 1.0f : fast_exp2(m[nt][e] - y);
                        m[nt][e] = y;
                        l[nt][e] *= alpha;
#pragma unroll
                        for (int t = 0; t < 2 * NG; ++t) {
                            const float f = S::kF32 ? alpha : alpha * beta[t / 2];
                            o[nt][t][e] *= f;
                            o[nt][t][e + 2] *= f;
                        }
#pragma unroll
                        for (int j = 0; j < NU; ++j) {
                            // (products rounded as y was: a fused one leaves y's rounding, past 2^30 or so a large number)
                            w[j][nt][e] = __fsub_rn(__fmul_rn(x[j][nt][e], sl[nt][e]), y);
                            w[j][nt][e + 2] = __fsub_rn(__fmul_rn(x[j][nt][e + 2], sl[nt][e]), y);
                        }
                    }
                }
            }
            if (!S::kF32) {   // exact: powers of two
#pragma unroll
                for (int j = 0; j < NU; ++j)
#pragma unroll
                    for (int g = 0; g < NG / 2; ++g) {
                        vz0[j][g] = mul_bf16x2(vz0[j][g], up[g]);
                        vz1[j][g] = mul_bf16x2(vz1[j][g], up[g]);
                    }
            }
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[j][nt][e] = fast_exp2(w[j][nt][e]);
                        l[nt][e & 1] += x[j][nt][e];
                    }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int j = kDown ? NU - 1 - i : i;
                const uint8_t *vc = at[j] + S::kCodes;
                constexpr int NW = NG / 2;       // words of a lane's share of a V row
                uint32_t vw[4][NW];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint8_t *row = vc + (t & 1 ? v_at1 : v_at0) + (t < 2 ? 0 : two_rows_v);
                    if constexpr (D == 128) *reinterpret_cast<uint2 *>(vw[t]) = *reinterpret_cast<const uint2 *>(row);
                    else vw[t][0] = *reinterpret_cast<const uint32_t *>(row);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s0 = scale_of(vz0[j], g), s1 = scale_of(vz1[j], g);
                    const uint32_t v01 = __byte_perm(vw[0][g / 2], vw[1][g / 2], g & 1 ? 0x7632 : 0x5410);
                    const uint32_t v23 = __byte_perm(vw[2][g / 2], vw[3][g / 2], g & 1 ? 0x7632 : 0x5410);
                    uint32_t a[4][2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[e][0] = S::kF32 ? minus_136(nibbles_128(v01 >> (4 * e))) : nibbles_f16(v01, e);
                        a[e][1] = S::kF32 ? minus_136(nibbles_128(v23 >> (4 * e))) : nibbles_f16(v23, e);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // the only rounding of a weight: p times V's scale, to fp16 (fp32 calls: three bf16 parts)
                        float y[4] = {x[j][nt][0] * s0, x[j][nt][1] * s0, x[j][nt][2] * s1, x[j][nt][3] * s1};
                        if constexpr (S::kF32) {
                            // summed apart and added with rounding: the matrix sum cuts, and over a long sequence
                            // its cuts would all point one way
                            float u0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int k = 0; k < NS; ++k) {
                                const float y0 = bf16_part(y[0]), y1 = bf16_part(y[1]);
                                const float y2 = bf16_part(y[2]), y3 = bf16_part(y[3]);
                                const uint32_t b0 = movmatrix_trans(pack_bf16x2(y0, y1));
                                const uint32_t b1 = movmatrix_trans(pack_bf16x2(y2, y3));
                                mma_bf16_16816(u0, a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
                                mma_bf16_16816(u1, a[2][0], a[3][0], a[2][1], a[3][1], b0, b1);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[nt][2 * g][e] += u0[e];
                                o[nt][2 * g + 1][e] += u1[e];
                            }
                        } else {
                            const uint32_t b0 = movmatrix_trans(pack_f16x2(y[0], y[1]));
                            const uint32_t b1 = movmatrix_trans(pack_f16x2(y[2], y[3]));
                            constexpr uint32_t e8 = 0x80088008u, f8 = 0x80808080u;   // -8 2^-24 and -8 2^-20, twice
                            mma_f16_16816(o[nt][2 * g], a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
                            mma_f16_16816(o[nt][2 * g + 1], a[2][0], a[3][0], a[2][1], a[3][1], b0, b1);
                            mma_f16_16816(o[nt][2 * g], e8, f8, e8, f8, b0, b1);
                            mma_f16_16816(o[nt][2 * g + 1], e8, f8, e8, f8, b0, b1);
                        }
                    }
                }
            }
            __syncwarp();   // every lane is done with the units' places
        };
        int due = kStages;   // copies to set off: the units' places are free
        while (left > 0) {
#pragma unroll 1
            for (; due > 0; --due) issue();
            if (fresh) {
                fresh = false;
                u_first = u;
                if (!kEarly) request_q(s, vh);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[NG][8];
#pragma unroll
                    for (int g = 0; g < NG; ++g) to_floats(x[g], q_raw[nt][g]);
                    float most = 0.0f;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int d = 0; d < 8; ++d) most = fmaxf(most, fabsf(x[g][d]));
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    // Exponent fields: of the factor that brings `most` into [2^14, 2^15) (fp32 calls: [2^-9, 2^-8), where a
                    // group's sum over its codes stays below 1), and of its inverse, times the 2^24 that the codes of bf16
                    // calls carry.  An inverse with the scale past the largest fp32 leaves 2^24 of itself to the logits
                    // (`far`: the q-heads that do, four bits each).
                    const int e = (int)(__float_as_uint(most) >> 23);
                    const int lift_q = S::kF32 ? max(1, 245 - e) : min(254, 268 - e);
                    const int inverse = (S::kF32 ? 254 : 278) - lift_q;
                    float up_q = __uint_as_float((uint32_t)lift_q << 23);
                    float back = __uint_as_float((uint32_t)min(254, inverse) << 23) * p.scale_log2;
                    const bool too_far = inverse > 254 || fabsf(back) > 0x1.fffffep127f;
                    if (too_far) back = __uint_as_float((uint32_t)(inverse - 24) << 23) * p.scale_log2;
                    far[nt] = __ballot_sync(0xffffffffu, too_far);
                    sl[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
                    sl[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
                    if constexpr (S::kF32) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
#pragma unroll
                            for (int d = 0; d < 8; ++d) x[g][d] *= up_q;
#pragma unroll
                            for (int k = 0; k < NS; ++k)
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    qf[nt][k][g][d] = pack_bf16x2(bf16_part(x[g][d]), bf16_part(x[g][d + 4]));
                        }
                    } else {
                        float any = 0.0f;   // NaN if an element is NaN or infinite
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int d = 0; d < 8; ++d) any = fmaf(x[g][d], 0.0f, any);
                        any += __shfl_xor_sync(0xffffffffu, any, 1);
                        any += __shfl_xor_sync(0xffffffffu, any, 2);
                        up_q += any;
                        float sums[NG];
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            float sum = 0.0f;
#pragma unroll
                            for (int d = 0; d < 8; ++d) {
                                x[g][d] *= up_q;
                                sum += x[g][d];
                            }
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                qf[nt][0][g][d] = d & 1 ? pack_f16x2(x[g][d] * 0.0625f, x[g][d + 4] * 0.0625f)
                                                        : pack_f16x2(x[g][d], x[g][d + 4]);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                            sums[g] = sum * (-8.0f * 0x1p-24f);
                        }
                        // K index i of the product with the scales: part i / NG, group i % NG
                        q8[nt][0] = q8[nt][1] = 0;
#pragma unroll
                        for (int k = 0; k < 3; ++k)
#pragma unroll
                            for (int g = 0; g < NG; g += 2) {
                                const uint32_t y = pack_bf16x2(bf16_part(sums[g]), bf16_part(sums[g + 1]));
                                const int at = (k * NG + g) / 2;   // word of K: lane c = at % 4, register at / 4
                                if (c == at % 4) q8[nt][at / 4] = y;
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)   // never 0: masked logits are -inf * sl * sl
                        if (sl[nt][e] == 0.0f) sl[nt][e] = 0x1p-126f;
#pragma unroll
                    for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.0f;
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.0f;
                }
#pragma unroll
                for (int g = 0; g < NG / 2; ++g) {
                    up[g] = 0x7e807e80u;   // 2^126: scales from 2^-118 up bring it down
                    cap[g] = cap_of(up[g]);
                }
            }
            const int pair = left > 1 && u + 1 < nu ? 2 : 1;
            if (pair == 2) step(std::integral_constant<int, 2>());
            else step(std::integral_constant<int, 1>());
            due = pair;
            u += pair;
            left -= pair;
            if (left > 0 && u < nu) continue;

            // ---- the end of a (sequence, head) or of the warp's part
            const int part = vh % p.split, h0 = (vh / p.split) * p.group + part * p.hw;
            const int heads = min(p.hw, p.group - part * p.hw);
            const int s_done = s, vh_done = vh, nu_done = nu;
            left -= kHeadCost;
            if (++vh == VH && left > 0) {
                vh = 0;
                do {
                    ctx = uniform(ctxs[++s]);
                    nu = units_of(ctx, max_tokens);
                } while (nu == 0);
            }
            if (kEarly && left > 0) request_q(s, vh);
            // rows r of a tile carry 2^-24 (bf16 calls), rows r + 8 2^-20; the dims of a group its scales' power of two
            float down[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
                down[g] = S::kF32 ? 1.0f : __uint_as_float((254 - (up[g / 2] >> (g & 1 ? 23 : 7) & 0xff)) << 23);
            constexpr float kUp0 = S::kF32 ? 1.0f : 0x1p24f, kUp1 = S::kF32 ? 1.0f : 0x1p20f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < 2 * NG; ++t) {
                    o[nt][t][0] *= kUp0;
                    o[nt][t][1] *= kUp0;
                    o[nt][t][2] *= kUp1;
                    o[nt][t][3] *= kUp1;
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
                }
            if (u_first == 0 && u == nu_done) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = 8 * nt + 2 * c + e;
                        if (h >= heads) continue;
                        T *dst = static_cast<T *>(p.out) + ((int64_t)s_done * p.num_heads + h0 + h) * D + 4 * r;
                        const float inv = 1.0f / l[nt][e];
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const float y0 = o[nt][2 * g][e] * inv * down[g], y1 = o[nt][2 * g][e + 2] * inv * down[g];
                            const float y2 = o[nt][2 * g + 1][e] * inv * down[g], y3 = o[nt][2 * g + 1][e + 2] * inv * down[g];
                            T *d = dst + 32 * g;
                            if (!p.vec) {
                                d[0] = from_float<T>(y0); d[1] = from_float<T>(y1);
                                d[2] = from_float<T>(y2); d[3] = from_float<T>(y3);
                            } else if constexpr (S::kF32) {
                                *reinterpret_cast<float4 *>(d) = make_float4(y0, y1, y2, y3);
                            } else {
                                *reinterpret_cast<uint2 *>(d) = make_uint2(pack_bf16x2(y0, y1), pack_bf16x2(y2, y3));
                            }
                        }
                    }
            } else {
                // the warp's first piece has a place of its own; a later one is its last and takes the drained ring
                float *piece = first_piece;
                if (!at_start) {
                    cp_async_wait<0>();
                    __syncwarp();
                    piece = reinterpret_cast<float *>(ring);
                }
                if (lane == 0) meta[2 * warp + (at_start ? 0 : 1)] = {s_done, vh_done, u_first, u, nu_done};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = 8 * nt + 2 * c + e;
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            *reinterpret_cast<float4 *>(piece + h * D + 32 * g + 4 * r) =
                                make_float4(o[nt][2 * g][e] * down[g], o[nt][2 * g][e + 2] * down[g],
                                            o[nt][2 * g + 1][e] * down[g], o[nt][2 * g + 1][e + 2] * down[g]);
                        if (r == 0) {
                            piece[HW * D + 2 * h] = m[nt][e];
                            piece[HW * D + 2 * h + 1] = l[nt][e];
                        }
                    }
            }
            fresh = true;
            at_start = false;
            u = 0;
        }
        cp_async_wait<0>();
    }
    __syncthreads();

    // ---- merge the CTA's pieces: pieces of one (sequence, head) are neighbours in stream order
    constexpr int PER = D / 32;   // dims a lane
    auto piece_of = [&](int j) -> const float * {
        return j & 1 ? reinterpret_cast<const float *>(smem + (j >> 1) * S::kRing)
                     : reinterpret_cast<const float *>(smem + kWarps * S::kRing) + (j >> 1) * S::kPiece;
    };
    // lane j of every warp looks at piece j; a run is the pieces of one head, and (run, q-head) pairs go round the warps
    PieceMeta mine = {-1, 0, 0, 0, 0};
    if (lane < 2 * kWarps) mine = meta[lane];
    const bool valid = mine.seq >= 0;
    const uint32_t some = __ballot_sync(0xffffffffu, valid), below = some & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : lane;
    const int prev_seq = __shfl_sync(0xffffffffu, mine.seq, prev), prev_vh = __shfl_sync(0xffffffffu, mine.vh, prev);
    const uint32_t starts = __ballot_sync(0xffffffffu, valid && (!below || prev_seq != mine.seq || prev_vh != mine.vh));
    const int runs = __popc(starts), run = __popc(starts & (0xffffffffu >> (31 - lane))) - 1;
    for (int task = warp; task < runs * p.hw; task += kWarps) {
        const int i = task / p.hw, h = task - i * p.hw;
        const uint32_t in = __ballot_sync(0xffffffffu, valid && run == i);
        const int j0 = __ffs(in) - 1, j1 = 31 - __clz(in);
        const int seq = __shfl_sync(0xffffffffu, mine.seq, j0), vh = __shfl_sync(0xffffffffu, mine.vh, j0);
        const int u0 = __shfl_sync(0xffffffffu, mine.u0, j0), nu = __shfl_sync(0xffffffffu, mine.nu, j0);
        const int u1 = __shfl_sync(0xffffffffu, mine.u1, j1);
        const int part = vh % p.split, h0 = (vh / p.split) * p.group + part * p.hw;
        if (h >= min(p.hw, p.group - part * p.hw)) continue;
        const bool member = in >> lane & 1;
        const float *ml = piece_of(lane < 2 * kWarps ? lane : 0) + HW * D + 2 * h;
        const float m = member ? ml[0] : -INFINITY;
        float M = m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float f = member ? fast_exp2(m - M) : 0.0f;
        float L = member ? f * ml[1] : 0.0f, acc[PER];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll
        for (int d = 0; d < PER; ++d) acc[d] = 0.0f;
        for (int j = j0; j <= j1; ++j) {
            if (!(in >> j & 1)) continue;
            const float fj = __shfl_sync(0xffffffffu, f, j);
            const float *pc = piece_of(j) + h * D + lane;
#pragma unroll
            for (int d = 0; d < PER; ++d) acc[d] += fj * pc[d * 32];
        }
        if (u0 == 0 && u1 == nu) {
            T *dst = static_cast<T *>(p.out) + ((int64_t)seq * p.num_heads + h0 + h) * D + lane;
            const float inv = 1.0f / L;
#pragma unroll
            for (int d = 0; d < PER; ++d) dst[d * 32] = from_float<T>(acc[d] * inv);
        } else {   // a head that other CTAs share: cut on its left, or on its right only
            float *dst = p.part + ((int64_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * S::kPiece;
#pragma unroll
            for (int d = 0; d < PER; ++d) dst[h * D + d * 32 + lane] = acc[d];
            if (lane == 0) {
                dst[HW * D + 2 * h] = M;
                dst[HW * D + 2 * h + 1] = L;
            }
        }
    }
    // a head cut on the right only is the last run's; its first unit lies u1 before the end of the CTA's share
    if (warp == 0 && some) {
        const int j0 = 31 - __clz(starts), j1 = 31 - __clz(some);
        const int seq = __shfl_sync(0xffffffffu, mine.seq, j0), vh = __shfl_sync(0xffffffffu, mine.vh, j0);
        const int u0 = __shfl_sync(0xffffffffu, mine.u0, j0), nu = __shfl_sync(0xffffffffu, mine.nu, j0);
        const int u1 = __shfl_sync(0xffffffffu, mine.u1, j1);
        if (lane == 0 && u0 == 0 && u1 < nu) {
            const int64_t end = share_s[1] - u1 + nu - 1, share = share_s[2];
            p.cuts[blockIdx.x] = {seq, vh, (int)(share >> 31 ? end / share : quotient(end, (int)share)), 0};
        }
    }
}

// Heads cut between CTAs: CTA (c, h) merges the pieces of q-head h of the one cut at the end of the decode kernel's
// CTA c.  Warp w adds pieces w, w + 4, ... and the four sums are added in order, so the order is fixed.
constexpr int kMergeWarps = 4;
template <typename T, int D, int HW>
__global__ void __launch_bounds__(kMergeWarps * 32) q4_merge_kernel(const Q4Params p) {
    constexpr int PER = D / 32, kPiece = HW * (D + 2);
    __shared__ float sum_s[kMergeWarps][D + 1];
    const int c0 = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    const Cut a = p.cuts[c0];
    if (a.seq < 0) return;
    const int part = a.vh % p.split, h0 = (a.vh / p.split) * p.group + part * p.hw;
    if (h >= min(p.hw, p.group - part * p.hw)) return;
    // the first CTA's piece is the one cut on its right
    auto src = [&](int cta) { return p.part + ((int64_t)cta * 2 + (cta == c0 ? 1 : 0)) * kPiece; };
    float M = -INFINITY, L = 0.0f, acc[PER];
#pragma unroll
    for (int d = 0; d < PER; ++d) acc[d] = 0.0f;
    for (int cta = c0 + lane; cta <= a.last; cta += 32) M = fmaxf(M, src(cta)[HW * D + 2 * h]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int base = c0 + warp; base <= a.last; base += 32 * kMergeWarps) {   // lane i: the warp's i-th piece from here
        const int cta = base + lane * kMergeWarps, n = min(32, (a.last - base) / kMergeWarps + 1);
        float f = 0.0f;
        if (lane < n) {
            f = fast_exp2(src(cta)[HW * D + 2 * h] - M);
            L += f * src(cta)[HW * D + 2 * h + 1];
        }
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            const float *pc = src(base + i * kMergeWarps) + h * D + lane;
#pragma unroll
            for (int d = 0; d < PER; ++d) acc[d] += fi * pc[d * 32];
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll
    for (int d = 0; d < PER; ++d) sum_s[warp][d * 32 + lane] = acc[d];
    if (lane == 0) sum_s[warp][D] = L;
    __syncthreads();
    T *dst = static_cast<T *>(p.out) + ((int64_t)a.seq * p.num_heads + h0 + h) * D;
    for (int d = threadIdx.x; d < D; d += kMergeWarps * 32) {
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            o += sum_s[w][d];
            l += sum_s[w][D];
        }
        dst[d] = from_float<T>(o * (1.0f / l));
    }
}

// q-heads a warp takes: 16 for groups above 8 (K and V codes are then turned into operands once for both
// tiles of 8), 8 otherwise and for fp32 calls, whose split operands leave no registers for a second tile.
bool two_tiles(int group, bool f32) { return group > 8 && !f32; }

int64_t prefix_bytes(int num_seqs) { return ((int64_t)(num_seqs + 1) * 8 + 255) / 256 * 256; }

template <typename T, int D, int NT>
cudaError_t launch_typed(Q4Params p, const AttnArgs &a, cudaStream_t stream) {
    using S = Q4Shape<T, D, NT>;
    auto kern = q4_decode_kernel<T, D, NT>;
    // the kernel's shared-memory size is an attribute of each device's context: set at the first call there, and
    // again should a launch fail (a context made anew has forgotten it)
    static std::atomic<uint64_t> known{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    auto set = [&] {
        const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemMost);
        if (r == cudaSuccess) known.fetch_or(bit);
        return r;
    };
    const bool had = (known.load() & bit) != 0;
    if (!had && (e = set()) != cudaSuccess) return e;
    p.split = (p.group + S::HW - 1) / S::HW;
    p.hw = (p.group + p.split - 1) / p.split;
    const int sms = min(kMaxCtas, device_sm_count()), max_tokens = a.max_blocks * a.block_size;
    const int64_t heads = (int64_t)a.num_seqs * a.num_kv_heads * p.split;
    p.scan = a.num_seqs <= kScanSeqs;
    // One CTA a head: one launch, and nothing is cut between CTAs.  The split over all SMs costs its second kernel,
    // some 3 us, and gains the more the fewer heads there are: 8 heads of 512 tokens take 8.0 us this way and 9.5
    // split, of 1024 10.2 and 10.1, of 2048 14.1 and 11.2; 128 heads of 2048 tokens 14.7 and 16.5, of 4096 22.5 and
    // 23.1.
    p.by_head = heads <= sms && max_tokens <= kU * (64 + 128 * heads / sms);
    // Many heads over short tables: shares that end between heads are uneven by a head at most, and nothing is left
    // to merge (64 x 128-384 tokens of 32 heads 25.7 -> 23.9 us, 50 x 1-500 of 8 heads 13.3 -> 11.7; with tables of
    // 64 units 100 x 300-1000 of 8 heads 24.8 -> 25.1, with 256 the power-law batch 40.6 -> 49.2).
    p.whole = !p.by_head && heads >= 2 * sms && max_tokens <= 32 * kU;
    const int grid = p.by_head ? (int)heads : sms;
    const size_t smem = S::kSmem + (p.scan ? (size_t)(a.num_seqs + 2) * 12 : 0);
    if (!p.scan) {
        e = launch_dependent(q4_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a.context_lens, a.num_seqs,
                             max_tokens, p.prefix, a.status);
        if (e != cudaSuccess) return e;
    }
    e = launch_dependent(kern, dim3(grid), dim3(S::kWarps * 32), smem, stream, p);
    if (e == cudaErrorInvalidValue && had) {
        cudaGetLastError();
        if ((e = set()) == cudaSuccess) e = launch_dependent(kern, dim3(grid), dim3(S::kWarps * 32), smem, stream, p);
    }
    if (e != cudaSuccess || p.by_head || p.whole) return e;
    return launch_dependent(q4_merge_kernel<T, D, S::HW>, dim3(grid, p.hw), dim3(kMergeWarps * 32), 0, stream, p);
}

}  // namespace

size_t decode_q4_workspace(int num_seqs, int num_heads, int num_kv_heads, int head_dim) {
    const int hw = two_tiles(num_heads / num_kv_heads, false) ? 16 : 8;
    const size_t part = (size_t)kMaxCtas * 2 * hw * (head_dim + 2) * sizeof(float);
    return prefix_bytes(num_seqs) + kMaxCtas * sizeof(Cut) + (part + 255) / 256 * 256;
}

cudaError_t launch_decode_q4(const AttnArgs &a, void *workspace, size_t, cudaStream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Q4Params p = {};
    p.q = a.q;
    p.out = a.out;
    p.k = static_cast<const uint8_t *>(a.k_cache);
    p.v = static_cast<const uint8_t *>(a.v_cache);
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.prefix = reinterpret_cast<int64_t *>(ws);
    p.cuts = reinterpret_cast<Cut *>(ws + prefix_bytes(a.num_seqs));
    p.part = reinterpret_cast<float *>(ws + prefix_bytes(a.num_seqs) + kMaxCtas * sizeof(Cut));
    p.num_seqs = a.num_seqs;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_heads / a.num_kv_heads;
    p.log2b = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.slab = q4_slab_bytes(a.block_size, a.head_dim);
    p.block_bytes = p.slab * a.num_kv_heads;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    p.vec = (reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.out)) % 16 == 0;
    const bool two = two_tiles(p.group, a.dtype == PA_DTYPE_F32), wide = a.head_dim == 128;
    if (a.dtype == PA_DTYPE_F32)
        return wide ? launch_typed<float, 128, 1>(p, a, stream) : launch_typed<float, 64, 1>(p, a, stream);
    if (two)
        return wide ? launch_typed<__nv_bfloat16, 128, 2>(p, a, stream) : launch_typed<__nv_bfloat16, 64, 2>(p, a, stream);
    return wide ? launch_typed<__nv_bfloat16, 128, 1>(p, a, stream) : launch_typed<__nv_bfloat16, 64, 1>(p, a, stream);
}

}  // namespace pa
