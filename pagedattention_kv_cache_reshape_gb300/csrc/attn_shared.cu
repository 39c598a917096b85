// attn_shared.cu -- decode attention for a batch whose sequences share
// prefixes: what a group of sequences has in common is read and computed once
// for all of them.
//
// For query row (s, h), kv-head g(h), group c of s with C = C_c shared tokens
// (shared_plan.cuh), softmax weights of the two parts of the context add up
// when both are kept as (m, l, o) = (max x, sum 2^{x - m}, sum 2^{x - m} V):
//     M = max m_i,  out = sum 2^{m_i - M} o_i / sum 2^{m_i - M} l_i
// over the pieces i of keys 0 .. C-1 (the group's rows together: a matrix
// product whose K and V come from memory once) and of C .. ctx-1 (the
// sequence's own rows).
//
// shared_plan_kernel   C_c, and the two streams of key tiles
// shared_rows_kernel, shared_few_kernel  CUDA-core products, any dtype (fp32 in and
//                      out of them): each persistent CTA takes equal shares of the
//                      groups' and the sequences' key tiles
// shared_merge_kernel  one warp or four a row: the row's pieces in a fixed order
#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "shared_plan.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanSmemGroups = 4096;   // group starts and smallest contexts kept in shared memory
// Nanoseconds of an SM for a tile of the prefix kernel: head_dim 64, 128; 128 keys of one M-tile, of two, 64 keys of two
// kv-heads; and for an item's begin and end.  The SMs' split follows them, so they were set by sweeps of it.
constexpr int kTcTileNs[2][3] = {{800, 1100, 800}, {1500, 1850, 1450}};
constexpr int kTcItemNs = 3000;
// Two parts to a sequence mean a longer way to its result, about 4 us.  Short prefixes have to save that: 189 sequences in 7
// groups of 16-64 shared tokens 38.0 us shared and 31.9 not, 49 in 10 of 32 27.7 and 23.7 (flushed L2).  Long ones are
// shared however little they save, which pays for groups by themselves from about 256 tokens on (32 / 8 heads x 128, the
// call replayed with and without prefix lengths; 100-300 own tokens): 4 sequences over 256 20.7 and 21.1 us, 8 over 256
// 20.9 and 20.7, 2 over 512 17.4 and 20.5, 8 over 512 20.6 and 23.5, 8 over 1024 21.6 and 25.5.  It does not pay where such a
// group stands among many sequences that share nothing, whose blocks keep HBM busy while shared ones come from L2: 2 over
// 512 and 60 alone 29.3 and 27.0, 8 over 512 and 250 alone 73.4 and 71.2, 128 of 256 over 256 99.0 and 95.0.
constexpr int64_t kLeastSavedNs = 1000;   // of every SM
constexpr int kLongPrefix = 256;
// CUDA cores: head_dim 64, 128; 64 keys of up to 8, 32 and 64 rows; an item's begin and end; and what sharing has to save,
// since a tile of many rows takes its CTA long (9 sequences over 64-1056 tokens, 32 / 1 heads x 64: 40 us shared, 24 not).
constexpr int kCcTileNs[2][3] = {{1000, 3300, 4500}, {2000, 6500, 9000}}, kCcItemNs = 2000;
constexpr int64_t kCcLeastSavedNs = 4000;   // of every SM
constexpr int kMaxCtas = 512;           // partial slots reserved for share boundaries

constexpr size_t kAlign = 32;           // of the pieces' rows (32-byte stores); a caller's workspace lies on 16 bytes

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ------------------------------------------------------------------ plan
// One CTA: the groups' plan, and the own stream's starts (own_start[s]: tiles
// of one kv-head of the sequences before).
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const SharedGroups g, const SharedPlan plan, int32_t *scratch, int64_t *own_start, int32_t *status) {
    __shared__ int32_t starts_s[kPlanSmemGroups], lens_s[kPlanSmemGroups];
    __shared__ int64_t tot[1][kPlanThreads / 32];
    const int tid = threadIdx.x;
    grid_dependency_wait();
    grid_dependents_launch();
    const bool in_smem = g.num_groups <= kPlanSmemGroups;
    int32_t *lens = in_smem ? lens_s : scratch;
    const bool ok = shared_lens<kPlanThreads>(g, in_smem ? starts_s : nullptr, lens, status);
    shared_write_plan<kPlanThreads>(g, plan, ok, in_smem ? starts_s : g.starts, lens);
    int64_t own = 0;
    for (int base = 0; base < g.num_seqs; base += kPlanThreads) {
        const int s = base + tid, len = s < g.num_seqs ? plan.own_len[s] : 0;   // (this thread wrote it)
        int64_t at[1] = {(len + g.keys_per_tile - 1) / g.keys_per_tile}, total[1];
        block_scan<kPlanThreads, 1>(at, tot, total);
        if (s < g.num_seqs) own_start[s] = own + at[0];
        own += total[0];
    }
    if (tid == 0) own_start[g.num_seqs] = own;
}

// ------------------------------------------------------------------ CUDA-core kernel
constexpr int kRows = 64;     // rows of an item at most
constexpr int kKeys = 64;     // keys of a tile
constexpr int kCcThreads = 256;
constexpr int kFewHeads = 8;

struct CcParams {
    const void *q;
    const void *k_cache;
    const void *v_cache;
    const int32_t *block_tables;
    const int32_t *group_starts;
    SharedPlan plan;
    const int64_t *own_start;
    float *pre_o;      // prefix pieces: [rows][D]
    float2 *pre_ml;    // [rows]
    float *own_o;      // own pieces: [num_seqs * num_heads + shares * G][D]
    float2 *own_ml;
    int item_rows;     // seqs_per_item * G
    int seqs_per_item;
    int num_seqs;
    int num_groups;
    int num_heads;
    int num_kv_heads;
    int block_size;
    int log2b;
    int max_blocks;
    int num_blocks;
    int aligned;       // pools and q on 16 bytes
    float scale_log2;
    int32_t *status;
};

// One piece: rows [0, rows) (row r: sequence s0 + r / G, q-head r % G of kv-head kvh) against keys key0 .. key1-1 of
// the block table `table`.
struct CcPiece {
    const int32_t *table;
    int s0, rows, kvh, key0, key1;
    float *o;      // [rows][D]
    float2 *ml;    // [rows]
};

// 16 bytes from global to shared memory in the background; zeros without `read` (src is any valid address then).
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T> struct Vec16 { T v[16 / sizeof(T)]; };

// 16 bytes of a row, as floats; element by element where rows need not be aligned.
template <typename T>
__device__ __forceinline__ void load_floats(const T *p, bool aligned, float (&x)[16 / sizeof(T)]) {
    constexpr int n = 16 / sizeof(T);
    Vec16<T> r;
    if (aligned) *reinterpret_cast<uint4 *>(&r) = __ldg(reinterpret_cast<const uint4 *>(p));
    else {
#pragma unroll
        for (int i = 0; i < n; ++i) r.v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = to_float(r.v[i]);
}

// Shared memory: Q [kRows][D + 4] | K [kKeys][D + 4], whose place the weights [kRows][kKeys + 4] take | V [kKeys][D].
// (Rows of D + 4: the two rows of a warp's half warps, and the keys of its lanes, lie in different banks.)
template <int D> constexpr int cc_smem_floats() { return kRows * (D + 4) + kKeys * (D + 4) + kKeys * D; }

// Bound by what shared memory delivers (L1 76 % and FMA 53 % busy; 4 x 4 logits of a thread take 8 loads of 16 bytes for 64
// products).  fp32, items of 64 rows, 32 / 8 heads x 128, sequences behind 8192 tokens, this kernel alone: 64 of them 213
// us, 256 776, 40 and 44 TFLOP/s; 16 74 us; x 64, 64 of them 126 us, 34 TFLOP/s.  Thread (ty, tx) of 16 x 16 holds logits
// of rows ty * RT + i and keys tx + 16 j, and of the outputs the same rows and dims 4 tx + 64 j + (0..3).  A row's 16
// threads are half a warp.  RT = 1, 2 or 4: 16, 32 or 64 rows.
template <typename T, int D, int RT>
__device__ __forceinline__ void cc_piece(const CcParams &p, const CcPiece &w, float *smem) {
    constexpr int kVec = 16 / sizeof(T), kKS = D + 4, kPS = kKeys + 4, kDJ = D / 64;
    static_assert(kRows * kPS <= kKeys * kKS, "the weights fit the keys' place");
    float *qs = smem, *ks = qs + kRows * kKS, *ps = ks, *vs = ks + kKeys * kKS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ty = tid >> 4, tx = tid & 15;
    const int G = p.num_heads / p.num_kv_heads;
    const bool al = p.aligned != 0;
    for (int e = tid; e < 16 * RT * (D / kVec); e += kCcThreads) {
        const int r = e / (D / kVec), d = (e - r * (D / kVec)) * kVec;
        float x[kVec] = {};
        if (r < w.rows)
            load_floats(static_cast<const T *>(p.q) +
                            ((int64_t)(w.s0 + r / G) * p.num_heads + w.kvh * G + r % G) * D + d, al, x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) qs[r * kKS + d + i] = x[i];
    }
    float m[RT], l[RT];
    float2 o[RT][kDJ][2];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kDJ; ++j) o[i][j][0] = o[i][j][1] = make_float2(0.f, 0.f);
    }
    const int64_t tok_stride = (int64_t)p.num_kv_heads * D;
    for (int key = w.key0; key < w.key1; key += kKeys) {
        // warp w loads keys 8 w .. 8 w + 7, which lie in one block (tiles start at multiples of 8 tokens)
        const int t0 = key + 8 * warp;
        int blk = -1;
        if (t0 < w.key1) {
            blk = __ldg(w.table + t0 / p.block_size);
            if (blk < 0 || blk >= p.num_blocks) {
                if (lane == 0) set_status(p.status, PA_ERR_OUT_OF_RANGE);
                blk = -1;
            }
        }
        const int64_t base = ((int64_t)max(blk, 0) * p.block_size + t0 % p.block_size) * tok_stride + (int64_t)w.kvh * D;
        const int live = blk < 0 ? 0 : min(8, w.key1 - t0);   // rows behind them may hold anything: not read
        if (sizeof(T) == 4 && al) {
            // all of the tile's rows in flight at once, zeros for those that are not read
            const float *kc = static_cast<const float *>(p.k_cache) + base, *vc = static_cast<const float *>(p.v_cache) + base;
#pragma unroll
            for (int e0 = 0; e0 < 8 * (D / 4); e0 += 32) {
                const int e = e0 + lane, r = e / (D / 4), d = (e - r * (D / 4)) * 4;
                const int64_t at = r < live ? r * tok_stride + d : 0;
                cp_async16(ks + (8 * warp + r) * kKS + d, kc + at, r < live);
                cp_async16(vs + (8 * warp + r) * D + d, vc + at, r < live);
            }
            cp_async_wait();
        } else {
#pragma unroll
            for (int e0 = 0; e0 < 8 * (D / kVec); e0 += 32) {
                const int e = e0 + lane, r = e / (D / kVec), d = (e - r * (D / kVec)) * kVec;
                float x[kVec] = {}, y[kVec] = {};
                if (r < live) {
                    load_floats(static_cast<const T *>(p.k_cache) + base + r * tok_stride + d, al, x);
                    load_floats(static_cast<const T *>(p.v_cache) + base + r * tok_stride + d, al, y);
                }
#pragma unroll
                for (int i = 0; i < kVec; i += 4) {
                    *reinterpret_cast<float4 *>(ks + (8 * warp + r) * kKS + d + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    *reinterpret_cast<float4 *>(vs + (8 * warp + r) * D + d + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                }
            }
        }
        __syncthreads();
        float x[RT][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 a[RT], b[4];
#pragma unroll
            for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4 *>(qs + (ty * RT + i) * kKS + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * j) * kKS + d);
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
                    x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
                    x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
                    x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
                }
        }
        // a key is seen if its block was (the warp that loaded it says so) and it lies before key1
        unsigned seen = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int kk = tx + 16 * j, t = key + kk;
            if (t < w.key1) {
                const int b = __ldg(w.table + t / p.block_size);
                if (b >= 0 && b < p.num_blocks) seen |= 1u << j;
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = (seen >> j) & 1 ? x[i][j] * p.scale_log2 : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float mn = fmaxf(m[i], top);
            const float ref = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: weights 0
            const float alpha = fast_exp2(m[i] - ref);
            m[i] = mn;
            l[i] *= alpha;
#pragma unroll
            for (int j = 0; j < kDJ; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) o[i][j][u] = make_float2(o[i][j][u].x * alpha, o[i][j][u].y * alpha);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = fast_exp2(x[i][j] - ref);
                l[i] += x[i][j];
            }
        }
        __syncthreads();   // the keys have been read
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ps[(ty * RT + i) * kPS + tx + 16 * j] = x[i][j];
        __syncwarp();      // a row's weights are written and read by the same half warp
#pragma unroll 4
        for (int kk = 0; kk < kKeys; kk += 4) {
            float4 a[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4 *>(ps + (ty * RT + i) * kPS + kk);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < kDJ; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(vs + (kk + u) * D + 4 * tx + 64 * j);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float c = u == 0 ? a[i].x : u == 1 ? a[i].y : u == 2 ? a[i].z : a[i].w;
                        o[i][j][0] = fma_f32x2(make_float2(c, c), make_float2(b.x, b.y), o[i][j][0]);
                        o[i][j][1] = fma_f32x2(make_float2(c, c), make_float2(b.z, b.w), o[i][j][1]);
                    }
                }
        }
        __syncthreads();   // weights and values have been read
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float sum = l[i];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int r = ty * RT + i;
        if (r >= w.rows) continue;
#pragma unroll
        for (int j = 0; j < kDJ; ++j)
            *reinterpret_cast<float4 *>(w.o + (int64_t)r * D + 4 * tx + 64 * j) =
                make_float4(o[i][j][0].x, o[i][j][0].y, o[i][j][1].x, o[i][j][1].y);
        if (tx == 0) w.ml[r] = make_float2(m[i], sum);
    }
}

// Four neighbouring elements as floats.
template <typename T>
__device__ __forceinline__ float4 load_four(const T *p, bool aligned) {
    if constexpr (sizeof(T) == 4) {
        if (aligned) return __ldg(reinterpret_cast<const float4 *>(p));
    } else {
        if (aligned) {
            const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
            return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                               __uint_as_float(r.y & 0xffff0000u));
        }
    }
    return make_float4(to_float(p[0]), to_float(p[1]), to_float(p[2]), to_float(p[3]));
}

// Up to R = 1, 2, 4 or 8 rows: bound by the cache's bytes, which go straight to registers.  L lanes take a key, each
// the same dims of its K and V rows, of the queries and of the outputs: 4 (i L + lane) + (0..3), so that the L lanes'
// loads are contiguous.  Every group of L lanes is a stream of its own with its running maximum and sums; the streams
// of the CTA are joined at the end of the piece.  A logit's parts are added up so that the lanes share the rows out among
// themselves (R / 2 values exchanged, then R / 4, ...): li / (L / R) is the row whose logit, maximum and sum a lane ends
// up with, and it hands the weight to the others.  A warp takes every eighth chunk of 8 keys (which lie in one block), 32 / L
// keys a step, and requests a step's rows two steps ahead.  A stream moves its maximum only when a logit exceeds it by
// more than 2^8 (its weights stay below that).  60 sequences of 1000-2000 tokens, fp32, 32 / 8 heads x 128, 187 us, 4.1
// TB/s; through shared memory, as the rows kernel has it, 483.
template <typename T, int D, int R>
__device__ __forceinline__ void cc_few(const CcParams &p, const CcPiece &w, float *smem) {
    constexpr int L = (R > 4 ? R : 4) * D / 32, kV = D / 4 / L, kWarps = kCcThreads / 32, kSlots = 32 / L;
    constexpr int kStreams = kWarps * kSlots, kSteps = 8 / kSlots;
    static_assert(kSteps >= 2, "rows are requested two steps ahead");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slot = lane / L, li = lane % L;
    const int G = p.num_heads / p.num_kv_heads, log2b = p.log2b;
    const bool al = p.aligned != 0;
    const int tok_stride = p.num_kv_heads * D;
    const T *kc = static_cast<const T *>(p.k_cache) + (int64_t)w.kvh * D + 4 * li + (int64_t)slot * tok_stride;
    const T *vc = static_cast<const T *>(p.v_cache) + (int64_t)w.kvh * D + 4 * li + (int64_t)slot * tok_stride;
    const int n = w.key1 - w.key0, chunks = (n + 7) >> 3;
    auto block_of = [&](int c) {   // of chunk c; -1: none
        if (c >= chunks) return -1;
        const int blk = __ldg(w.table + ((w.key0 + 8 * c) >> log2b));
        if (blk >= 0 && blk < p.num_blocks) return blk;
        set_status(p.status, PA_ERR_OUT_OF_RANGE);
        return -1;
    };
    float4 k[2][kV], v[2][kV];
    bool seen[2];
    auto request = [&](int b, int c, int blk, int step) {
        seen[b] = blk >= 0 && 8 * c + step * kSlots + slot < n;
        if (!seen[b]) return;
        const int64_t at = (((int64_t)blk << log2b) + ((w.key0 + 8 * c) & ((1 << log2b) - 1)) + step * kSlots) * tok_stride;
#pragma unroll
        for (int u = 0; u < kV; ++u) {
            k[b][u] = load_four(kc + at + 4 * L * u, al);
            v[b][u] = load_four(vc + at + 4 * L * u, al);
        }
    };
    float4 q[R][kV], o[R][kV];
    float m = -INFINITY, l = 0.f;      // of the lane's row
    constexpr int kShare = L / R;
    auto of_row = [&](float x, int r) { return __shfl_sync(0xffffffffu, x, (lane & ~(L - 1)) + r * kShare); };
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int u = 0; u < kV; ++u) {
            o[r][u] = q[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < w.rows)
                q[r][u] = load_four(static_cast<const T *>(p.q) +
                                        ((int64_t)(w.s0 + r / G) * p.num_heads + w.kvh * G + r % G) * D + 4 * (L * u + li), al);
        }
    }
    int blk = block_of(warp), blk1 = block_of(warp + kWarps);
    request(0, warp, blk, 0);
    request(1, warp, blk, 1);
    for (int c = warp; c < chunks; c += kWarps) {
        const int blk2 = block_of(c + 2 * kWarps);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            const int b = step & 1;
            const bool here = seen[b];
            float x[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 y = make_float2(0.f, 0.f);
#pragma unroll
                for (int u = 0; u < kV; ++u) {
                    y = fma_f32x2(make_float2(q[r][u].x, q[r][u].y), make_float2(k[b][u].x, k[b][u].y), y);
                    y = fma_f32x2(make_float2(q[r][u].z, q[r][u].w), make_float2(k[b][u].z, k[b][u].w), y);
                }
                x[r] = y.x + y.y;
            }
#pragma unroll
            for (int h = R / 2, off = L / 2; h > 0; h >>= 1, off >>= 1) {
                const bool upper = (li & off) != 0;
#pragma unroll
                for (int r = 0; r < h; ++r) {
                    const float give = upper ? x[r] : x[r + h], keep = upper ? x[r + h] : x[r];
                    x[r] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            }
#pragma unroll
            for (int off = kShare / 2; off > 0; off >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
            const float y = x[0] * p.scale_log2;
            const bool up = here && y > m + 8.f;
            if (__any_sync(0xffffffffu, up)) {
                const float alpha = up ? fast_exp2(m - y) : 1.f;
                if (up) m = y;
                l *= alpha;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = of_row(alpha, r);
#pragma unroll
                    for (int u = 0; u < kV; ++u)
                        o[r][u] = make_float4(o[r][u].x * f, o[r][u].y * f, o[r][u].z * f, o[r][u].w * f);
                }
            }
            // (a maximum of -inf: the logit is -inf too, weight 0, or NaN)
            const float weight = fast_exp2(y - (m == -INFINITY ? 0.f : m));
            if (here) l += weight;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float e = of_row(weight, r);
                if (here) {
#pragma unroll
                    for (int u = 0; u < kV; ++u) {
                        const float2 f = fma_f32x2(make_float2(e, e), make_float2(v[b][u].x, v[b][u].y), make_float2(o[r][u].x, o[r][u].y));
                        const float2 g = fma_f32x2(make_float2(e, e), make_float2(v[b][u].z, v[b][u].w), make_float2(o[r][u].z, o[r][u].w));
                        o[r][u] = make_float4(f.x, f.y, g.x, g.y);
                    }
                }
            }
            if (step + 2 < kSteps) request(b, c, blk, step + 2);
            else request(b, c + kWarps, blk1, step + 2 - kSteps);
        }
        blk = blk1;
        blk1 = blk2;
    }
    // the streams joined: [stream][R][D] and their (m, l)
    float *os = smem;
    float2 *mls = reinterpret_cast<float2 *>(smem + kStreams * R * D);
    const int stream = warp * kSlots + slot;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int u = 0; u < kV; ++u) *reinterpret_cast<float4 *>(os + (stream * R + r) * D + 4 * (L * u + li)) = o[r][u];
    }
    if (li % kShare == 0) mls[stream * R + li / kShare] = make_float2(m, l);
    __syncthreads();
    for (int e = tid; e < w.rows * (D / 4); e += kCcThreads) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 4
        for (int s = 0; s < kStreams; ++s) top = fmaxf(top, mls[s * R + r].x);
        const float ref = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < kStreams; ++s) {
            const float2 ml = mls[s * R + r];
            if (ml.y == 0.f) continue;   // nothing seen (a NaN stays)
            const float f = fast_exp2(ml.x - ref);
            const float4 y = *reinterpret_cast<const float4 *>(os + (s * R + r) * D + d);
            sum += ml.y * f;
            acc = make_float4(acc.x + y.x * f, acc.y + y.y * f, acc.z + y.z * f, acc.w + y.w * f);
        }
        *reinterpret_cast<float4 *>(w.o + (int64_t)r * D + d) = acc;
        if (d == 0) w.ml[r] = make_float2(top, sum);
    }
    __syncthreads();   // the streams have been read
}

// A CTA's share of the sequences' own parts: by sequence, then kv-head.
template <typename Piece>
__device__ __forceinline__ void own_share(const CcParams &p, int D, Piece piece) {
    const int G = p.num_heads / p.num_kv_heads;
    const int64_t T1 = p.own_start[p.num_seqs] * p.num_kv_heads, P1 = min((int64_t)gridDim.x, T1), c = blockIdx.x;
    const int64_t rows0 = (int64_t)p.num_seqs * p.num_heads;
    int64_t t = c < P1 ? share_begin(c, T1, P1) : 0;   // (no share is empty)
    const int64_t t_end = c < P1 ? share_begin(c + 1, T1, P1) : 0;
    while (t < t_end) {
        const int s = last_at_most_warp(p.own_start, p.num_seqs, t / p.num_kv_heads);
        const int len = p.plan.own_len[s], kt = (len + kKeys - 1) / kKeys;
        const int64_t local = t - p.own_start[s] * p.num_kv_heads;
        const int kvh = (int)(local / kt), tile = (int)(local - (int64_t)kvh * kt);
        const int tiles = (int)min((int64_t)(kt - tile), t_end - t);
        const int C = p.plan.shared_len[p.plan.seq_group[s]];
        const int64_t row = tile == 0 ? (int64_t)s * p.num_heads + kvh * G : rows0 + c * G;
        CcPiece w;
        w.table = p.block_tables + (int64_t)s * p.max_blocks;
        w.s0 = s;
        w.rows = G;
        w.kvh = kvh;
        w.key0 = C + tile * kKeys;
        w.key1 = (int)min((int64_t)C + len, (int64_t)w.key0 + (int64_t)tiles * kKeys);
        w.o = p.own_o + row * D;
        w.ml = p.own_ml + row;
        piece(w);
        t += tiles;
    }
}

// The groups' shared tokens and, with more than kFewHeads q-heads a kv-head, the own parts.  The four forms of a piece under
// the 128 registers of two CTAs an SM spill 76-132 bytes a thread in fp32 (36-160 in bf16).
template <typename T, int D>
__global__ void __launch_bounds__(kCcThreads, 2) shared_rows_kernel(const CcParams p) {
    extern __shared__ __align__(16) float cc_smem[];
    grid_dependency_wait();
    grid_dependents_launch();
    const int G = p.num_heads / p.num_kv_heads;
    const int64_t c = blockIdx.x, T0 = p.plan.tile_start[p.num_groups], P0 = min((int64_t)gridDim.x, T0);
    const int64_t rows0 = (int64_t)p.num_seqs * p.num_heads;
    auto piece = [&](const CcPiece &w) {
        if (w.rows <= 8) cc_few<T, D, 8>(p, w, cc_smem);
        else if (w.rows <= 16) cc_piece<T, D, 1>(p, w, cc_smem);
        else if (w.rows <= 32) cc_piece<T, D, 2>(p, w, cc_smem);
        else cc_piece<T, D, 4>(p, w, cc_smem);
    };
    int64_t t = c < P0 ? share_begin(c, T0, P0) : 0;   // (no share is empty)
    const int64_t t_end = c < P0 ? share_begin(c + 1, T0, P0) : 0;
    while (t < t_end) {
        const PrefixItem it = prefix_item(p.plan, p.group_starts, p.num_groups, p.num_kv_heads, p.seqs_per_item, kKeys, 0, 1, -1, t);
        const int tiles = (int)min((int64_t)(it.of.kt - it.tile), t_end - t), i0 = it.part * p.seqs_per_item;
        const int64_t row = it.tile == 0 ? item_row(it.s0, it.n, it.kvh, i0, p.num_heads, G) : rows0 + c * p.item_rows;
        CcPiece w;
        w.table = p.block_tables + (int64_t)it.s0 * p.max_blocks;
        w.s0 = it.s0 + i0;
        w.rows = min(p.seqs_per_item, it.n - i0) * G;
        w.kvh = it.kvh;
        w.key0 = it.tile * kKeys;
        w.key1 = (int)min((int64_t)it.C, (int64_t)(it.tile + tiles) * kKeys);
        w.o = p.pre_o + row * D;
        w.ml = p.pre_ml + row;
        piece(w);
        t += tiles;
    }
    if (G > kFewHeads) own_share(p, D, piece);
}

// The own parts of at most kFewHeads q-heads a kv-head.  It needs the plan alone, which was complete before the kernel
// in front began, so it takes the SMs that one leaves; at its end it waits for it, so that what follows may rely on
// both.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kCcThreads, 2) shared_few_kernel(const CcParams p) {
    extern __shared__ __align__(16) float cc_smem[];
    grid_dependents_launch();
    own_share(p, D, [&](const CcPiece &w) { cc_few<T, D, R>(p, w, cc_smem); });
    grid_dependency_wait();
}

// ------------------------------------------------------------------ merge
struct MergeParams {
    void *out;
    const int32_t *group_starts;
    SharedPlan plan;
    const int64_t *own_start;   // null: own_o holds the own parts whole, in their first pieces' rows
    const float *pre_o;
    const float2 *pre_ml;
    const float *own_o;
    const float2 *own_ml;
    const int32_t *pre_shares_dev;   // CTAs that cut the prefix stream; null: pre_shares
    int pre_shares;
    int own_shares;     // CTAs that cut the own stream
    int item_rows;
    int seqs_per_item;
    int keys_per_tile;
    int pair_seqs;
    int num_seqs;
    int num_groups;
    int num_heads;
    int num_kv_heads;
    int out_aligned;    // rows of out on 4 bytes
};

constexpr int kMergeThreads = 128;
constexpr int64_t kFewRows = 2100;
constexpr int kRowsPerWarp = 4;

// The running (M, L, acc) of one row; lane: D / 32 consecutive dims.
template <int D> struct RowSum {
    float M = -INFINITY, L = 0.f, acc[D / 32] = {};
    __device__ __forceinline__ void add(float2 ml, const float (&o)[D / 32]) {
        if (ml.y == 0.f) return;   // nothing seen (a NaN stays)
        const float Mn = fmaxf(M, ml.x), a = fast_exp2(M - Mn), b = fast_exp2(ml.x - Mn);
        L = L * a + ml.y * b;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc[u] = acc[u] * a + o[u] * b;
        M = Mn;
    }
};

template <int D>
__device__ __forceinline__ void load_dims(const float *src, float (&v)[D / 32]) {
    if constexpr (D == 128) {
        const float4 t = __ldcg(reinterpret_cast<const float4 *>(src));
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
        v[0] = t.x; v[1] = t.y;
    }
}

// Where one row's pieces of a stream lie: the first in row `first`, the others in rows other, other + step, ...
struct RowPieces {
    int first = 0, other = 0, step = 0, n = 0;   // (rows are counted in 31 bits)
    // tiles [t0, t0 + n) of a stream of T tiles in at most P shares; share c's rows begin at extra + c * rows
    __device__ __forceinline__ RowPieces(int row0, int extra, int rows, int64_t t0, int64_t count, int64_t T, int64_t P) {
        P = min(P, T);
        const int64_t c0 = share_of(t0, T, P), c1 = share_of(t0 + count - 1, T, P);
        first = row0;
        other = extra + ((int)c0 + 1) * rows;
        step = rows;
        n = (int)(c1 - c0 + 1);
    }
    __device__ __forceinline__ RowPieces() {}
    __device__ __forceinline__ RowPieces of_lane(int l) const {
        RowPieces x;
        x.first = __shfl_sync(0xffffffffu, first, l);
        x.other = __shfl_sync(0xffffffffu, other, l);
        x.step = __shfl_sync(0xffffffffu, step, l);
        x.n = __shfl_sync(0xffffffffu, n, l);
        return x;
    }
    __device__ __forceinline__ int at(int i) const { return i == 0 ? first : other + (i - 1) * step; }
};

// R rows a warp or W warps a row (one of them is 1).  Lane l finds what the pieces of row l % R are, before the wait for
// the kernel in front (the plan was complete before that kernel began); the loads of kBatch pieces of every row are then
// in flight at a time, the groups' pieces first, the sequence's own behind them.
template <typename T, int D, int W, int R>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const MergeParams p) {
    constexpr int kPer = D / 32, kRowsPerCta = kMergeThreads / 32 / W * R, kBatch = R > 1 ? 3 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
    const int row0 = blockIdx.x * kRowsPerCta + warp / W * R, r = row0 + lane % R;   // (rows are counted in 31 bits)
    const bool in = r < p.num_seqs * p.num_heads;
    const int s = in ? r / p.num_heads : 0, h = in ? r - s * p.num_heads : 0;
    const int len = in ? p.plan.own_len[s] : 0;
    const int g = in ? p.plan.seq_group[s] : 0;
    // all that may be needed, in two round trips
    const bool teams = p.plan.width != nullptr;
    const int width = teams ? *p.plan.width : 1;
    const int64_t P = p.pre_shares_dev ? *p.pre_shares_dev : p.pre_shares;
    const int64_t T0 = p.plan.tile_start[p.num_groups], T1 = teams ? p.plan.team_start[p.num_groups] : 0;
    const int C = p.plan.shared_len[g], s0 = __ldg(p.group_starts + g), s1 = __ldg(p.group_starts + g + 1);
    const int64_t begin0 = p.plan.tile_start[g], begin1 = teams ? p.plan.team_start[g] : 0;
    if (!p.own_start && T0 + T1 == 0) {   // nothing is shared: the decode kernel writes all rows
        grid_dependency_wait();           // (and has written them when this grid, the call's last, is done)
        return;
    }
    // a context length out of range leaves its row as it was; without shared tokens the decode kernel wrote it
    const bool mine = len > 0 && (p.own_start || C > 0);
    const int G = p.num_heads / p.num_kv_heads, kvh = h / G, hh = h - kvh * G;
    const int rows0 = p.num_seqs * p.num_heads;
    RowPieces pre, own;   // (of the lane's row)
    if (mine && C > 0) {
        const int n = s1 - s0;
        const GroupItems x = group_items(n, C, p.num_kv_heads, p.seqs_per_item, p.keys_per_tile, p.pair_seqs, width);
        const int part = x.pair ? 0 : (s - s0) / p.seqs_per_item;
        const int i = x.pair ? (kvh & 1) * n + s - s0 : s - s0 - part * p.seqs_per_item;   // row / G in the item
        const int first = (int)item_row(s0, n, kvh, s - s0, p.num_heads, G) + hh;
        if (part < x.blocks * width)
            pre = RowPieces(first, rows0 + ((part % width) * 2 + 1) * p.item_rows + i * G + hh, 2 * width * p.item_rows,
                            begin1 + (int64_t)(kvh * x.blocks + part / width) * x.kt, x.kt,
                            T1, P / width);
        else
            pre = RowPieces(first, rows0 + i * G + hh, (teams ? 2 : 1) * p.item_rows,
                            begin0 + (int64_t)(x.pair ? kvh >> 1 : kvh * x.rest + part - x.blocks * width) * x.kt,
                            x.kt, T0, P);
    }
    if (mine && p.own_start) {
        const int64_t kt = (len + p.keys_per_tile - 1) / p.keys_per_tile;
        own = RowPieces(r, rows0 + hh, G, p.own_start[s] * p.num_kv_heads + kvh * kt, kt,
                        p.own_start[p.num_seqs] * p.num_kv_heads, p.own_shares);
    } else if (mine) {
        own.first = r;
        own.n = 1;
    }
    grid_dependency_wait();
    grid_dependents_launch();
    RowSum<D> sum[R];
    RowPieces a[R], b[R];   // every row's, in all lanes
    int most = 0;
#pragma unroll
    for (int q = 0; q < R; ++q) {
        a[q] = pre.of_lane(q);
        b[q] = own.of_lane(q);
        most = max(most, a[q].n + b[q].n);
    }
    for (int i = w; i < most; i += W * kBatch) {
        float2 ml[R][kBatch];
        float v[R][kBatch][kPer];
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int x = i + W * k, y = x - a[q].n;
                if (y >= b[q].n) continue;
                const int64_t at = y < 0 ? a[q].at(x) : b[q].at(y);   // (times D below)
                ml[q][k] = __ldcg((y < 0 ? p.pre_ml : p.own_ml) + at);
                load_dims<D>((y < 0 ? p.pre_o : p.own_o) + at * D + lane * kPer, v[q][k]);
            }
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i + W * k < a[q].n + b[q].n) sum[q].add(ml[q][k], v[q][k]);
    }
    if (W > 1) {
        __shared__ float2 ml_s[W];
        __shared__ float o_s[W][D];
        if (lane == 0) ml_s[w] = make_float2(sum[0].M, sum[0].L);
#pragma unroll
        for (int u = 0; u < kPer; ++u) o_s[w][lane * kPer + u] = sum[0].acc[u];
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int i = 1; i < W; ++i) {
            float v[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) v[u] = o_s[i][lane * kPer + u];
            sum[0].add(ml_s[i], v);
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if (a[q].n + b[q].n == 0) continue;   // not this kernel's row
        T *dst = static_cast<T *>(p.out) + (int64_t)(row0 + q) * D + lane * kPer;
        const float inv = 1.f / sum[q].L;
        if (sizeof(T) == 2 && p.out_aligned) {
#pragma unroll
            for (int u = 0; u < kPer; u += 2)
                *reinterpret_cast<uint32_t *>(dst + u) = pack_bf16x2(sum[q].acc[u] * inv, sum[q].acc[u + 1] * inv);
        } else {
#pragma unroll
            for (int u = 0; u < kPer; ++u) dst[u] = from_float<T>(sum[q].acc[u] * inv);
        }
    }
}

// ------------------------------------------------------------------ host side
// Workspace: the plan's arrays, then the pieces.
struct Layout {
    size_t seq_group, own_len, shared_len, scratch, tile_start, own_start, pre_ml, pre_o, own_ml, own_o, total;
};

Layout layout(int num_seqs, int num_groups, int num_heads, int num_kv_heads, int head_dim) {
    Layout w;
    const size_t S = num_seqs, NG = num_groups, G = num_heads / num_kv_heads > 0 ? num_heads / num_kv_heads : 1;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t a = at; at = align_up(at + bytes, 256); return a; };
    w.seq_group = take(4 * S);
    w.own_len = take(4 * S);
    w.shared_len = take(4 * NG);
    w.scratch = take(4 * NG);
    w.tile_start = take(8 * (NG + 1));
    w.own_start = take(8 * (S + 1));
    const size_t spi = kRows / G > 0 ? kRows / G : 1;
    const size_t pre_rows = S * num_heads + kMaxCtas * (spi < S ? spi : S) * G, own_rows = S * num_heads + kMaxCtas * G;
    w.pre_ml = take(8 * pre_rows);
    w.pre_o = take(4 * pre_rows * head_dim);
    w.own_ml = take(8 * own_rows);
    w.own_o = take(4 * own_rows * head_dim);
    w.total = at;
    return w;
}

template <typename T, int D>
cudaError_t launch_merge(const MergeParams &mg, cudaStream_t stream) {
    // A row has about P / items pieces and an item at most 256 rows, so with few rows there may be many pieces each:
    // then four warps share them.  Else four rows a warp, so that they all are resident at once.  Both ways, 32 / 8 heads x
    // 128, the whole call with a flushed L2: 64 sequences over 32,768 tokens 68.7 and 72.8 us, 72 79.0 and 74.2, 128 97.4
    // and 87.1; 64 over 131,072 136.3 and 140.4, 80 187.5 and 183.4; 128 over up to 5120 74.2 and 66.7.
    const int64_t rows = (int64_t)mg.num_seqs * mg.num_heads;
    constexpr int kWarps = kMergeThreads / 32, kCta = kWarps * kRowsPerWarp;
    if (rows < kFewRows)
        return launch_dependent(shared_merge_kernel<T, D, kWarps, 1>, dim3((unsigned)rows), dim3(kMergeThreads), 0, stream, mg);
    return launch_dependent(shared_merge_kernel<T, D, 1, kRowsPerWarp>, dim3((unsigned)((rows + kCta - 1) / kCta)),
                            dim3(kMergeThreads), 0, stream, mg);
}

template <typename T, int D, int R>
cudaError_t launch_few(const CcParams &cc, int grid, cudaStream_t stream) {
    constexpr int L = (R > 4 ? R : 4) * D / 32, kStreams = kCcThreads / L;
    return launch_dependent(shared_few_kernel<T, D, R>, dim3(grid), dim3(kCcThreads), kStreams * R * (D + 2) * sizeof(float),
                            stream, cc);
}

template <typename T, int D>
cudaError_t launch_typed(const CcParams &cc, const MergeParams &mg, int grid, cudaStream_t stream) {
    auto kern = shared_rows_kernel<T, D>;
    constexpr size_t smem = cc_smem_floats<D>() * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(grid), dim3(kCcThreads), smem, stream, cc);
    if (e != cudaSuccess) return e;
    const int G = cc.num_heads / cc.num_kv_heads;
    if (G <= kFewHeads) {
        // (bf16 comes here only with unaligned rows or a scale that is not positive: one form will do)
        if (sizeof(T) == 2 || G > 4) e = launch_few<T, D, 8>(cc, grid, stream);
        else if (G > 2) e = launch_few<float, D, 4>(cc, grid, stream);
        else e = launch_few<float, D, 2>(cc, grid, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_merge<T, D>(mg, stream);
}

// Workspace of the tensor-core path: the plan's arrays, the prefix pieces, the own parts, the decode kernel's.
struct TcLayout {
    size_t seq_group, own_len, shared_len, tile_start, team_start, shares, pre_ml, pre_o, own_ml, own_o, decode, total;
    int item_rows;
};

TcLayout tc_layout(int num_seqs, int num_groups, int num_heads, int num_kv_heads, int head_dim, int max_blocks, int B) {
    TcLayout w;
    const size_t S = num_seqs, NG = num_groups;
    const int G = num_heads / num_kv_heads > 0 ? num_heads / num_kv_heads : 1;
    const int spi = G <= 128 ? prefix_seqs_per_item(G) : 1;
    w.item_rows = (spi < 2 * num_seqs ? spi : 2 * num_seqs) * G;   // (two kv-heads of a small group)
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t a = at; at = align_up(at + bytes, 256); return a; };
    w.seq_group = take(4 * S);
    w.own_len = take(4 * S);
    w.shared_len = take(4 * NG);
    w.tile_start = take(8 * (NG + 1));
    w.team_start = take(8 * (NG + 1));
    w.shares = take(8);   // and the teams' width
    const size_t rows = S * num_heads, pre_rows = rows + (size_t)2 * kMaxPrefixCtas * w.item_rows;
    w.pre_ml = take(8 * pre_rows);
    w.pre_o = take(4 * pre_rows * head_dim);
    w.own_ml = take(8 * rows);
    w.own_o = take(4 * rows * head_dim);
    w.decode = take(split_decode_workspace(num_seqs, num_heads, head_dim, max_blocks, B));
    w.total = at;
    return w;
}

// The tensor-core path takes what the split decode takes (out on 4 bytes: no kernel stores wider to it), a positive scale
// (the running maximum is that of the unscaled products) and groups whose starts the plan's CTAs hold in shared memory.
bool tc_supported(const AttnArgs &a, int num_groups) {
    return split_decode_supported(a) && a.scale > 0.f && a.scale < INFINITY && num_groups <= kMaxPrefixGroups;
}

cudaError_t launch_tc(const AttnArgs &a, const int32_t *group_starts, const int32_t *prefix_lens, int num_groups,
                      void *workspace, cudaStream_t stream) {
    const TcLayout w = tc_layout(a.num_seqs, num_groups, a.num_heads, a.num_kv_heads, a.head_dim, a.max_blocks, a.block_size);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int spi = prefix_seqs_per_item(a.num_heads / a.num_kv_heads), pair = a.num_kv_heads % 2 == 0 ? spi / 2 : 0;
    const int (&tile_ns)[3] = kTcTileNs[a.head_dim == 64 ? 0 : 1];
    SharedJob job;
    job.groups = {a.context_lens, group_starts, prefix_lens, a.num_seqs, num_groups, a.num_kv_heads, a.block_size,
                  (int64_t)a.max_blocks * a.block_size, spi, kPrefixKeys, pair, device_sm_count() > 2 * kMaxTeam ? kMaxTeam : 1, 16,
                  split_decode_unit_ns(a.num_heads, a.num_kv_heads, a.head_dim), {spi / 2, spi / 2},
                  {tile_ns[0], tile_ns[0], tile_ns[1], tile_ns[2]}, kTcItemNs, kLeastSavedNs * device_sm_count(),
                  kLongPrefix};
    job.plan = {reinterpret_cast<int32_t *>(ws + w.seq_group), reinterpret_cast<int32_t *>(ws + w.own_len),
                reinterpret_cast<int32_t *>(ws + w.shared_len), reinterpret_cast<int64_t *>(ws + w.tile_start),
                reinterpret_cast<int64_t *>(ws + w.team_start), reinterpret_cast<int32_t *>(ws + w.shares) + 1};
    job.shares = reinterpret_cast<int32_t *>(ws + w.shares);
    job.pre_o = reinterpret_cast<float *>(ws + w.pre_o);
    job.pre_ml = reinterpret_cast<float2 *>(ws + w.pre_ml);
    job.item_rows = w.item_rows;
    job.own_o = reinterpret_cast<float *>(ws + w.own_o);
    job.own_ml = reinterpret_cast<float2 *>(ws + w.own_ml);
    const std::function<cudaError_t()> prefix = [&] { return launch_prefix(a, job, stream); };
    cudaError_t e = launch_split_decode(a, ws + w.decode, w.total - w.decode, stream, false, nullptr, nullptr, &prefix, &job);
    if (e != cudaSuccess) return e;
    MergeParams mg = {a.out, group_starts, job.plan, nullptr, job.pre_o, job.pre_ml, job.own_o, job.own_ml, job.shares, 0, 0,
                      job.item_rows, spi, kPrefixKeys, pair, a.num_seqs, num_groups, a.num_heads, a.num_kv_heads, 1};
    return a.head_dim == 64 ? launch_merge<__nv_bfloat16, 64>(mg, stream) : launch_merge<__nv_bfloat16, 128>(mg, stream);
}

}  // namespace

size_t shared_prefix_workspace(int num_seqs, int num_groups, int num_heads, int num_kv_heads, int head_dim, int max_blocks,
                               int block_size) {
    const size_t cc = layout(num_seqs, num_groups, num_heads, num_kv_heads, head_dim).total;
    const size_t tc = tc_layout(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_blocks, block_size).total;
    return (cc > tc ? cc : tc) + kAlign - 16;
}

cudaError_t launch_shared_prefix(const AttnArgs &a, const int32_t *group_starts, const int32_t *prefix_lens, int num_groups,
                                 void *workspace, cudaStream_t stream) {
    workspace = reinterpret_cast<void *>(align_up(reinterpret_cast<uintptr_t>(workspace), kAlign));
    if (tc_supported(a, num_groups)) return launch_tc(a, group_starts, prefix_lens, num_groups, workspace, stream);
    const Layout w = layout(a.num_seqs, num_groups, a.num_heads, a.num_kv_heads, a.head_dim);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int G = a.num_heads / a.num_kv_heads, spi = kRows / G;
    const SharedPlan plan = {reinterpret_cast<int32_t *>(ws + w.seq_group), reinterpret_cast<int32_t *>(ws + w.own_len),
                             reinterpret_cast<int32_t *>(ws + w.shared_len), reinterpret_cast<int64_t *>(ws + w.tile_start), nullptr,
                             nullptr};
    int64_t *own_start = reinterpret_cast<int64_t *>(ws + w.own_start);
    const int (&tile_ns)[3] = kCcTileNs[a.head_dim == 64 ? 0 : 1];
    const SharedGroups groups = {a.context_lens, group_starts, prefix_lens, a.num_seqs, num_groups, a.num_kv_heads,
                                 a.block_size, (int64_t)a.max_blocks * a.block_size, spi, kKeys, 0, 1, kKeys,
                                 a.num_kv_heads * tile_ns[G <= 8 ? 0 : 1], {8 / G, 32 / G},
                                 {tile_ns[0], tile_ns[1], tile_ns[2], 0}, kCcItemNs, kCcLeastSavedNs * device_sm_count(),
                                 INT_MAX};
    cudaError_t e = launch_dependent(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, groups, plan,
                                     reinterpret_cast<int32_t *>(ws + w.scratch), own_start, a.status);
    if (e != cudaSuccess) return e;
    auto in16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const int sms = device_sm_count(), grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    CcParams cc = {a.q, a.k_cache, a.v_cache, a.block_tables, group_starts, plan, own_start};
    cc.pre_o = reinterpret_cast<float *>(ws + w.pre_o);
    cc.pre_ml = reinterpret_cast<float2 *>(ws + w.pre_ml);
    cc.own_o = reinterpret_cast<float *>(ws + w.own_o);
    cc.own_ml = reinterpret_cast<float2 *>(ws + w.own_ml);
    cc.item_rows = (spi < a.num_seqs ? spi : a.num_seqs) * G;
    cc.seqs_per_item = spi;
    cc.num_seqs = a.num_seqs;
    cc.num_groups = num_groups;
    cc.num_heads = a.num_heads;
    cc.num_kv_heads = a.num_kv_heads;
    cc.block_size = a.block_size;
    cc.log2b = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    cc.max_blocks = a.max_blocks;
    cc.num_blocks = a.num_blocks;
    cc.aligned = in16(a.q) && in16(a.k_cache) && in16(a.v_cache) ? 1 : 0;
    cc.scale_log2 = a.scale * 1.4426950408889634f;
    cc.status = a.status;
    MergeParams mg = {a.out, group_starts, plan, own_start, cc.pre_o, cc.pre_ml, cc.own_o, cc.own_ml, nullptr, grid, grid, cc.item_rows, spi,
                      kKeys, 0, a.num_seqs, num_groups, a.num_heads, a.num_kv_heads,
                      reinterpret_cast<uintptr_t>(a.out) % 4 == 0};
    if (a.dtype == PA_DTYPE_F32)
        return a.head_dim == 64 ? launch_typed<float, 64>(cc, mg, grid, stream)
                                : launch_typed<float, 128>(cc, mg, grid, stream);
    return a.head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(cc, mg, grid, stream)
                            : launch_typed<__nv_bfloat16, 128>(cc, mg, grid, stream);
}

}  // namespace pa
