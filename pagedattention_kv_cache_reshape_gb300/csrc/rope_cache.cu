// rope_cache.cu -- position rotation of the step's queries and keys, with the
// K/V rows written into the paged pools on the way (16/32-bit or 4-bit pools).
//
// For token t at position p = positions[t], R = rot_dim / 2 and the pair
// (a, b) = (x[i], x[i + R]) (halves) or (x[2i], x[2i + 1]) (interleaved):
//     a' = a cos_i - b sin_i,   b' = b cos_i + a sin_i,
// cos_i = cos_sin[p][i], sin_i = cos_sin[p][R + i]; dims from rot_dim on pass
// through.  The row is rounded to the inputs' type and stored like
// reshape_and_cache's, or quantised from there (q4_format.cuh).
//
// Bound by HBM: every row is read and written once.  A thread of the fast
// kernel owns the two vectors of 8 dims whose elements pair up, so it needs 8
// cosines and 8 sines for 16 values, no exchange with other lanes, and may
// write q in place; a CTA takes a token's rows in one pass, K and V rows among
// them.  Rows that do not come in 16-byte pieces (head_dim or rot_dim no
// multiple of 16, odd addresses or strides) take the element-wise kernel.
// Measured: 8192 tokens of 32 + 8 + 8 rows of 128 bf16 (204 MB) 34.6 us, 5.9 TB/s;
// 256 tokens 2.6 us; fp32 67 us, 6.0 TB/s.  Into 4-bit pools 8191 tokens take 43
// us from cold caches at 63 % of the issue slots: the keys' exact rotation and
// the codes cost it half as many instructions again (29.1 M against 19.5 M);
// fp32 69 us.  Head sizes of other lanes: 32 + 8 + 8 rows of 96 30.0 us, of 192
// 55.4.  The element-wise kernel is far slower: with 72 or 36 of the dims turned
// the 8192 tokens take 165 us (neighbouring pairs 171-175), into 4-bit pools
// 440-470.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;
// Threads of a CTA of the fast kernel.  One token a CTA (few tokens): all rows of a usual token at once.  Two: small
// CTAs, 16 of them with 64 registers an SM, whose loads and stores overlap (8192 tokens of 48 rows: 64 threads 34.4
// us, 128 35.3, 192 36.9, 384 40.5).
constexpr int vec_threads(int U) { return U == 1 ? 384 : 64; }

// a c + b s (s negated: a c - b s), the exact value rounded once to fp32, or, where
// a product or the sum is not finite, what fp32 gives: both products are split
// into value and error (fma), the sum into value and error, and the errors are
// added last.  The 4-bit code of a key depends on which side of a border its
// rotated value lies, so the rotation must not add an error of its own there.
// kQ4: for 4-bit pools, where a group with an infinity and one with a NaN are
// the same; the instruction that keeps infinities is left out there (8191
// tokens with the expansion of their blocks 51.3 us against 52.4).
template <bool kQ4>
__device__ __forceinline__ float rotate_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), ep = __fmaf_rn(a, c, -p);
    const float w = __fmul_rn(b, s), ew = __fmaf_rn(b, s, -w);
    const float sum = __fadd_rn(p, w);
    const float bb = __fsub_rn(sum, p);
    const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, bb)), __fsub_rn(w, bb));
    const float err = __fadd_rn(es, __fadd_rn(ep, ew));
    // With infinite products or sums err is NaN (inf - inf in es), and the maximum takes its other operand: an
    // infinite sum stays what it is.  The errors of a finite sum are three half steps, 2^103 each, at most.
    return __fadd_rn(sum, kQ4 ? err : fmaxf(err, -0x1p105f));
}

// A pair turned in place: keys exactly, queries with one rounding more.
template <bool kQ4>
__device__ __forceinline__ void turn(float &a, float &b, float c, float s, bool is_q) {
    const float x = a, y = b;
    if (is_q) {
        a = __fmaf_rn(x, c, -__fmul_rn(y, s));
        b = __fmaf_rn(y, c, __fmul_rn(x, s));
    } else {
        a = rotate_exact<kQ4>(x, c, y, -s);
        b = rotate_exact<kQ4>(y, c, x, s);
    }
}

template <typename T, bool kQ4>
__device__ __forceinline__ float rotated(const RopeArgs &a, const T *row, const float *cs, int d) {
    const int R = a.rot_dim / 2;
    const float x = to_float(row[d]);
    if (d >= a.rot_dim) return x;
    int i, o;
    bool first;
    if (a.interleaved) { i = d >> 1; first = (d & 1) == 0; o = d ^ 1; }
    else { first = d < R; i = first ? d : d - R; o = first ? d + R : d - R; }
    const float y = to_float(row[o]);
    return rotate_exact<kQ4>(x, cs[i], y, first ? -cs[R + i] : cs[R + i]);
}

// Any shape, element by element: one CTA per token.
template <typename T, bool kQ4>
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const RopeArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0) return;   // padding token
    const int pos = a.rot_dim > 0 ? a.positions[t] : 0;
    if (slot >= (int64_t)a.num_blocks * a.block_size || pos < 0 || (a.rot_dim > 0 && pos >= a.max_position)) {
        if (tid == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const float *cs = a.cos_sin + (int64_t)pos * a.rot_dim;
    const int D = a.head_dim;
    // queries: a thread owns both dims of a pair (q_out may be q)
    for (int64_t e = tid; e < (int64_t)a.num_heads * D; e += kThreads) {
        const int h = (int)(e / D), d = (int)(e - (int64_t)h * D);
        const T *row = static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)h * D;
        T *out = static_cast<T *>(a.q_out) + ((int64_t)t * a.num_heads + h) * D;
        if (d >= a.rot_dim) { out[d] = row[d]; continue; }
        const int R = a.rot_dim / 2;
        if (a.interleaved ? (d & 1) : d >= R) continue;
        const int o = a.interleaved ? d + 1 : d + R;
        const int i = a.interleaved ? d >> 1 : d;
        float x = to_float(row[d]), y = to_float(row[o]);
        turn<kQ4>(x, y, cs[i], cs[R + i], true);
        out[d] = from_float<T>(x);
        out[o] = from_float<T>(y);
    }
    const T *key = static_cast<const T *>(a.key) + t * a.key_stride;
    const T *value = static_cast<const T *>(a.value) + t * a.value_stride;
    if (!kQ4) {
        T *kd = static_cast<T *>(a.k_cache) + slot * ((int64_t)a.num_kv_heads * D);
        T *vd = static_cast<T *>(a.v_cache) + slot * ((int64_t)a.num_kv_heads * D);
        for (int64_t e = tid; e < (int64_t)a.num_kv_heads * D; e += kThreads) {
            const int h = (int)(e / D), d = (int)(e - (int64_t)h * D);
            kd[e] = from_float<T>(rotated<T, kQ4>(a, key + (int64_t)h * D, cs, d));
            vd[e] = value[e];
        }
        return;
    }
    // rows of 4 or 8 neighbouring lanes, 16 dims a lane
    const int lanes = D / 16, k = lane % lanes;
    const int64_t blk = slot / a.block_size;
    const int off = (int)(slot - blk * a.block_size);
    const int64_t slab = q4_slab_bytes(a.block_size, D);
    for (int j0 = warp * (32 / lanes); j0 < 2 * a.num_kv_heads; j0 += (kThreads / 32) * (32 / lanes)) {
        const int j = j0 + lane / lanes;
        const bool in = j < 2 * a.num_kv_heads, is_v = in && j >= a.num_kv_heads;
        const int h = in ? (is_v ? j - a.num_kv_heads : j) : 0;
        Raw8<T> x[2];
        for (int i = 0; i < 16; ++i)
            reinterpret_cast<T *>(x)[i] = is_v ? value[(int64_t)h * D + 16 * k + i]
                                               : from_float<T>(rotated<T, kQ4>(a, key + (int64_t)h * D, cs, 16 * k + i));
        uint8_t *s = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) + (blk * a.num_kv_heads + h) * slab;
        uint8_t *row = s + off * q4_row_bytes(D);
        uint16_t *scales = reinterpret_cast<uint16_t *>(s + a.block_size * q4_row_bytes(D)) + off * (D / kQ4Group);
        if (D == 128) q4_store16<128>(x[0], x[1], k, is_v, row, scales, in);
        else q4_store16<64>(x[0], x[1], k, is_v, row, scales, in);
    }
}

// The two vectors of 8 that a thread owns, turned and rounded to T.
template <typename T, bool kQ4>
__device__ __forceinline__ void turn_rows(Raw8<T> &rx, Raw8<T> &ry, const RopeArgs &a, int pos, int j, bool is_q) {
    float c[8], s[8], x[8], y[8];
    const float *cs = a.cos_sin + (int64_t)pos * a.rot_dim + 8 * j;
    to_floats(c, load_raw8(cs));
    to_floats(s, load_raw8(cs + a.rot_dim / 2));
    to_floats(x, rx);
    to_floats(y, ry);
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // pair i is (x[2i], x[2i + 1]) or, from 4 on, y's
            float &v = i < 4 ? x[2 * i] : y[2 * i - 8], &w = i < 4 ? x[2 * i + 1] : y[2 * i - 7];
            turn<kQ4>(v, w, c[i], s[i], is_q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn<kQ4>(x[i], y[i], c[i], s[i], is_q);
    }
    rx = from_floats<T>(x);
    ry = from_floats<T>(y);
}

// One CTA per U tokens, `passes` x `rows` head rows of a token at a time, D / 16 threads a row.  Rows 0 ..
// num_heads - 1 are queries, then keys, then values.  Thread j of a row, j < rot_dim / 16: the rotated vectors 8 j
// and R + 8 j (halves) or 16 j and 16 j + 8 (interleaved); the others: the vectors from rot_dim on.  The rows are
// requested before the slots and positions that decide what becomes of them.  4-bit pools, kQ4 = 1: rows that turn
// as a whole or not at all are quantised by the lanes that hold them (a group is 2 or 4 neighbouring lanes);
// kQ4 = 2: with rot_dim between, the rotated keys and the values meet in shared memory, where 16 consecutive dims
// go to a lane.
template <typename T, int kQ4, int U>
__global__ void __launch_bounds__(vec_threads(U), U == 1 ? 2 : 16) rope_cache_vec_kernel(const RopeArgs a, int rows, int passes) {
    extern __shared__ __align__(16) uint8_t smem[];
    T *kv_s = reinterpret_cast<T *>(smem);   // [U][2 num_kv_heads][D], kQ4 = 2 only
    const int D = a.head_dim, lanes = D / 16, tid = threadIdx.x;
    const int row0 = tid / lanes, j = tid - row0 * lanes, R = a.rot_dim / 2;
    const int H = a.num_heads, HK = a.num_kv_heads, all = H + 2 * HK;
    const bool turns = j < R / 8;
    const int d0 = turns ? (a.interleaved ? 16 * j : 8 * j) : 16 * j;
    const int d1 = turns && !a.interleaved ? R + 8 * j : d0 + 8;
    const int t0 = blockIdx.x * U;
    const int log2b = 31 - __clz(a.block_size);   // 4-bit pools: 8, 16 or 32
    grid_dependency_wait();
    grid_dependents_launch();
    int64_t slot[U];
    int pos[U];
    bool live[U];
    for (int pass = 0; pass < passes; ++pass) {
        const int row = row0 + pass * rows;
        const bool mine = row0 < rows && row < all;
        const bool is_q = row < H, is_v = row >= H + HK;
        const int h = is_q ? row : is_v ? row - H - HK : row - H;
        const T *base = static_cast<const T *>(is_q ? a.q : is_v ? a.value : a.key) + (int64_t)h * D;
        const int64_t stride = is_q ? a.q_stride : is_v ? a.value_stride : a.key_stride;
        Raw8<T> rx[U], ry[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (mine && t0 + u < a.num_tokens) {
                rx[u] = load_raw8(base + (t0 + u) * stride + d0);
                ry[u] = load_raw8(base + (t0 + u) * stride + d1);
            }
        if (pass == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = t0 + u < a.num_tokens;
                slot[u] = in ? __ldg(a.slot_mapping + t0 + u) : -1;
                pos[u] = in && a.rot_dim > 0 ? __ldg(a.positions + t0 + u) : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                live[u] = slot[u] >= 0;   // else padding
                if (live[u] && (slot[u] >= (int64_t)a.num_blocks * a.block_size || pos[u] < 0 ||
                                (a.rot_dim > 0 && pos[u] >= a.max_position))) {
                    live[u] = false;
                    if (tid == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
                }
            }
        }
        const bool quant = kQ4 == 1 && mine && !is_q;
        if (kQ4 == 1 ? !__any_sync(0xffffffffu, mine) : !mine) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!live[u]) continue;   // the same in every thread
            if (kQ4 == 1) {
                if (mine && turns && !is_v) turn_rows<T, kQ4 != 0>(rx[u], ry[u], a, pos[u], j, is_q);
                if (mine && is_q) {
                    T *dst = static_cast<T *>(a.q_out) + ((int64_t)(t0 + u) * H + h) * D;
                    store_raw8(dst + d0, rx[u]);
                    store_raw8(dst + d1, ry[u]);
                }
                if (__any_sync(0xffffffffu, quant)) {
                    const int64_t blk = slot[u] >> log2b;
                    const int off = (int)slot[u] & (a.block_size - 1);
                    const int64_t slab = q4_slab_bytes(a.block_size, D);
                    uint8_t *to = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) + (blk * HK + (quant ? h : 0)) * slab;
                    uint8_t *codes = to + off * q4_row_bytes(D);
                    uint16_t *scales = reinterpret_cast<uint16_t *>(to + a.block_size * q4_row_bytes(D)) + off * (D / kQ4Group);
                    const bool v = is_v && quant;
                    if (a.rot_dim > 0 && !a.interleaved) {
                        if (D == 128) q4_store8x2<128>(rx[u], ry[u], j, v, codes, scales, quant);
                        else q4_store8x2<64>(rx[u], ry[u], j, v, codes, scales, quant);
                    } else {
                        if (D == 128) q4_store16<128>(rx[u], ry[u], j, v, codes, scales, quant);
                        else q4_store16<64>(rx[u], ry[u], j, v, codes, scales, quant);
                    }
                }
                continue;
            }
            T *dst;
            if (is_q) dst = static_cast<T *>(a.q_out) + ((int64_t)(t0 + u) * H + h) * D;
            else if (kQ4 == 2) dst = kv_s + (u * 2 * HK + row - H) * D;
            else dst = static_cast<T *>(is_v ? a.v_cache : a.k_cache) + (slot[u] * HK + h) * D;
            if (turns && !is_v) turn_rows<T, kQ4 != 0>(rx[u], ry[u], a, pos[u], j, is_q);
            store_raw8(dst + d0, rx[u]);
            store_raw8(dst + d1, ry[u]);
        }
    }
    if (kQ4 != 2) return;
    __syncthreads();
    const int per = D / 16, k = tid % per;   // a row's lanes lie in one warp: per is 4 or 8
    const int64_t slab = q4_slab_bytes(a.block_size, D);
    for (int r0 = 0; r0 < U * 2 * HK; r0 += blockDim.x / per) {
        if (r0 + (tid & ~31) / per >= U * 2 * HK) break;   // whole warps
        const int r = r0 + tid / per, u = U > 1 && r >= 2 * HK ? 1 : 0, row = r - u * 2 * HK;
        const int64_t sl = U > 1 && u ? slot[U - 1] : slot[0];
        const bool in = r < U * 2 * HK && (U > 1 && u ? live[U - 1] : live[0]), is_v = in && row >= HK;
        const int64_t blk = in ? sl >> log2b : 0;
        const int off = in ? (int)sl & (a.block_size - 1) : 0;
        const T *src = kv_s + (in ? r : 0) * D + 16 * k;
        uint8_t *to = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) +
                      (blk * HK + (in ? row - (is_v ? HK : 0) : 0)) * slab;
        uint8_t *codes = to + off * q4_row_bytes(D);
        uint16_t *scales = reinterpret_cast<uint16_t *>(to + a.block_size * q4_row_bytes(D)) + off * (D / kQ4Group);
        if (D == 128) q4_store16<128>(load_raw8(src), load_raw8(src + 8), k, is_v, codes, scales, in);
        else q4_store16<64>(load_raw8(src), load_raw8(src + 8), k, is_v, codes, scales, in);
    }
}

template <typename T, int kQ4>
cudaError_t launch_vec(const RopeArgs &a, int64_t kv_bytes, cudaStream_t stream) {
    const int lanes = a.head_dim / 16;
    const int64_t all = (int64_t)a.num_heads + 2 * a.num_kv_heads;
    // whole rows a pass, evened out over the passes: rows <= threads / lanes, so that a CTA, rounded up to whole warps,
    // stays within the kernel's launch bound (`threads` is a multiple of 32) whatever head_dim / 16 is
    auto shape = [&](int threads, int &rows, int &passes) {
        const int most = threads / lanes;
        passes = (int)((all + most - 1) / most);
        rows = (int)((all + passes - 1) / passes);
        return dim3((rows * lanes + 31) / 32 * 32);
    };
    int rows, passes;
    // Two tokens a CTA once one each would fill the GPU several times over: twice the loads in flight.  32 + 8 + 8
    // rows of 128 bf16, one a CTA against two: 608 tokens 4.7 and 7.2 us, 912 6.4 and 7.7, 1216 8.1 and 8.1, 1520 9.9
    // and 8.5, 2432 15.0 and 9.8; into 4-bit pools 912 8.3 and 10.7, 1216 10.6 and 11.1, 1520 13.0 and 11.7.
    if (a.num_tokens >= 8 * device_sm_count() && 2 * kv_bytes <= 48 * 1024) {
        const dim3 block = shape(vec_threads(2), rows, passes);
        return launch_dependent(rope_cache_vec_kernel<T, kQ4, 2>, dim3((a.num_tokens + 1) / 2), block,
                                (size_t)(2 * kv_bytes), stream, a, rows, passes);
    }
    const dim3 block = shape(vec_threads(1), rows, passes);
    return launch_dependent(rope_cache_vec_kernel<T, kQ4, 1>, dim3(a.num_tokens), block, (size_t)kv_bytes, stream, a,
                            rows, passes);
}

template <typename T>
cudaError_t launch_typed(const RopeArgs &a, bool q4, cudaStream_t stream) {
    // the fast kernel's rows come in 16-byte pieces; a token's keys and values fit shared memory
    const bool whole = a.rot_dim == 0 || a.rot_dim == a.head_dim;
    const int64_t kv_bytes = q4 && !whole ? (int64_t)2 * a.num_kv_heads * a.head_dim * sizeof(T) : 0;
    auto in16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const int64_t e = sizeof(T);
    bool vec = a.head_dim % 16 == 0 && a.rot_dim % 16 == 0 && a.head_dim <= 512 && kv_bytes <= 48 * 1024 &&
               a.key_stride * e % 16 == 0 && a.value_stride * e % 16 == 0 && in16(a.key) && in16(a.value) &&
               in16(a.k_cache) && in16(a.v_cache) && (a.rot_dim == 0 || in16(a.cos_sin));
    if (a.num_heads > 0) vec = vec && a.q_stride * e % 16 == 0 && in16(a.q) && in16(a.q_out);
    if (vec && q4) return whole ? launch_vec<T, 1>(a, 0, stream) : launch_vec<T, 2>(a, kv_bytes, stream);
    if (vec) return launch_vec<T, 0>(a, 0, stream);
    const dim3 grid(a.num_tokens), block(kThreads);
    return q4 ? launch_dependent(rope_cache_kernel<T, true>, grid, block, 0, stream, a)
              : launch_dependent(rope_cache_kernel<T, false>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs &a, bool q4, cudaStream_t stream) {
    if (a.num_tokens == 0) return cudaSuccess;
    return a.dtype == PA_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(a, q4, stream) : launch_typed<float>(a, q4, stream);
}

}  // namespace pa
