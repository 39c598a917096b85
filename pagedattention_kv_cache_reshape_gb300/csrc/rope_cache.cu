// rope_cache.cu -- position rotation of the step's queries and keys, with the
// K/V rows written into the paged pools on the way (16/32-bit or 4-bit pools).
//
// For token t at position p = positions[t], R = rot_dim / 2 and the pair
// (a, b) = (x[i], x[i + R]) (halves) or (x[2i], x[2i + 1]) (interleaved):
//     a' = a cos_i - b sin_i,   b' = b cos_i + a sin_i,
// cos_i = cos_sin[p][i], sin_i = cos_sin[p][R + i]; dims from rot_dim on pass
// through.  The row is rounded to the inputs' type and stored like
// reshape_and_cache's, or quantised from there (q4_format.cuh).
#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;

// a c - b s (sign = -1) or a c + b s (sign = +1), the exact value rounded once to
// fp32: both products are split into value and error (fma), the sum into value
// and error, and the errors are added last.  The 4-bit code of a key depends
// on which side of a border its rotated value lies, so the rotation must not
// add an error of its own there.
__device__ __forceinline__ float rotate_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), ep = __fmaf_rn(a, c, -p);
    const float w = __fmul_rn(b, s), ew = __fmaf_rn(b, s, -w);
    const float sum = __fadd_rn(p, w);
    const float bb = __fsub_rn(sum, p);
    const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, bb)), __fsub_rn(w, bb));
    return __fadd_rn(sum, __fadd_rn(es, __fadd_rn(ep, ew)));
}

template <typename T>
__device__ __forceinline__ float rotated(const RopeArgs &a, const T *row, const float *cs, int d) {
    const int R = a.rot_dim / 2;
    const float x = to_float(row[d]);
    if (d >= a.rot_dim) return x;
    int i, o;
    bool first;
    if (a.interleaved) { i = d >> 1; first = (d & 1) == 0; o = d ^ 1; }
    else { first = d < R; i = first ? d : d - R; o = first ? d + R : d - R; }
    const float y = to_float(row[o]);
    return rotate_exact(x, cs[i], y, first ? -cs[R + i] : cs[R + i]);
}

// One CTA per token.
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
        const float y0 = rotated(a, row, cs, d), y1 = rotated(a, row, cs, o);
        out[d] = from_float<T>(y0);
        out[o] = from_float<T>(y1);
    }
    const T *key = static_cast<const T *>(a.key) + t * a.key_stride;
    const T *value = static_cast<const T *>(a.value) + t * a.value_stride;
    if (!kQ4) {
        T *kd = static_cast<T *>(a.k_cache) + slot * ((int64_t)a.num_kv_heads * D);
        T *vd = static_cast<T *>(a.v_cache) + slot * ((int64_t)a.num_kv_heads * D);
        for (int64_t e = tid; e < (int64_t)a.num_kv_heads * D; e += kThreads) {
            const int h = (int)(e / D), d = (int)(e - (int64_t)h * D);
            kd[e] = from_float<T>(rotated(a, key + (int64_t)h * D, cs, d));
            vd[e] = value[e];
        }
        return;
    }
    // one warp per (head, group, K or V), a lane per dim
    const int ng = D / kQ4Group;
    const int64_t blk = slot / a.block_size;
    const int off = (int)(slot - blk * a.block_size);
    const int64_t slab = q4_slab_bytes(a.block_size, D);
    for (int j = warp; j < 2 * a.num_kv_heads * ng; j += kThreads / 32) {
        const int is_v = j & 1, g = (j >> 1) % ng, h = (j >> 1) / ng;
        const int d = g * kQ4Group + lane;
        const float x = is_v ? to_float(value[(int64_t)h * D + d])
                             : to_float(from_float<T>(rotated(a, key + (int64_t)h * D, cs, d)));
        float amax = fabsf(x);
        const bool finite = __all_sync(0xffffffffu, amax <= 3.402823466e38f);
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const uint16_t sb = q4_scale_bits(amax, finite);
        uint32_t w = q4_code(x, q4_scale_value(sb)) << (4 * (lane & 7));
        for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
        uint8_t *s = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) +
                     (blk * a.num_kv_heads + h) * slab;
        uint8_t *row = s + off * q4_row_bytes(D);
        if (!is_v) {
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t *>(row + q4_k_word(d, D)) = w;
        } else if ((lane & 3) == 0) {
            *reinterpret_cast<uint16_t *>(row + q4_v_unit(d, D)) = (uint16_t)((lane & 4) ? w >> 16 : w);
        }
        if (lane == 0)
            reinterpret_cast<uint16_t *>(s + a.block_size * q4_row_bytes(D))[off * ng + g] = sb;
    }
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs &a, bool q4, cudaStream_t stream) {
    if (a.num_tokens == 0) return cudaSuccess;
    const dim3 grid(a.num_tokens), block(kThreads);
    if (a.dtype == PA_DTYPE_BF16)
        return q4 ? launch_dependent(rope_cache_kernel<__nv_bfloat16, true>, grid, block, 0, stream, a)
                  : launch_dependent(rope_cache_kernel<__nv_bfloat16, false>, grid, block, 0, stream, a);
    return q4 ? launch_dependent(rope_cache_kernel<float, true>, grid, block, 0, stream, a)
              : launch_dependent(rope_cache_kernel<float, false>, grid, block, 0, stream, a);
}

}  // namespace pa
