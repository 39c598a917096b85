// attn_decode_q4.cu -- paged decode attention over 4-bit pools (q4_format.cuh):
//     out[s][h] = sum_j softmax_j(scale <q[s][h], K_s[j][g]>) V_s[j][g]
// with K and V the values their codes and scales stand for.
#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

// One CTA per (sequence, q-head); warp w takes tokens w, w + 4, ...; a lane
// holds D/32 dims (dim 32 g + lane).
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_q4_kernel(const AttnArgs a) {
    constexpr int NG = D / kQ4Group;
    __shared__ float o_s[kWarps][D], m_s[kWarps], l_s[kWarps];
    grid_dependency_wait();
    grid_dependents_launch();
    const int s = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = a.block_size, H = a.num_kv_heads, hk = h / (a.num_heads / H);
    const int ctx = a.context_lens[s];
    if (ctx <= 0 || (int64_t)ctx > (int64_t)a.max_blocks * B) {
        if (threadIdx.x == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const int64_t slab = q4_slab_bytes(B, D);
    const int64_t qo = ((int64_t)s * a.num_heads + h) * D;
    float q[NG], o[NG], m = -INFINITY, l = 0.0f;
    for (int g = 0; g < NG; ++g) {
        q[g] = to_float(static_cast<const T *>(a.q)[qo + 32 * g + lane]) * a.scale;
        o[g] = 0.0f;
    }
    for (int j = warp; j < ctx; j += kWarps) {
        const int32_t blk = a.block_tables[(int64_t)s * a.max_blocks + j / B];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
            continue;
        }
        const int tok = j % B;
        const int64_t at = ((int64_t)blk * H + hk) * slab;
        const uint8_t *ks = static_cast<const uint8_t *>(a.k_cache) + at;
        const uint8_t *vs = static_cast<const uint8_t *>(a.v_cache) + at;
        float x = 0.0f, v[NG];
        for (int g = 0; g < NG; ++g) {
            const int d = 32 * g + lane;
            const float ksc = q4_scale_value(reinterpret_cast<const uint16_t *>(ks + B * (D / 2))[tok * NG + g]);
            const float vsc = q4_scale_value(reinterpret_cast<const uint16_t *>(vs + B * (D / 2))[tok * NG + g]);
            const int kn = (ks[tok * (D / 2) + q4_k_word(d & ~7, D) + ((d & 7) >> 1)] >> (4 * (d & 1))) & 15;
            const int vn = (vs[tok * (D / 2) + q4_v_unit(d & ~3, D) + ((d & 3) >> 1)] >> (4 * (d & 1))) & 15;
            x += q[g] * ((kn - 8) * ksc);
            v[g] = (vn - 8) * vsc;
        }
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const float mn = fmaxf(m, x), alpha = expf(m - mn), p = expf(x - mn);
        l = l * alpha + p;
        for (int g = 0; g < NG; ++g) o[g] = o[g] * alpha + p * v[g];
        m = mn;
    }
    for (int g = 0; g < NG; ++g) o_s[warp][32 * g + lane] = o[g];
    if (lane == 0) { m_s[warp] = m; l_s[warp] = l; }
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w]);
    for (int w = 0; w < kWarps; ++w) L += m_s[w] == -INFINITY ? 0.0f : l_s[w] * expf(m_s[w] - M);
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float r = 0.0f;
        for (int w = 0; w < kWarps; ++w) r += m_s[w] == -INFINITY ? 0.0f : o_s[w][d] * expf(m_s[w] - M);
        static_cast<T *>(a.out)[qo + d] = from_float<T>(r / L);
    }
}

}  // namespace

size_t decode_q4_workspace(int, int, int, int) { return 256; }

cudaError_t launch_decode_q4(const AttnArgs &a, void *, size_t, cudaStream_t stream) {
    const dim3 grid(a.num_seqs, a.num_heads), block(kWarps * 32);
    if (a.dtype == PA_DTYPE_BF16)
        return a.head_dim == 128 ? launch_dependent(decode_q4_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, a)
                                 : launch_dependent(decode_q4_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, a);
    return a.head_dim == 128 ? launch_dependent(decode_q4_kernel<float, 128>, grid, block, 0, stream, a)
                             : launch_dependent(decode_q4_kernel<float, 64>, grid, block, 0, stream, a);
}

}  // namespace pa
