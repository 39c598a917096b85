// q4_blocks.cu -- whole cache blocks between the 16/32-bit pools and the 4-bit
// pools (q4_format.cuh), along a list of (source, destination) block pairs.
//  quantize:   a prompt prefilled in a bf16 pool goes over to the 4-bit pool
//              its decode steps read;
//  dequantize: a cached 4-bit prefix is expanded for a prefill over it.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

// A warp per (pair, K or V, token row, group): a lane per dim.
template <typename T, bool kQuantize>
__global__ void __launch_bounds__(kThreads) q4_convert_kernel(const Q4BlocksArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t src = a.pairs[2 * (int64_t)i], dst = a.pairs[2 * (int64_t)i + 1];
    if (src < 0 || dst < 0) return;
    if (src >= a.src_num_blocks || dst >= a.dst_num_blocks) {
        if (threadIdx.x == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const int D = a.head_dim, ng = D / kQ4Group, B = a.block_size, H = a.num_kv_heads;
    const int64_t slab = q4_slab_bytes(B, D);
    const int32_t wide_blk = kQuantize ? src : dst, q4_blk = kQuantize ? dst : src;
    for (int j = warp; j < 2 * H * B * ng; j += kThreads / 32) {
        int r = j;
        const int is_v = r & 1; r >>= 1;
        const int g = r % ng; r /= ng;
        const int h = r % H, tok = r / H;
        const int d = g * kQ4Group + lane;
        const int64_t wide = (((int64_t)wide_blk * B + tok) * H + h) * D + d;
        const int64_t s0 = ((int64_t)q4_blk * H + h) * slab;
        const int64_t at = s0 + tok * q4_row_bytes(D) +
                           (is_v ? q4_v_unit(d & ~3, D) + ((d & 3) >> 1) : q4_k_word(d & ~7, D) + ((d & 7) >> 1));
        const int64_t sc = s0 + B * q4_row_bytes(D) + 2 * (tok * ng + g);
        if (kQuantize) {
            const float x = to_float(static_cast<const T *>(is_v ? a.src_v : a.src_k)[wide]);
            float amax = fabsf(x);
            const bool finite = __all_sync(0xffffffffu, amax <= 3.402823466e38f);
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint16_t sb = q4_scale_bits(amax, finite);
            const uint32_t n = q4_code(x, q4_scale_value(sb));
            const uint32_t hi = __shfl_down_sync(0xffffffffu, n, 1);
            uint8_t *out = static_cast<uint8_t *>(is_v ? a.dst_v : a.dst_k);
            if ((lane & 1) == 0) out[at] = (uint8_t)(n | (hi << 4));
            if (lane == 0) *reinterpret_cast<uint16_t *>(out + sc) = sb;
        } else {
            const uint8_t *in = static_cast<const uint8_t *>(is_v ? a.src_v : a.src_k);
            const uint32_t n = (in[at] >> (4 * (lane & 1))) & 15u;
            const float s = q4_scale_value(*reinterpret_cast<const uint16_t *>(in + sc));
            static_cast<T *>(is_v ? a.dst_v : a.dst_k)[wide] = from_float<T>(((int)n - 8) * s);
        }
    }
}

}  // namespace

cudaError_t launch_q4_blocks(const Q4BlocksArgs &a, bool quantize, cudaStream_t stream) {
    if (a.num_pairs == 0) return cudaSuccess;
    const dim3 grid(a.num_pairs), block(kThreads);
    if (a.dtype == PA_DTYPE_BF16)
        return quantize ? launch_dependent(q4_convert_kernel<__nv_bfloat16, true>, grid, block, 0, stream, a)
                        : launch_dependent(q4_convert_kernel<__nv_bfloat16, false>, grid, block, 0, stream, a);
    return quantize ? launch_dependent(q4_convert_kernel<float, true>, grid, block, 0, stream, a)
                    : launch_dependent(q4_convert_kernel<float, false>, grid, block, 0, stream, a);
}

}  // namespace pa
