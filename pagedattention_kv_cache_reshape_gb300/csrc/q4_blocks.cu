// q4_blocks.cu -- whole cache blocks between the 16/32-bit pools and the 4-bit
// pools (q4_format.cuh), along a list of (source, destination) block pairs.
//  quantize:   a prompt prefilled in a bf16 pool goes over to the 4-bit pool
//              its decode steps read;
//  dequantize: a cached 4-bit prefix is expanded for a prefill over it.
// Both move (e + 9/16) bytes a value (e = 2 or 4) and are bound by HBM.  A thread
// takes 8 consecutive dims of a token row (16 or 32 bytes of the wide pool, 4
// of the codes), a warp 256 dims: whole 128-byte lines of codes, and rows of
// the wide pool in pieces of D e bytes.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;   // loads in flight a thread

// grid: (pair, part of the block).  Items of a block: [K, V][head][token][8 dims].
template <typename T, int D, bool kQuantize>
__global__ void __launch_bounds__(kThreads) q4_convert_kernel(const Q4BlocksArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int i = blockIdx.x;
    const int32_t src = __ldg(a.pairs + 2 * (int64_t)i), dst = __ldg(a.pairs + 2 * (int64_t)i + 1);
    if (src < 0 || dst < 0) return;
    if (src >= a.src_num_blocks || dst >= a.dst_num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
        return;
    }
    constexpr int kRow = D / 8, NG = D / kQ4Group;   // threads and groups of a row
    const int B = a.block_size, H = a.num_kv_heads, half = H * B * kRow;
    const int64_t slab = q4_slab_bytes(B, D);
    const int64_t wide_blk = (int64_t)(kQuantize ? src : dst) * B * H * D, q4_blk = (kQuantize ? dst : src) * H * slab;
    const T *wide_k = static_cast<const T *>(kQuantize ? a.src_k : a.dst_k) + wide_blk;
    const T *wide_v = static_cast<const T *>(kQuantize ? a.src_v : a.dst_v) + wide_blk;
    const uint8_t *q4_k = static_cast<const uint8_t *>(kQuantize ? a.dst_k : a.src_k) + q4_blk;
    const uint8_t *q4_v = static_cast<const uint8_t *>(kQuantize ? a.dst_v : a.src_v) + q4_blk;
    const int first = blockIdx.y * kThreads * kPerThread + threadIdx.x;
    // half is a multiple of 32 (B * D / 8 is one of 64): a warp's items are all of K, all of V or all outside
    float x[kPerThread][8];
    uint32_t w[kPerThread];
    uint16_t sb[kPerThread];
    auto place = [&](int u, bool &is_v, int &k, int64_t &wide, int64_t &row, int64_t &scale) {
        int e = first + u * kThreads;
        const bool in = e < 2 * half;
        if (!in) e = 0;
        is_v = e >= half;
        if (is_v) e -= half;
        k = e % kRow;
        const int t = e / kRow, tok = t % B, h = t / B;
        wide = ((int64_t)tok * H + h) * D + k * 8;
        row = h * slab + tok * (D / 2);
        scale = h * slab + B * (D / 2) + tok * (NG * 2);
        return in;
    };
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        bool is_v;
        int k;
        int64_t wide, row, scale;
        if (!place(u, is_v, k, wide, row, scale)) continue;
        if (kQuantize) {
            load8(x[u], (is_v ? wide_v : wide_k) + wide);
        } else {
            const uint8_t *p = is_v ? q4_v : q4_k;
            const int g = k / 4, r = 2 * (k & 3) + (g & 1);
            w[u] = *reinterpret_cast<const uint32_t *>(p + row + (is_v ? (r * NG + (g & ~1)) * 2 : q4_k_word(8 * k, D)));
            sb[u] = *reinterpret_cast<const uint16_t *>(p + scale + 2 * g);
        }
    }
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        bool is_v;
        int k;
        int64_t wide, row, scale;
        if (!place(u, is_v, k, wide, row, scale)) continue;   // whole warps
        if (kQuantize) {
            uint8_t *p = const_cast<uint8_t *>(is_v ? q4_v : q4_k);
            q4_store8<D>(x[u], k, is_v, p + row, reinterpret_cast<uint16_t *>(p + scale), true);
        } else {
            const int g = k / 4;
            if (is_v) {   // (r, g), (r, g + 1) against the neighbour group's (r + 1, g), (r + 1, g + 1)
                const uint32_t other = __shfl_xor_sync(0xffffffffu, w[u], 4);
                w[u] = g & 1 ? __byte_perm(other, w[u], 0x7632) : __byte_perm(w[u], other, 0x5410);
            }
            const float s = q4_scale_value(sb[u]);
            float y[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) y[n] = (float)((int)((w[u] >> (4 * n)) & 15u) - 8) * s;
            store8(const_cast<T *>(is_v ? wide_v : wide_k) + wide, y);
        }
    }
}

template <typename T, int D>
cudaError_t launch_typed(const Q4BlocksArgs &a, bool quantize, cudaStream_t stream) {
    const int64_t items = (int64_t)2 * a.num_kv_heads * a.block_size * (D / 8);
    const int64_t parts = (items + kThreads * kPerThread - 1) / (kThreads * kPerThread);
    if (parts > 65535) return cudaErrorNotSupported;
    const dim3 grid(a.num_pairs, (unsigned)parts), block(kThreads);
    return quantize ? launch_dependent(q4_convert_kernel<T, D, true>, grid, block, 0, stream, a)
                    : launch_dependent(q4_convert_kernel<T, D, false>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_q4_blocks(const Q4BlocksArgs &a, bool quantize, cudaStream_t stream) {
    if (a.num_pairs == 0) return cudaSuccess;
    if (a.dtype == PA_DTYPE_BF16)
        return a.head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(a, quantize, stream)
                                 : launch_typed<__nv_bfloat16, 64>(a, quantize, stream);
    return a.head_dim == 128 ? launch_typed<float, 128>(a, quantize, stream)
                             : launch_typed<float, 64>(a, quantize, stream);
}

}  // namespace pa
