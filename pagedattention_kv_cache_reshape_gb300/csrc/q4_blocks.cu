// q4_blocks.cu -- whole cache blocks between the 16/32-bit pools and the 4-bit
// pools (q4_format.cuh), along a list of (source, destination) block pairs.
//  quantize:   a prompt prefilled in a bf16 pool goes over to the 4-bit pool
//              its decode steps read;
//  dequantize: a cached 4-bit prefix is expanded for a prefill over it.
// Both move (e + 9/16) bytes a value (e = 2 or 4): HBM is the bound, with the
// instruction issue close behind.  A thread takes 16 (quantize)
// or 8 consecutive dims of a token row, a warp whole lines of the codes, and
// rows of the wide pool in pieces of D e bytes.
// Measured: 2048 pairs of 16 tokens x 8 heads x 128 bf16 (172 MB each way) there
// and back 62.4 us, 5.5 TB/s; each alone from cold caches, quantizing takes 38.4 us
// at 70 % of the issue slots and dequantizing 28.5 us at 77 %.  Five CTAs an SM (62.3 us) beat
// four (65.6), eight items a thread 61.8 but slow small calls (256 blocks 9.2
// against 7.8 us with the append before them).
#include "pa_device.cuh"
#include "pa_internal.h"
#include "q4_format.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;   // loads in flight a thread

// (n - 8) s of a word's 8 nibbles, rounded once.  bf16: 0x4300 | n is 128 + n, and the difference and the product
// of 4 by 8 bits come out of packed bf16 instructions as if rounded from exact.
__device__ __forceinline__ void expand8(__nv_bfloat16 *dst, uint32_t w, uint16_t scale) {
    const uint32_t ss = (uint32_t)scale * 0x10001u;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // nibbles i and i + 4
        uint32_t t;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(t) : "r"(w >> (4 * i)), "r"(0x43004300u));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(t) : "r"(t), "r"(0x43084308u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(t), "r"(ss));
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                                 __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}
__device__ __forceinline__ void expand8(float *dst, uint32_t w, uint16_t scale) {
    const float s = q4_scale_value(scale);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = (__uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u) - (8388608.0f + 8.0f)) * s;
    store_raw8(dst, from_floats<float>(y));
}

// grid: (pair, part of the block).  Items of a block: [K, V][head][token][16 or 8 dims].
template <typename T, int D, bool kQuantize>
__global__ void __launch_bounds__(kThreads, 5) q4_convert_kernel(const Q4BlocksArgs a, int log2b) {
    constexpr int kDims = kQuantize ? 16 : 8, kItems = kQuantize ? kPerThread / 2 : kPerThread;
    constexpr int kRow = D / kDims, NG = D / kQ4Group;   // threads and groups of a row
    const int H = a.num_kv_heads, half = (H * kRow) << log2b, slab = q4_slab_bytes(1 << log2b, D);
    grid_dependency_wait();
    grid_dependents_launch();
    const int i = blockIdx.x;
    const int32_t src = __ldg(a.pairs + 2 * (int64_t)i), dst = __ldg(a.pairs + 2 * (int64_t)i + 1);
    if (src < 0 || dst < 0) return;
    if (src >= a.src_num_blocks || dst >= a.dst_num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_status(a.status, PA_ERR_OUT_OF_RANGE);
        return;
    }
    const int64_t wide_blk = (int64_t)(kQuantize ? src : dst) * half * kDims;
    const int64_t q4_blk = (int64_t)(kQuantize ? dst : src) * H * slab;
    // the thread's place in a row is the same for all its items; half is a multiple of 32 (B * D / 16 is one), so
    // a warp's items are all of K, all of V or all outside
    const int k = threadIdx.x % kRow, g = k / 4, r = 2 * (k & 3) + (g & 1);   // (g, r: of 8 dims)
    const int first = blockIdx.y * kThreads * kItems + threadIdx.x;
    Raw8<T> lo[kQuantize ? kItems : 1], hi[kQuantize ? kItems : 1];
    uint32_t w[kItems];
    uint16_t sb[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const int e = first + u * kThreads;
        if (e >= 2 * half) break;
        const bool is_v = e >= half;
        const int t = (is_v ? e - half : e) / kRow, tok = t & ((1 << log2b) - 1), h = t >> log2b;
        if constexpr (kQuantize) {
            const T *p = static_cast<const T *>(is_v ? a.src_v : a.src_k) + wide_blk + (tok * H + h) * D + k * 16;
            lo[u] = load_raw8(p);
            hi[u] = load_raw8(p + 8);
        } else {
            const uint8_t *p = static_cast<const uint8_t *>(is_v ? a.src_v : a.src_k) + q4_blk + h * slab;
            w[u] = *reinterpret_cast<const uint32_t *>(p + tok * (D / 2) + (is_v ? (r * NG + (g & ~1)) * 2 : q4_k_word(8 * k, D)));
            sb[u] = *reinterpret_cast<const uint16_t *>(p + ((D / 2) << log2b) + tok * (NG * 2) + 2 * g);
        }
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const int e = first + u * kThreads;
        if (e >= 2 * half) break;
        const bool is_v = e >= half;
        const int t = (is_v ? e - half : e) / kRow, tok = t & ((1 << log2b) - 1), h = t >> log2b;
        if constexpr (kQuantize) {
            uint8_t *p = static_cast<uint8_t *>(is_v ? a.dst_v : a.dst_k) + q4_blk + h * slab;
            q4_store16<D>(lo[u], hi[u], k, is_v, p + tok * (D / 2),
                          reinterpret_cast<uint16_t *>(p + ((D / 2) << log2b) + tok * (NG * 2)), true);
        } else {
            if (is_v) {   // (r, g), (r, g + 1) against the neighbour group's (r + 1, g), (r + 1, g + 1)
                const uint32_t other = __shfl_xor_sync(0xffffffffu, w[u], 4);
                w[u] = g & 1 ? __byte_perm(other, w[u], 0x7632) : __byte_perm(w[u], other, 0x5410);
            }
            expand8(static_cast<T *>(is_v ? a.dst_v : a.dst_k) + wide_blk + (tok * H + h) * D + k * 8, w[u], sb[u]);
        }
    }
}

template <typename T, int D>
cudaError_t launch_typed(const Q4BlocksArgs &a, bool quantize, cudaStream_t stream) {
    const int64_t items = (int64_t)2 * a.num_kv_heads * a.block_size * (D / 8);
    const int64_t parts = (items + kThreads * kPerThread - 1) / (kThreads * kPerThread);
    if (parts > 65535 || items * 8 > INT32_MAX) return cudaErrorNotSupported;
    const int log2b = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    const dim3 grid(a.num_pairs, (unsigned)parts), block(kThreads);
    return quantize ? launch_dependent(q4_convert_kernel<T, D, true>, grid, block, 0, stream, a, log2b)
                    : launch_dependent(q4_convert_kernel<T, D, false>, grid, block, 0, stream, a, log2b);
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
