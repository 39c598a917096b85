// q4_format.cuh -- the 4-bit cache row format, shared by the kernels that write
// it (rope_cache.cu, q4_blocks.cu) and read it (q4_blocks.cu, attn_decode_q4.cu).
//
// A pool holds [num_blocks][num_kv_heads] slabs.  A slab is one block of one
// kv-head: B token rows of D / 2 code bytes, then B rows of D / 32 bf16
// scales (9 bits per two values: 4.5 bits a value).  A group is 32 consecutive
// dims of one row; with amax = max |x| over the group,
//     s = bf16(amax / 7),  n = 8 + clamp(rint(x / s), -7, 7),  value (n - 8) s.
// A token's bytes are its own (no byte is shared by two tokens), so tokens of
// one block can be written by different calls or threads.  A slab keeps one
// (block, head) contiguous: a decode warp reads it with full-line loads, and
// a block of a pool is one contiguous piece, as whole-block copies need.
//
// Inside a row the dims are laid out for the decode kernel's matrix fragments
// (m16n8k16, lane = 4 r + c), so that a lane's share of a row is contiguous:
//   K: lane c of a row's four reads word c of every group: the row is
//      [4 c][D/32 groups] words of 8 dims, dim 32 g + 8 c + n in nibble n;
//   V: lane r of a row's eight reads 4 dims of every group: the row is
//      [8 r][D/32 groups] 16-bit units, dim 32 g + 4 r + n in nibble n.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace pa {

constexpr int kQ4Group = 32;

__host__ __device__ constexpr int q4_row_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int q4_slab_bytes(int block_size, int d) {
    return block_size * (d / 2 + d / kQ4Group * 2);
}
// byte offset of 8 consecutive dims' word in a K row (dim a multiple of 8)
__host__ __device__ constexpr int q4_k_word(int dim, int d) {
    return (((dim % kQ4Group) / 8) * (d / kQ4Group) + dim / kQ4Group) * 4;
}
// byte offset of 4 consecutive dims' unit in a V row (dim a multiple of 4)
__host__ __device__ constexpr int q4_v_unit(int dim, int d) {
    return (((dim % kQ4Group) / 4) * (d / kQ4Group) + dim / kQ4Group) * 2;
}

// The scale of a group whose largest magnitude is amax, in bf16 bits.  A group
// with a NaN or an infinity (`finite` false) takes a NaN scale: all its values
// read back as NaN.
__device__ __forceinline__ uint16_t q4_scale_bits(float amax, bool finite) {
    if (!finite) return 0x7fc0u;
    return __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(amax, 7.0f)));
}
__device__ __forceinline__ float q4_scale_value(uint16_t bits) {
    return __uint_as_float((uint32_t)bits << 16);
}
// The nibble of x in a group of scale s (0 or NaN: every nibble 8).
__device__ __forceinline__ uint32_t q4_code(float x, float s) {
    if (!(s > 0.0f)) return 8u;
    const float n = fminf(fmaxf(rintf(__fdiv_rn(x, s)), -7.0f), 7.0f);
    return (uint32_t)((int)n + 8);
}

}  // namespace pa
