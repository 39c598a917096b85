// q4_format.cuh -- the 4-bit cache row format, shared by the kernels that write
// it (rope_cache.cu, q4_blocks.cu) and read it (q4_blocks.cu, attn_decode_q4.cu).
//
// A pool holds [num_blocks][num_kv_heads] slabs.  A slab is one block of one
// kv-head: B token rows of D / 2 code bytes, then B rows of D / 32 bf16
// scales (9 bits per two values: 4.5 bits a value).  A group is 32 consecutive
// dims of one row; with amax = max |x| over the group,
//     s = bf16(amax fp32(1/7)),  n = 8 + clamp(rint(x / s), -7, 7),  value (n - 8) s.
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

// Bits of the scale of a group from the bits of its largest magnitude.  NaN and
// infinities have the largest bit patterns, so a group that holds one is found
// by the same integer maximum; it takes a NaN scale and reads back as NaN.
__device__ __forceinline__ uint16_t q4_scale_bits(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 0x7fc0u;
    return __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(__uint_as_float(amax_bits), 1.0f / 7.0f)));
}
__device__ __forceinline__ float q4_scale_value(uint16_t bits) {
    return __uint_as_float((uint32_t)bits << 16);
}

// The word of 8 values' nibbles (x[0] lowest) in a group of scale s.
// The quotient x / s is the correctly rounded one, by Markstein's correction
// of x r, r the correctly rounded 1 / s, with the exact remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990); the range of s keeps the remainders of quotients from 1/4 up normal,
// and smaller quotients round to 0 either way.  Adding 1.5 2^23 + 8 rounds a
// quotient to the nearest integer, ties to even, with n + 8 in the low bits;
// |x / s| <= 7 (1 + 2^-8) there, so no clamp is needed.
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], float s) {
    constexpr float kRound = 12582912.0f + 8.0f;
    uint32_t w = 0;
    if (s >= 0x1p-90f && s <= 0x1p90f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float q0 = __fmul_rn(x[i], r);
            const float q = __fmaf_rn(__fmaf_rn(-q0, s, x[i]), r, q0);
            w = w * 16u + __float_as_uint(__fadd_rn(q, kRound));
        }
        // the eight sums carry the exponent field of 1.5 2^23 each: 0x4b400000 (1 + 16 + ... + 16^7) mod 2^32
        return w - 0x3f400000u;
    }
    if (!(s > 0.0f)) return 0x88888888u;   // 0 or NaN
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float n = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.0f), 7.0f);
        w = w * 16u + (uint32_t)((int)n + 8);
    }
    return w;
}

// 8 consecutive values of a row as they lie in memory (16-byte aligned), and as fp32.
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };
template <typename T> __device__ __forceinline__ Raw8<T> load_raw8(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = *(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
__device__ __forceinline__ void to_floats(float (&x)[8], const Raw8<__nv_bfloat16> &r) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(float (&x)[8], const Raw8<float> &r) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
// Bits of the largest magnitude of 8 values, as fp32.
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<__nv_bfloat16> &r) {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(r.v[0].x & m, r.v[0].y & m), __vmaxu2(r.v[0].z & m, r.v[0].w & m));
    return max(t << 16, t & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<float> &r) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = r.v[i];
        a = max(a, max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu)));
    }
    return a;
}
template <typename T> __device__ __forceinline__ Raw8<T> from_floats(const float (&x)[8]);
template <> __device__ __forceinline__ Raw8<__nv_bfloat16> from_floats<__nv_bfloat16>(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return {{make_uint4(w[0], w[1], w[2], w[3])}};
}
template <> __device__ __forceinline__ Raw8<float> from_floats<float>(const float (&x)[8]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    return {{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])}};
}
template <typename T> __device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) *(reinterpret_cast<uint4 *>(p) + i) = r.v[i];
}

// Quantises 16 values, dims 16 k .. 16 k + 15 of a token row (half a group), and
// stores them: called by whole warps in which the D / 16 lanes of a row are
// neighbours in order of k, a row's first lane a multiple of D / 16.  `row` is
// the row's code bytes and `scales` its scales; lanes with store = false only
// take part in the shuffles.
template <int D, typename T>
__device__ __forceinline__ void q4_store16(const Raw8<T> &lo, const Raw8<T> &hi, int k, bool is_v, uint8_t *row,
                                           uint16_t *scales, bool store) {
    constexpr int NG = D / kQ4Group;
    uint32_t amax = max(amax_bits8(lo), amax_bits8(hi));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const uint16_t sb = q4_scale_bits(amax);
    const float s = q4_scale_value(sb);
    const int g = k >> 1, h = k & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x[8];
        to_floats(x, i ? hi : lo);
        const uint32_t w = q4_word(x, s);
        // V: a word holds units r = 4 h + 2 i and r + 1 of group g; with its neighbour group's lane the lane makes
        // the 4 bytes (r, g), (r, g + 1) or (r + 1, g - 1), (r + 1, g)
        const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 2);
        if (!store) continue;
        if (is_v) {
            const uint32_t pair = g & 1 ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
            *reinterpret_cast<uint32_t *>(row + ((4 * h + 2 * i + (g & 1)) * NG + (g & ~1)) * 2) = pair;
        } else {
            *reinterpret_cast<uint32_t *>(row + ((2 * h + i) * NG + g) * 4) = w;
        }
    }
    if (store && h == 0) scales[g] = sb;
}

// The same for the 8 values from dim 8 j and the 8 from D / 2 + 8 j, j the lane's
// place among the D / 16 of its row (what a rotation of halves leaves a lane).
template <int D, typename T>
__device__ __forceinline__ void q4_store8x2(const Raw8<T> &lo, const Raw8<T> &hi, int j, bool is_v, uint8_t *row,
                                            uint16_t *scales, bool store) {
    constexpr int NG = D / kQ4Group;
    uint32_t w[2];
    uint16_t sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t amax = amax_bits8(i ? hi : lo);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        sb[i] = q4_scale_bits(amax);
        float x[8];
        to_floats(x, i ? hi : lo);
        w[i] = q4_word(x, q4_scale_value(sb[i]));
    }
    const int c = j & 3, g = j >> 2;   // g: 0 or 1 of the row's half (head_dim 64: 0)
    // (a warp may hold rows of K and of V: every lane takes part in the exchange)
    const uint32_t o0 = __shfl_xor_sync(0xffffffffu, w[0], 4), o1 = __shfl_xor_sync(0xffffffffu, w[1], 4);
    if (is_v && NG == 4) {             // units r = 2 c (g = 0) or 2 c + 1 of all four groups: 8 bytes
        const uint2 v = g ? make_uint2(__byte_perm(o0, w[0], 0x7632), __byte_perm(o1, w[1], 0x7632))
                          : make_uint2(__byte_perm(w[0], o0, 0x5410), __byte_perm(w[1], o1, 0x5410));
        if (store) *reinterpret_cast<uint2 *>(row + (2 * c + g) * 8) = v;
    } else if (is_v) {                 // units 2 c and 2 c + 1 of both groups: 8 bytes
        if (store)
            *reinterpret_cast<uint2 *>(row + c * 8) = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
    } else if (store) {
        *reinterpret_cast<uint32_t *>(row + (c * NG + g) * 4) = w[0];
        *reinterpret_cast<uint32_t *>(row + (c * NG + NG / 2 + g) * 4) = w[1];
    }
    if (store && c == 0) {
        scales[g] = sb[0];
        scales[NG / 2 + g] = sb[1];
    }
}

}  // namespace pa
