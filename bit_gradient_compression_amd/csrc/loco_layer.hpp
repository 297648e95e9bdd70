// Device helpers of the layer operators (layer norm, activation checkpoints, matrix
// products): chunks of eight consecutive elements, activations and their slopes, and the
// 8-bit checkpoint's arithmetic.
#pragma once

#include "loco_device.hpp"

namespace loco {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- chunks of eight elements ------------------------------------------------------
//
// Rows of an odd width start at any multiple of the element size, so chunks are moved with
// 16-byte accesses that promise only the element's alignment: on gfx950 that is the same
// instruction as an aligned access, and an aligned address runs at full speed.  The last
// chunk of a row may hold fewer than eight elements (`valid`) and goes element by element.

__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// Streaming stores, for what is not read again soon: they leave the caches to what is.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
__device__ __forceinline__ void stream16(void* p, u32x4 v) { __builtin_nontemporal_store(v, (u32x4_any*)p); }
__device__ __forceinline__ void stream8(void* p, u32x2 v) { __builtin_nontemporal_store(v, (u32x2_any*)p); }

__device__ __forceinline__ void unpack_bf16x8(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ u32x4 pack_bf16x8(const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // one v_cvt_pk_bf16_f32 each
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2 * i], v[2 * i + 1]}), bf16x2));
    return w;
}

// p points at the chunk's first element; elements at and past `valid` read as 0.
__device__ __forceinline__ void load_chunk(const uint16_t* p, int valid, float (&v)[8]) {
    if (valid >= 8) {
        unpack_bf16x8(load16(p), v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f;
    }
}
__device__ __forceinline__ void load_chunk(const float* p, int valid, float (&v)[8]) {
    if (valid >= 8) {
        const u32x4 a = load16(p), b = load16(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void store_chunk(uint16_t* p, int valid, const float (&v)[8]) {
    if (valid >= 8) {
        store16(p, pack_bf16x8(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = bf16_rne(v[i]);
    }
}
__device__ __forceinline__ void store_chunk(float* p, int valid, const float (&v)[8]) {
    if (valid >= 8) {
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(v[i]);
            b[i] = __float_as_uint(v[4 + i]);
        }
        store16(p, a);
        store16(p + 4, b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = v[i];
    }
}

// A chunk as it lies in memory: half the registers of its values for bf16.
template <typename T>
struct RawChunk;
template <>
struct RawChunk<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t* p, int valid) {
        if (valid >= 8) {
            w = load16(p);
        } else {
            w = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_bf16x8(w, v); }
};
template <>
struct RawChunk<float> {
    float w[8];
    __device__ __forceinline__ void load(const float* p, int valid) { load_chunk(p, valid, w); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i];
    }
};

// A chunk of a buffer whose type is known at run time only (wave-uniform branch).
__device__ __forceinline__ void load_chunk_any(const void* base, bool f32, int64_t at, int valid, float (&v)[8]) {
    if (f32) load_chunk((const float*)base + at, valid, v);
    else load_chunk((const uint16_t*)base + at, valid, v);
}
__device__ __forceinline__ void store_chunk_any(void* base, bool f32, int64_t at, int valid, const float (&v)[8]) {
    if (f32) store_chunk((float*)base + at, valid, v);
    else store_chunk((uint16_t*)base + at, valid, v);
}

// ---- activations --------------------------------------------------------------------

// 1 / (1 + exp(-x)): the hardware's base-2 exponential and reciprocal, each within one
// unit in the last place.  Below x = -80 both are taken at 2^-32 of their arguments: they flush
// subnormal results to 0, which would lose z * sigmoid(z) from z = -87 on, where it is still
// 1e-36.  Nearer to 0 that shift would cost what the exponent's argument loses beside 32 (2^-19,
// a relative error of 7e-7 of the activation instead of 1.4e-7).
__device__ __forceinline__ float sigmoid(float x) {
    const bool far = x < -80.0f;
    const float one = far ? 0x1p-32f : 1.0f;
    const float t = __builtin_amdgcn_exp2f(__builtin_fmaf(x, -1.4426950408889634f, far ? -32.0f : 0.0f));
    return __builtin_amdgcn_rcpf(one + t) * one;
}

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == 1) return z < 0.0f ? 0.0f : z;  // a NaN stays one
    else if constexpr (ACT == 2)
        return z * sigmoid(z * __builtin_fmaf(kGelu2C * kGeluA * z, z, kGelu2C));
    else if constexpr (ACT == 3) return z * sigmoid(z);
    else return z;
}

// s = sigmoid(x) and q = 1 - s, each with its own relative accuracy (1 - s formed by subtraction
// loses it where s is near 1): with u = exp(-|x|) the larger of them is 1 / (1 + u) and the smaller
// u times that.  Nothing overflows, past |x| = 87 the smaller is 0, however large a factor z it
// meets, and a NaN is in both: no minimum or clamp, which would drop it, touches x.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& q) {
    const float u = __builtin_amdgcn_exp2f(__builtin_fabsf(x) * -1.4426950408889634f);
    const float large = __builtin_amdgcn_rcpf(1.0f + u), small = u * large;
    s = x < 0.0f ? small : large;
    q = x < 0.0f ? large : small;
}

// The derivative of act_value.  GELU's second term is 0 in fp32 past |z| = 16, where its factors
// overflow, so it takes z held within that (the clamp turns a NaN into a number); a NaN reaches the
// result through s.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == 1) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    else if constexpr (ACT == 2) {
        float s, q;
        sigmoid_pair(z * __builtin_fmaf(kGelu2C * kGeluA * z, z, kGelu2C), s, q);
        const float c = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);
        return __builtin_fmaf(c * (s * q), __builtin_fmaf(3.0f * kGelu2C * kGeluA * c, c, kGelu2C), s);
    } else if constexpr (ACT == 3) {
        float s, q;
        sigmoid_pair(z, s, q);
        return __builtin_fmaf(z, s * q, s);
    } else
        return 1.0f;
}

template <int ACT>
__device__ __forceinline__ void act_chunk(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value<ACT>(v[i]);
}
__device__ __forceinline__ void act_chunk_any(int act, float (&v)[8]) {
    if (act == 1) act_chunk<1>(v);
    else if (act == 2) act_chunk<2>(v);
    else if (act == 3) act_chunk<3>(v);
}
template <int ACT>
__device__ __forceinline__ void slope_chunk(const float (&z)[8], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= act_slope<ACT>(z[i]);
}
__device__ __forceinline__ void slope_chunk_any(int act, const float (&z)[8], float (&v)[8]) {
    if (act == 1) slope_chunk<1>(z, v);
    else if (act == 2) slope_chunk<2>(z, v);
    else if (act == 3) slope_chunk<3>(z, v);
}

// ---- the 8-bit checkpoint -----------------------------------------------------------
//
// A block of 32 or 64 consecutive elements of a row has one step, a power of two: the least
// 2^s >= 2^-126 with max|x| < 127.5 * 2^s.  Codes are q = rint(x / 2^s), ties to even, in
// [-127, 127], and the block's byte holds s + 127.  x * 2^-s is exact, so each code has one
// rounding; and q * 2^s has at most 7 significant bits, so it is a bf16 number: the matrix
// cores read a checkpoint without rounding it again.  A block that holds an infinity or a
// NaN gets the byte 255 and codes 0, which read back as 0 * inf = NaN.

// The block's byte from the largest |x| of the block, as a bit pattern.  127.5 * 2^s is the
// pattern of 1.9921875 * 2^(s+6): adding 2^16 carries into the exponent from there on.
__device__ __forceinline__ uint32_t ckpt_exp(uint32_t top) {
    const uint32_t e = (top + 0x10000u) >> 23;
    return top >= 0x7f800000u ? 255u : max(e, 7u) - 6u;
}
// 2^-s and 2^s of the byte; 0 and inf for 255 (codes 0 and values NaN).
__device__ __forceinline__ float ckpt_inv(uint32_t e) { return e == 255u ? 0.0f : __uint_as_float((254u - e) << 23); }
__device__ __forceinline__ float ckpt_step(uint32_t e) { return __uint_as_float(e << 23); }

// Largest |v| of the block that this lane's chunk belongs to: blocks are aligned groups of
// 4 (32 elements) or 8 lanes.  All 64 lanes take part.
__device__ __forceinline__ uint32_t block_top(const float (&v)[8], bool block64) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = group_max_u32<4>(m);
    return block64 ? max(m, dpp<0x141>(m)) : m;  // row_half_mirror: the other four lanes of eight
}

// The chunk's eight code bytes.  A block with an infinity or NaN has codes 0: inf * 0 is NaN,
// so they are cleared by the byte and not by the product.
__device__ __forceinline__ u32x2 ckpt_codes(const float (&v)[8], uint32_t e) {
    const float inv = ckpt_inv(e);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __builtin_rintf(v[i] * inv);
    uint32_t lo, hi;
    pack_codes8<8>(q, lo, hi);
    if (e == 255u) lo = hi = 0u;
    return u32x2{lo, hi};
}

// Codes are read in the backward pass, long after they are written: their stores stream.
__device__ __forceinline__ void store_codes(int8_t* p, int valid, u32x2 w) {
    if (valid >= 8) {
        stream8(p, w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}
__device__ __forceinline__ u32x2 load_codes(const int8_t* p, int valid) {
    u32x2 w = {0u, 0u};
    if (valid >= 8) {
        __builtin_memcpy(&w, p, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    }
    return w;
}

// The values of eight codes, each exact.  For the byte 255 the step is inf and 0 * inf is NaN.
__device__ __forceinline__ void decode_codes(u32x2 w, uint32_t e, float (&v)[8]) {
    const float step = ckpt_step(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * step;
}

// ---- wave sums ----------------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
    v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

}  // namespace loco
