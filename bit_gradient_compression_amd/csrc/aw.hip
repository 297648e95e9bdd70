// AdamW over many tensors at once, with states in fp32 or in 8 bits.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) * (m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// in that order of IEEE fp32 operations, so that any elementwise form of it has the same bits.
//
// In 8 bits, a block of B elements shares a power of two.  m is a float8 (4 exponent bits, 3
// mantissa bits) times 2^s, the least that keeps the block's largest |m| within 448.  v, which is
// never negative, spends the sign's bit on its exponent: 5 bits of it, counted down from the
// block's largest, and 3 mantissa bits.  Both have four significant bits (an error of at most 2^-4);
// m reaches 2^-17 of the block's largest, v 2^-31, and a v that is not 0 never becomes 0: under
// it m would be divided by eps alone.  The weights' update takes the new m and v before they are
// rounded.
//
// A step changes v by (1 - b2) of itself or so, which is less than half a step of its code as soon as
// 1 - b2 is below 1/18: rounded to nearest, v stays where it is for good, and so does a small m beside a large
// one.  Rounded up with the probability of the dropped part (RANDOM), a state is its average in the mean at
// any b1 and b2.  The random bits are a hash of the call's key and the element's position.
//
// Bound by HBM: every byte is moved once, 28 per element with fp32 weights and states, bf16 gradients and a bf16
// copy, 16 with 8-bit states.  One LLaMA-7B layer (202 million elements) takes 906 - 1025 us
// (6.3 - 5.5 TB/s, from one card to the next) and 523 us (6.2 TB/s, at 89 instructions per element), 547 with random
// rounding.  200 tensors of 100 to 40000 elements take 9 us in either.

#include "loco_device.hpp"
#include "loco_step_internal.hpp"

namespace loco {
namespace {

enum : int { kF32 = 0, kBF16 = 1 };

// ---- 8-bit states -----------------------------------------------------------------------
//
// Exponent bytes are biased by 127; 255 marks a block with a value that is not finite (codes 0),
// which reads as NaN.

// m: the byte of 2^s from the pattern of the block's largest |m|.  448 2^s is the pattern of
// 1.75 * 2^(s + 8): adding 0x1fffff carries into the exponent just past it.  s >= -117, so that
// the smallest code, 2^-9, is a normal number.
__device__ __forceinline__ uint32_t m_exp(uint32_t top) {
    return top >= 0x7f800000u ? 255u : max((top + 0x1fffffu) >> 23, 18u) - 8u;
}
__device__ __forceinline__ float pow2_of(uint32_t e) { return __uint_as_float(e << 23); }  // 255: inf, 0: 0
__device__ __forceinline__ float m_inv(uint32_t e) { return __uint_as_float((254u - min(e, 253u)) << 23); }

__device__ __forceinline__ void m_decode4(uint32_t w, uint32_t e, float* x) {
    const float step = pow2_of(e);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = lo[0] * step;
    x[1] = lo[1] * step;
    x[2] = hi[0] * step;
    x[3] = hi[1] * step;
}
__device__ __forceinline__ uint32_t m_encode4(const float* x, uint32_t e) {
    const float inv = m_inv(e);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, w, true);
    return e == 255u ? 0u : (uint32_t)w;
}

// v: the byte of the block's exponent, that of its largest value rounded to four significant bits.
// At least 32: the smallest exponent, 31 below it, is a normal number's.
__device__ __forceinline__ uint32_t v_exp(uint32_t top) { return min(max((top + 0x80000u) >> 23, 32u), 255u); }
// Where values may be rounded up: that of the largest rounded up, so that the largest code is not a limit.
__device__ __forceinline__ uint32_t v_exp_up(uint32_t top) { return min(max((top + 0xfffffu) >> 23, 32u), 255u); }

__device__ __forceinline__ void v_decode4(uint32_t w, uint32_t e, float* x) {
    const uint32_t base = (max(e, 32u) - 31u) << 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t c = (w >> (8 * j)) & 255u;
        const float f = c ? __uint_as_float((c + base) << 20) : 0.0f;
        x[j] = e == 255u ? __builtin_nanf("") : f;
    }
}
__device__ __forceinline__ uint32_t v_encode4(const float* x, uint32_t e) {
    const int base = (int)(e - 31u) << 3;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t b = __float_as_uint(x[j]);
        const int r = (int)((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20);  // four significant bits, ties to even
        const uint32_t c = x[j] > 0.0f ? (uint32_t)min(max(r - base, 1), 255) : 0u;
        w |= c << (8 * j);
    }
    return e == 255u ? 0u : w;
}

// ---- random rounding ----------------------------------------------------------------------
//
// A code keeps the upper bits of a pattern; 20 random bits are added to the 20 that it drops, and carry with
// the probability that these are of a step.  What is a code's value already drops zeros and stays.

// 32 random bits of an element: two rounds of shifts and products, each half of the key before one.  All bits
// depend on all of the position's and the key's (the tests count them).
__device__ __forceinline__ uint32_t element_bits(uint32_t pos, uint32_t k0, uint32_t k1) {
    uint32_t x = pos ^ k0;
    x = (x ^ (x >> 16)) * 0x9E3779B9u;
    x = x ^ k1;
    x = (x ^ (x >> 15)) * 0xB504F335u;
    return x ^ (x >> 16);
}
// m takes the upper 20 of them, v the lower 20 in reverse: what they share are the lowest bits of both.
__device__ __forceinline__ uint32_t m_encode4_random(const float* x, uint32_t e, const uint32_t* bits) {
    const float inv = m_inv(e);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float y = __builtin_fabsf(x[j] * inv);
        // below 2^-6 codes are equidistant, as the values from 2^-6 to 2^-5 are
        const bool small = y < 0x1p-6f;
        const uint32_t b = __float_as_uint(small ? y + 0x1p-6f : y);
        const uint32_t c = ((b + (bits[j] >> 12)) >> 20) - (small ? 121u << 3 : 120u << 3);
        w |= (c | (__float_as_uint(x[j]) >> 24 & 128u)) << (8 * j);
    }
    return e == 255u ? 0u : w;
}
__device__ __forceinline__ uint32_t v_encode4_random(const float* x, uint32_t e, const uint32_t* bits) {
    const int base = (int)(e - 31u) << 3;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = (int)((__float_as_uint(x[j]) + (__builtin_bitreverse32(bits[j]) >> 12)) >> 20);
        const uint32_t c = x[j] > 0.0f ? (uint32_t)min(max(r - base, 1), 255) : 0u;
        w |= c << (8 * j);
    }
    return e == 255u ? 0u : w;
}

// ---- loads and stores of four elements, of which `valid` exist ----------------------------

template <int K>
__device__ __forceinline__ void load4(const void* p, int64_t i0, int valid, float* x) {
    if (valid >= 4) {
        if constexpr (K == kBF16) {
            const u32x2 w = __builtin_nontemporal_load((const u32x2*)((const uint16_t*)p + i0));
            x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
        } else {
            const f32x4 w = __builtin_nontemporal_load((const f32x4*)((const float*)p + i0));
            x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = 0.0f;
            if (j < valid) {
                if constexpr (K == kBF16) x[j] = __uint_as_float((uint32_t)((const uint16_t*)p)[i0 + j] << 16);
                else x[j] = ((const float*)p)[i0 + j];
            }
        }
    }
}
template <int K>
__device__ __forceinline__ void store4(void* p, int64_t i0, int valid, const float* x) {
    if (valid >= 4) {
        if constexpr (K == kBF16)
            __builtin_nontemporal_store(u32x2{bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3])},
                                        (u32x2*)((uint16_t*)p + i0));
        else __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, (f32x4*)((float*)p + i0));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < valid) {
                if constexpr (K == kBF16) ((uint16_t*)p)[i0 + j] = bf16_rne(x[j]);
                else ((float*)p)[i0 + j] = x[j];
            }
    }
}
__device__ __forceinline__ uint32_t load4b(const uint8_t* p, int64_t i0, int valid) {
    if (valid >= 4) return __builtin_nontemporal_load((const uint32_t*)(p + i0));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < valid) w |= (uint32_t)p[i0 + j] << (8 * j);
    return w;
}
__device__ __forceinline__ void store4b(uint8_t* p, int64_t i0, int valid, uint32_t w) {
    if (valid >= 4) {
        __builtin_nontemporal_store(w, (uint32_t*)(p + i0));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < valid) p[i0 + j] = (uint8_t)(w >> (8 * j));
    }
}
// Eight elements in two pieces of four: SPLIT, 256 apart; else consecutive ones, moved together.
template <int K, bool SPLIT>
__device__ __forceinline__ void load8(const void* p, const int64_t (&i0)[2], const int (&valid)[2], float (&x)[8]) {
    if constexpr (!SPLIT && K == kBF16) {
        if (valid[1] >= 4) {
            const u32x4 w = __builtin_nontemporal_load((const u32x4*)((const uint16_t*)p + i0[0]));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
            return;
        }
    }
    load4<K>(p, i0[0], valid[0], x);
    load4<K>(p, i0[1], valid[1], x + 4);
}
template <int K, bool SPLIT>
__device__ __forceinline__ void store8(void* p, const int64_t (&i0)[2], const int (&valid)[2], const float (&x)[8]) {
    if constexpr (!SPLIT && K == kBF16) {
        if (valid[1] >= 4) {
            __builtin_nontemporal_store(u32x4{bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3]), bf16x2_rne(x[4], x[5]),
                                              bf16x2_rne(x[6], x[7])}, (u32x4*)((uint16_t*)p + i0[0]));
            return;
        }
    }
    store4<K>(p, i0[0], valid[0], x);
    store4<K>(p, i0[1], valid[1], x + 4);
}
template <bool SPLIT>
__device__ __forceinline__ void load8b(const uint8_t* p, const int64_t (&i0)[2], const int (&valid)[2], uint32_t (&w)[2]) {
    if (!SPLIT && valid[1] >= 4) {
        const u32x2 v = __builtin_nontemporal_load((const u32x2*)(p + i0[0]));
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = load4b(p, i0[0], valid[0]);
        w[1] = load4b(p, i0[1], valid[1]);
    }
}
template <bool SPLIT>
__device__ __forceinline__ void store8b(uint8_t* p, const int64_t (&i0)[2], const int (&valid)[2], const uint32_t (&w)[2]) {
    if (!SPLIT && valid[1] >= 4) {
        __builtin_nontemporal_store(u32x2{w[0], w[1]}, (u32x2*)(p + i0[0]));
    } else {
        store4b(p, i0[0], valid[0], w[0]);
        store4b(p, i0[1], valid[1], w[1]);
    }
}

__device__ __forceinline__ int valid4(int64_t n, int64_t i0) {
    const int64_t left = n - i0;
    return left >= 4 ? 4 : left > 0 ? (int)left : 0;
}

// The largest |x| of each block, as a bit pattern, for two pieces of four elements per lane:
// SPLIT, at 4 lane and 256 + 4 lane of the tile; else the eight consecutive ones at 8 lane.
template <int B, bool SPLIT>
__device__ __forceinline__ void block_tops(const float (&x)[8], uint32_t (&top)[2]) {
    uint32_t t[2];
#pragma unroll
    for (int pc = 0; pc < 2; ++pc) {
        t[pc] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) t[pc] = max(t[pc], __float_as_uint(x[4 * pc + j]) & 0x7fffffffu);
    }
    if constexpr (SPLIT && B <= 256) {
        top[0] = group_max_u32<B / 4>(t[0]);
        top[1] = group_max_u32<B / 4>(t[1]);
    } else {
        top[0] = top[1] = group_max_u32<B / 8>(max(t[0], t[1]));
    }
}
template <bool SPLIT>
__device__ __forceinline__ int piece(int lane, int pc) {
    return SPLIT ? pc * 256 + lane * 4 : lane * 8 + pc * 4;
}

// The tensor of a tile: the last one whose first tile is not past it.  Every dependent load of the table costs
// a small call a microsecond, so up to 256 starts are counted at once; of more, every 64th part first.
__device__ __forceinline__ int64_t find_segment(const int64_t* tile0, int64_t n, int64_t tile, int lane) {
    int64_t lo = 0;
    while (n > 256) {
        const int64_t step = (n + 63) / 64, i = lane * step;
        const bool before = i < n && tile0[lo + (i < n ? i : 0)] <= tile;
        const int64_t j = uniform(__builtin_popcountll(ballot(before))) - 1;
        lo += j * step;
        n = n - j * step < step ? n - j * step : step;
    }
    int64_t first[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t i = k * 64 + lane;
        first[k] = k * 64 < n ? tile0[lo + (i < n ? i : 0)] : 0;
    }
    int count = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) count += __builtin_popcountll(ballot(k * 64 + lane < n && first[k] <= tile));
    return lo + uniform(count) - 1;
}
__device__ __forceinline__ const AwSegDev* segments(const void* table, int64_t n) {
    return (const AwSegDev*)((const char*)table + (n * 8 + 15) / 16 * 16);
}

__global__ __launch_bounds__(256) void aw_fill_kernel(const AwFillParams p) {
    // descriptions move as words: a lane's share of one of them
    constexpr int WORDS = sizeof(AwSegDev) / 4;
    uint32_t* seg = (uint32_t*)((char*)p.table + (p.n * 8 + 15) / 16 * 16) + p.first * WORDS;
    for (int i = threadIdx.x; i < p.count * WORDS; i += 256) seg[i] = ((const uint32_t*)p.seg)[i];
    if ((int)threadIdx.x < p.count) ((int64_t*)p.table)[p.first + threadIdx.x] = p.tile0[threadIdx.x];
}

// ---- the step ---------------------------------------------------------------------------

// One-wave workgroups in runs of 128 on one XCD.  One LLaMA-7B layer, on one card, us with fp32 /
// 8-bit states, the latter read back: 967 / 739, against 1019 / 750 in workgroups of four waves in dispatch
// order, 992 / 763 in ones of one wave, 988 / 762 in runs of 64; two or four sub-tiles per wave are as fast here
// and slower for small tensors (19.6 and 24.5 against 17.3 for 200 of them).
constexpr int kAwThreads = 64;
constexpr int kAwXcdRun = 128;

// A sub-tile of 512 elements of a tensor.  FULL: all of them exist.  RANDOM: the states are rounded so.
template <int PK, int GK, int BLOCK, bool RANDOM, bool FULL>
struct AwSub {
    static constexpr bool SPLIT = PK == kF32 || GK == kF32 || BLOCK == 0;
    int64_t i0[2];
    int valid[2];
    float th[8], g[8], m[8], v[8];
    uint32_t mw[2], vw[2], me[2], ve[2];

    __device__ __forceinline__ void load(const AwSegDev& sg, int64_t t0, int lane) {
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            i0[pc] = t0 + piece<SPLIT>(lane, pc);
            valid[pc] = FULL ? 4 : valid4(sg.n, i0[pc]);
        }
        load8<GK, SPLIT>(sg.grad, i0, valid, g);
        load8<PK, SPLIT>(sg.param, i0, valid, th);
        if constexpr (BLOCK == 0) {
            load8<kF32, SPLIT>(sg.m, i0, valid, m);
            load8<kF32, SPLIT>(sg.v, i0, valid, v);
        } else {
            load8b<SPLIT>((const uint8_t*)sg.m, i0, valid, mw);
            load8b<SPLIT>((const uint8_t*)sg.v, i0, valid, vw);
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                me[pc] = valid[pc] ? sg.mexp[i0[pc] / BLOCK] : 0u;
                ve[pc] = valid[pc] ? sg.vexp[i0[pc] / BLOCK] : 0u;
            }
        }
    }
    // pos, key: of the sub-tile's first element, where RANDOM.
    __device__ __forceinline__ void step(const AwSegDev& sg, const AwParams& p, float gs, float decay, uint64_t pos,
                                         uint64_t key, int lane) {
        if constexpr (BLOCK != 0) {
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                m_decode4(mw[pc], me[pc], m + 4 * pc);
                v_decode4(vw[pc], ve[pc], v + 4 * pc);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = g[j] * gs;
            m[j] = p.beta1 * m[j] + p.omb1 * x;
            v[j] = p.beta2 * v[j] + p.omb2 * (x * x);
            const float u = m[j] / (__builtin_sqrtf(v[j]) * p.root + p.eps);
            th[j] = th[j] * decay - p.step_size * u;
        }
        store8<PK, SPLIT>(sg.param, i0, valid, th);
        if (PK == kF32 && sg.copy) store8<kBF16, SPLIT>(sg.copy, i0, valid, th);
        if constexpr (BLOCK == 0) {
            store8<kF32, SPLIT>(sg.m, i0, valid, m);
            store8<kF32, SPLIT>(sg.v, i0, valid, v);
        } else {
            if constexpr (!FULL) {
                // elements past the end, whose m and v are 0 * inf under an infinite gradient scale, do not count
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    m[j] = (j & 3) < valid[j / 4] ? m[j] : 0.0f;
                    v[j] = (j & 3) < valid[j / 4] ? v[j] : 0.0f;
                }
            }
            uint32_t mt[2], vt[2];
            block_tops<BLOCK, SPLIT>(m, mt);
            block_tops<BLOCK, SPLIT>(v, vt);
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                me[pc] = m_exp(mt[pc]);
                if constexpr (RANDOM) {
                    const uint32_t k0 = (uint32_t)key ^ (uint32_t)(pos >> 32) * 0x9E3779B9u, k1 = (uint32_t)(key >> 32);
                    uint32_t bits[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) bits[j] = element_bits((uint32_t)pos + piece<SPLIT>(lane, pc) + j, k0, k1);
                    ve[pc] = v_exp_up(vt[pc]);
                    mw[pc] = m_encode4_random(m + 4 * pc, me[pc], bits);
                    vw[pc] = v_encode4_random(v + 4 * pc, ve[pc], bits);
                } else {
                    ve[pc] = v_exp(vt[pc]);
                    mw[pc] = m_encode4(m + 4 * pc, me[pc]);
                    vw[pc] = v_encode4(v + 4 * pc, ve[pc]);
                }
                if (valid[pc] && i0[pc] % BLOCK == 0) {
                    sg.mexp[i0[pc] / BLOCK] = (uint8_t)me[pc];
                    sg.vexp[i0[pc] / BLOCK] = (uint8_t)ve[pc];
                }
            }
            store8b<SPLIT>((uint8_t*)sg.m, i0, valid, mw);
            store8b<SPLIT>((uint8_t*)sg.v, i0, valid, vw);
        }
    }
};

// One wave per tile of kAwTile elements.  BLOCK: 0 for states in fp32.
template <int PK, int GK, int BLOCK, bool RANDOM>
__global__ __launch_bounds__(kAwThreads) void aw_kernel(const AwParams p, int64_t tbase) {
    static_assert(kAwTile == 512, "a tile is a sub-tile");
    const int lane = threadIdx.x;
    const int64_t group = xcd_remap<kXcds, kAwXcdRun>(blockIdx.x, gridDim.x);
    const int64_t tile = tbase + group;
    if (tile >= p.ntiles) return;
    const int64_t* tile0 = (const int64_t*)p.table;
    const int64_t si = find_segment(tile0, p.n, tile, lane);
    const AwSegDev sg = segments(p.table, p.n)[si];
    const float decay = (float)(1.0 - p.lr * sg.weight_decay);
    const int64_t t0 = (tile - tile0[si]) * kAwTile;
    const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
    uint64_t key = 0;
    if constexpr (RANDOM) key = p.counter ? aw_mix(p.key + (uint64_t)*p.counter) : aw_mix(p.key);
    const uint64_t pos = (uint64_t)tile * kAwTile;
    if (t0 + kAwTile <= sg.n) {
        AwSub<PK, GK, BLOCK, RANDOM, true> s;
        s.load(sg, t0, lane);
        s.step(sg, p, gs, decay, pos, key, lane);
    } else {
        AwSub<PK, GK, BLOCK, RANDOM, false> s;
        s.load(sg, t0, lane);
        s.step(sg, p, gs, decay, pos, key, lane);
    }
}

template <int PK, int GK, bool RANDOM>
const void* pick_aw(int block) {
    switch (block) {
        case 64: return (const void*)&aw_kernel<PK, GK, 64, RANDOM>;
        case 128: return (const void*)&aw_kernel<PK, GK, 128, RANDOM>;
        case 256: return (const void*)&aw_kernel<PK, GK, 256, RANDOM>;
        case 512: return (const void*)&aw_kernel<PK, GK, 512, RANDOM>;
    }
    return nullptr;
}
template <int PK, int GK>
const void* pick_aw(int block, bool random) {
    if (block == 0) return (const void*)&aw_kernel<PK, GK, 0, false>;
    return random ? pick_aw<PK, GK, true>(block) : pick_aw<PK, GK, false>(block);
}

// ---- 8-bit states to and from values ------------------------------------------------------
//
// 2 x 202 million elements, us: read into bf16 / fp32 201 / 383 (6.0 / 5.3 TB/s), written from them 211 /
// 315; with 1024 elements per wave 243 and 512 324 into bf16, in runs of workgroups per XCD the same.

template <int K, int BLOCK, bool WRITE>
__global__ __launch_bounds__(kAwThreads) void aw_state_kernel(const void* table, int64_t n, int64_t ntiles, int64_t tbase) {
    const int lane = threadIdx.x;
    const int64_t tile = tbase + blockIdx.x;
    if (tile >= ntiles) return;
    const int64_t* tile0 = (const int64_t*)table;
    const int64_t si = find_segment(tile0, n, tile, lane);
    const AwSegDev st = segments(table, n)[si];
    uint8_t* codes = (uint8_t*)st.m;
    const bool second = st.second != 0;
    constexpr bool SPLIT = K == kF32;
    constexpr int U = kAwStateTile / 512;
    const int64_t t0 = (tile - tile0[si]) * kAwStateTile;
    int64_t i0[U][2];
    int valid[U][2];
    float x[U][8];
    uint32_t w[U][2], e[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            i0[u][pc] = t0 + u * 512 + piece<SPLIT>(lane, pc);
            valid[u][pc] = valid4(st.n, i0[u][pc]);
            if (!WRITE) e[u][pc] = valid[u][pc] ? st.mexp[i0[u][pc] / BLOCK] : 0u;
        }
        if constexpr (WRITE) load8<K, SPLIT>(st.param, i0[u], valid[u], x[u]);
        else load8b<SPLIT>(codes, i0[u], valid[u], w[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (WRITE) {
            uint32_t top[2];
            block_tops<BLOCK, SPLIT>(x[u], top);
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                const uint32_t ex = second ? v_exp(top[pc]) : m_exp(top[pc]);
                w[u][pc] = second ? v_encode4(x[u] + 4 * pc, ex) : m_encode4(x[u] + 4 * pc, ex);
                if (valid[u][pc] && i0[u][pc] % BLOCK == 0) st.mexp[i0[u][pc] / BLOCK] = (uint8_t)ex;
            }
            store8b<SPLIT>(codes, i0[u], valid[u], w[u]);
        } else {
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                if (second) v_decode4(w[u][pc], e[u][pc], x[u] + 4 * pc);
                else m_decode4(w[u][pc], e[u][pc], x[u] + 4 * pc);
            }
            store8<K, SPLIT>(st.param, i0[u], valid[u], x[u]);
        }
    }
}
template <int K, bool WRITE>
const void* pick_state(int block) {
    switch (block) {
        case 64: return (const void*)&aw_state_kernel<K, 64, WRITE>;
        case 128: return (const void*)&aw_state_kernel<K, 128, WRITE>;
        case 256: return (const void*)&aw_state_kernel<K, 256, WRITE>;
        case 512: return (const void*)&aw_state_kernel<K, 512, WRITE>;
    }
    return nullptr;
}

// One wave per tile; launches of at most kMaxGrid workgroups.  args[at] takes the first tile.
hipError_t launch_tiles(const void* k, void** args, int at, int64_t ntiles, hipStream_t stream) {
    if (!k) return hipErrorInvalidValue;
    for (int64_t tbase = 0; tbase < ntiles; tbase += kMaxGrid) {
        const int64_t tiles = ntiles - tbase < kMaxGrid ? ntiles - tbase : kMaxGrid;
        args[at] = (void*)&tbase;
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)tiles), dim3(kAwThreads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_aw_fill(const AwFillParams& p, hipStream_t stream) {
    void* args[] = {(void*)&p};
    return hipLaunchKernel((const void*)&aw_fill_kernel, dim3(1), dim3(256), args, 0, stream);
}

hipError_t launch_aw(const AwParams& p, bool param_f32, bool grad_f32, int block, bool random, hipStream_t stream) {
    const void* k = param_f32 ? (grad_f32 ? pick_aw<kF32, kF32>(block, random) : pick_aw<kF32, kBF16>(block, random))
                              : (grad_f32 ? pick_aw<kBF16, kF32>(block, random) : pick_aw<kBF16, kBF16>(block, random));
    void* args[] = {(void*)&p, nullptr};
    return launch_tiles(k, args, 1, p.ntiles, stream);
}

hipError_t launch_aw_state(const void* table, int64_t n, int64_t ntiles, int block, bool f32, bool write,
                           hipStream_t stream) {
    const void* k = f32 ? (write ? pick_state<kF32, true>(block) : pick_state<kF32, false>(block))
                        : (write ? pick_state<kBF16, true>(block) : pick_state<kBF16, false>(block));
    void* args[] = {(void*)&table, (void*)&n, (void*)&ntiles, nullptr};
    return launch_tiles(k, args, 3, ntiles, stream);
}

}  // namespace loco
