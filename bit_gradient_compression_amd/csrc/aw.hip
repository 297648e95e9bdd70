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

// The last of the `n` starts that is not past `tile` (lane i holds start i).
__device__ __forceinline__ int find_segment(const int64_t* tile0, int n, int64_t tile, int lane) {
    const bool before = lane < n && tile0[lane < n ? lane : 0] <= tile;
    return uniform(__builtin_popcountll(ballot(before)) - 1);
}

// ---- the step ---------------------------------------------------------------------------

constexpr int kAwThreads = 256;

// One wave per tile of 512 elements.  BLOCK: 0 for states in fp32.
template <int PK, int GK, int BLOCK>
__global__ __launch_bounds__(kAwThreads) void aw_kernel(const AwParams p, int64_t tbase) {
    constexpr bool SPLIT = PK == kF32 || GK == kF32 || BLOCK == 0;
    const int lane = threadIdx.x & 63;
    const int64_t tile = tbase + (int64_t)blockIdx.x * (kAwThreads / 64) + uniform(threadIdx.x >> 6);
    if (tile >= p.ntiles) return;  // whole waves
    const int si = find_segment(p.tile0, p.nseg, tile, lane);
    const AwSegDev sg = p.seg[si];
    const float decay = p.decay[si];
    const int64_t t0 = (tile - p.tile0[si]) * kAwTile;
    float th[8], g[8], m[8], v[8];
    uint32_t mw[2], vw[2], me[2], ve[2];
#pragma unroll
    for (int pc = 0; pc < 2; ++pc) {
        const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
        const int valid = valid4(sg.n, i0);
        load4<GK>(sg.grad, i0, valid, g + 4 * pc);
        load4<PK>(sg.param, i0, valid, th + 4 * pc);
        if constexpr (BLOCK == 0) {
            load4<kF32>(sg.m, i0, valid, m + 4 * pc);
            load4<kF32>(sg.v, i0, valid, v + 4 * pc);
        } else {
            mw[pc] = load4b((const uint8_t*)sg.m, i0, valid);
            vw[pc] = load4b((const uint8_t*)sg.v, i0, valid);
            me[pc] = valid ? sg.mexp[i0 / BLOCK] : 0u;
            ve[pc] = valid ? sg.vexp[i0 / BLOCK] : 0u;
        }
    }
    const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
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
    if constexpr (BLOCK != 0) {
        // elements past the end, whose m and v are 0 * inf under an infinite gradient scale, do not count
        uint32_t mt[2], vt[2];
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            const int valid = valid4(sg.n, t0 + piece<SPLIT>(lane, pc));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[4 * pc + j] = j < valid ? m[4 * pc + j] : 0.0f;
                v[4 * pc + j] = j < valid ? v[4 * pc + j] : 0.0f;
            }
        }
        block_tops<BLOCK, SPLIT>(m, mt);
        block_tops<BLOCK, SPLIT>(v, vt);
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            me[pc] = m_exp(mt[pc]);
            ve[pc] = v_exp(vt[pc]);
            mw[pc] = m_encode4(m + 4 * pc, me[pc]);
            vw[pc] = v_encode4(v + 4 * pc, ve[pc]);
        }
    }
#pragma unroll
    for (int pc = 0; pc < 2; ++pc) {
        const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
        const int valid = valid4(sg.n, i0);
        store4<PK>(sg.param, i0, valid, th + 4 * pc);
        if (PK == kF32 && sg.copy) store4<kBF16>(sg.copy, i0, valid, th + 4 * pc);
        if constexpr (BLOCK == 0) {
            store4<kF32>(sg.m, i0, valid, m + 4 * pc);
            store4<kF32>(sg.v, i0, valid, v + 4 * pc);
        } else {
            store4b((uint8_t*)sg.m, i0, valid, mw[pc]);
            store4b((uint8_t*)sg.v, i0, valid, vw[pc]);
            if (valid && i0 % BLOCK == 0) {
                sg.mexp[i0 / BLOCK] = (uint8_t)me[pc];
                sg.vexp[i0 / BLOCK] = (uint8_t)ve[pc];
            }
        }
    }
}

template <int PK, int GK>
const void* pick_aw(int block) {
    switch (block) {
        case 0: return (const void*)&aw_kernel<PK, GK, 0>;
        case 64: return (const void*)&aw_kernel<PK, GK, 64>;
        case 128: return (const void*)&aw_kernel<PK, GK, 128>;
        case 256: return (const void*)&aw_kernel<PK, GK, 256>;
        case 512: return (const void*)&aw_kernel<PK, GK, 512>;
    }
    return nullptr;
}

// ---- 8-bit states to and from values ------------------------------------------------------

template <int K, int BLOCK, bool WRITE>
__global__ __launch_bounds__(kAwThreads) void aw_state_kernel(const AwStateParams p, int64_t tbase) {
    const int lane = threadIdx.x & 63;
    const int64_t tile = tbase + (int64_t)blockIdx.x * (kAwThreads / 64) + uniform(threadIdx.x >> 6);
    if (tile >= p.ntiles) return;
    const int si = find_segment(p.tile0, p.nst, tile, lane);
    const AwStateDev st = p.st[si];
    const bool second = (p.second >> si) & 1u;
    constexpr bool SPLIT = K == kF32;
    const int64_t t0 = (tile - p.tile0[si]) * kAwTile;
    float x[8];
    if constexpr (WRITE) {
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
            load4<K>(st.values, i0, valid4(st.n, i0), x + 4 * pc);
        }
        uint32_t top[2];
        block_tops<BLOCK, SPLIT>(x, top);
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
            const int valid = valid4(st.n, i0);
            const uint32_t e = second ? v_exp(top[pc]) : m_exp(top[pc]);
            store4b(st.codes, i0, valid, second ? v_encode4(x + 4 * pc, e) : m_encode4(x + 4 * pc, e));
            if (valid && i0 % BLOCK == 0) st.exps[i0 / BLOCK] = (uint8_t)e;
        }
    } else {
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
            const int valid = valid4(st.n, i0);
            const uint32_t w = load4b(st.codes, i0, valid);
            const uint32_t e = valid ? st.exps[i0 / BLOCK] : 0u;
            if (second) v_decode4(w, e, x + 4 * pc);
            else m_decode4(w, e, x + 4 * pc);
        }
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            const int64_t i0 = t0 + piece<SPLIT>(lane, pc);
            store4<K>(st.values, i0, valid4(st.n, i0), x + 4 * pc);
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

// One wave per tile; launches of at most kMaxGrid workgroups.
template <typename P>
hipError_t launch_tiles(const void* k, const P& p, hipStream_t stream) {
    if (!k) return hipErrorInvalidValue;
    constexpr int64_t waves = kAwThreads / 64;
    for (int64_t tbase = 0; tbase < p.ntiles; tbase += kMaxGrid * waves) {
        const int64_t tiles = p.ntiles - tbase < kMaxGrid * waves ? p.ntiles - tbase : kMaxGrid * waves;
        void* args[] = {(void*)&p, (void*)&tbase};
        const hipError_t err =
            hipLaunchKernel(k, dim3((unsigned)((tiles + waves - 1) / waves)), dim3(kAwThreads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_aw(const AwParams& p, bool param_f32, bool grad_f32, int block, hipStream_t stream) {
    const void* k = param_f32 ? (grad_f32 ? pick_aw<kF32, kF32>(block) : pick_aw<kF32, kBF16>(block))
                              : (grad_f32 ? pick_aw<kBF16, kF32>(block) : pick_aw<kBF16, kBF16>(block));
    return launch_tiles(k, p, stream);
}

hipError_t launch_aw_state(const AwStateParams& p, int block, bool f32, bool write, hipStream_t stream) {
    const void* k = f32 ? (write ? pick_state<kF32, true>(block) : pick_state<kF32, false>(block))
                        : (write ? pick_state<kBF16, true>(block) : pick_state<kBF16, false>(block));
    return launch_tiles(k, p, stream);
}

}  // namespace loco
