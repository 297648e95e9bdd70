// Log probabilities of given tokens, the entropy of each row's distribution and its best
// alternatives; and the gradient with respect to the logits.
//
// With m = max x, d = x - m, S = sum exp(scale d) and T = sum exp(scale d) d of a row:
//   logprob = scale (x_t - m) - ln S,   entropy = ln S - scale T / S
//   dx_j = scale (dlogprob (1[j = t] - p_j) - dentropy p_j (ln p_j + entropy)),  p = exp(scale d) / S
// Forward, a row is read once: each lane keeps a running maximum with the sums relative to it, which
// move to a new maximum by one factor per batch of values.  The difference x - m is taken before
// the scale, so that values near the type's lowest do not overflow.  Sums are fp32.
//
// The best k: a row's lanes form 64 groups, each with the largest value it has seen and the first chunk
// that holds it.  Ordered by value and chunk, the k-th of the groups' best bounds the row's k best
// values from below, each of which is then in a lane whose own best is not below that bound.  Those
// lanes' values, some k of them at or above it, are collected and ranked by value and index.

#include "loco_layer.hpp"
#include "loco_step_internal.hpp"

namespace loco {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, __uint_as_float(dpp<0xB1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<0x4E>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<0x141>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<0x140>(__float_as_uint(v))));
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// The running maximum m of a lane, wave or row with S and T relative to it.  m starts at the lowest
// number, which minus infinity does not raise.
struct Sums {
    float m, s, t;
    // Moves to the maximum n >= m.  The difference may overflow (nothing summed yet, or only values near
    // the lowest); it is kept finite, as the factor 0 times it has to be 0.
    __device__ __forceinline__ void move(float n, float c) {
        const float dm = fmaxf(m - n, kLowest);
        const float r = __builtin_amdgcn_exp2f(dm * c);
        s *= r;
        t = __builtin_fmaf(s, dm, r * t);
        m = n;
    }
};

// scale (x - m), whose difference may overflow where the product does not: halves do not.
__device__ __forceinline__ float scaled_diff(float x, float m, float scale) {
    return (0.5f * x - 0.5f * m) * (2.0f * scale);
}

// A group's best value and the first chunk that holds it, as a number whose order is theirs: larger
// values first, then lower chunks.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // minus zero is zero
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(float x, uint32_t at) { return (uint64_t)ordered(x) << 32 | (uint32_t)~at; }

template <int LANES>
__device__ __forceinline__ uint64_t group_max_u64(uint64_t v) {
    const uint32_t hi = group_max_u32<LANES>((uint32_t)(v >> 32));
    const uint32_t lo = group_max_u32<LANES>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// Values of a chunk, minus infinity past the row's end.
template <typename T>
struct LpChunk;
template <>
struct LpChunk<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t* p, int valid) {
        if (valid >= 8) {
            w = load16(p);
        } else {
            w = u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) {
                    const uint32_t keep = i & 1 ? 0x0000ffffu : 0xffff0000u;
                    w[i >> 1] = (w[i >> 1] & keep) | (uint32_t)p[i] << (16 * (i & 1));
                }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_bf16x8(w, v); }
};
template <>
struct LpChunk<float> {
    float w[8];
    __device__ __forceinline__ void load(const float* p, int valid) {
        if (valid >= 8) {
            load_chunk(p, 8, w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i < valid ? p[i] : -__builtin_huge_valf();
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i];
    }
};

// ---- forward --------------------------------------------------------------------------

constexpr int kLpCand = 1024;  // candidates that are ranked at once

template <int THREADS>
struct LpShared {
    Sums wave[THREADS / 64];
    uint64_t group[64];
    uint64_t cand[kLpCand];
    uint16_t hit[THREADS];
    int nhit, ncand;
    uint64_t best;
};

// The row's best `top` values by THREADS threads, each of which has met the chunks of its own number
// plus multiples of THREADS, the best of them `mine`.
template <typename T, int THREADS>
__device__ void lp_top(const LpParams& p, const T* x, int64_t row, uint64_t mine, float m, float log_s, bool lost,
                       LpShared<THREADS>& sh) {
    const int tid = threadIdx.x, lane = tid & 63;
    int32_t* ids = p.top_ids + row * p.top;
    float* lps = p.top_logprobs + row * p.top;
    if (lost) {
        for (int i = tid; i < p.top; i += THREADS) {
            ids[i] = -1;
            lps[i] = __builtin_nanf("");
        }
        return;
    }
    const int nchunks = (p.vocab + 7) / 8;
    const int k = p.top < p.vocab ? p.top : p.vocab;
    // every wave ranks the groups' bests by itself
    const uint64_t own = sh.group[lane];
    int rank = 0;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) rank += sh.group[i] > own;
    const uint64_t at = ballot(rank == k - 1 && own != 0);
    // fewer groups than k have a chunk at all: everything counts
    uint64_t bound = 1;
    if (at) {
        const int src = __builtin_ctzll(at);
        bound = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(own >> 32), src) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((uint32_t)own, src);
    }
    if (mine >= bound) sh.hit[atomicAdd(&sh.nhit, 1)] = (uint16_t)tid;
    __syncthreads();
    const int turns = (nchunks + THREADS - 1) / THREADS, jobs = sh.nhit * turns;
    for (int job = tid; job < jobs; job += THREADS) {
        const int c = sh.hit[job / turns] + job % turns * THREADS;
        if (c >= nchunks) continue;
        const int left = p.vocab - c * 8, valid = left < 8 ? left : 8;
        LpChunk<T> ch;
        ch.load(x + (int64_t)c * 8, valid);
        float v[8];
        ch.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < valid && order_key(v[j], (uint32_t)c) >= bound) {
                const int n = atomicAdd(&sh.ncand, 1);
                if (n < kLpCand) sh.cand[n] = order_key(v[j], (uint32_t)(c * 8 + j));
            }
    }
    __syncthreads();
    const int n = sh.ncand;
    auto write = [&](int i, uint64_t key) {
        const uint32_t id = ~(uint32_t)key, u = (uint32_t)(key >> 32);
        const float v = __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
        ids[i] = (int32_t)id;
        lps[i] = v == -__builtin_huge_valf() ? v : scaled_diff(v, m, p.scale) - log_s;
    };
    if (n <= kLpCand) {
        for (int i = tid; i < n; i += THREADS) {
            const uint64_t key = sh.cand[i];
            int above = 0;
            for (int j = 0; j < n; ++j) above += sh.cand[j] > key;
            if (above < k) write(above, key);
        }
    } else {
        // More values in the hit lanes than fit, as where few lanes hold all the large ones: one after
        // the other, each the largest below the last.
        uint64_t last = ~(uint64_t)0;
        for (int i = 0; i < k; ++i) {
            uint64_t best = 0;
            for (int j = tid; j < p.vocab; j += THREADS) {
                float v;
                if constexpr (sizeof(T) == 2) v = __uint_as_float((uint32_t)x[j] << 16);
                else v = x[j];
                const uint64_t key = order_key(v, (uint32_t)j);
                best = key < last && key > best ? key : best;
            }
            best = group_max_u64<64>(best);
            if (tid == 0) sh.best = 0;
            __syncthreads();
            if (lane == 0) atomicMax((unsigned long long*)&sh.best, (unsigned long long)best);
            __syncthreads();
            last = sh.best;
            if (tid == 0) write(i, last);
            __syncthreads();
        }
    }
    for (int i = k + tid; i < p.top; i += THREADS) {
        ids[i] = -1;
        lps[i] = -__builtin_huge_valf();
    }
}

// One workgroup per row.
template <typename T, int THREADS, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(THREADS) void lp_kernel(const LpParams p, int64_t row0) {
    constexpr int WAVES = THREADS / 64, U = sizeof(T) == 2 ? 4 : 2;  // 64 bytes per lane at once
    __shared__ LpShared<THREADS> sh;
    const int64_t row = row0 + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const T* x = (const T*)p.logits + row * p.ld;
    const float c = p.scale * kLog2e;
    const int nchunks = (p.vocab + 7) / 8;
    if (TOP && tid == 0) sh.nhit = sh.ncand = 0;
    // the given token's logit, on its way beside the row's
    int64_t target = -1;
    float xt = 0.0f;
    if (tid == 0 && p.targets) {
        target = p.targets[row];
        if (target >= 0 && target < p.vocab) {
            if constexpr (sizeof(T) == 2) xt = __uint_as_float((uint32_t)x[target] << 16);
            else xt = x[target];
        }
    }
    Sums a = {kLowest, 0.0f, 0.0f};
    float best = -__builtin_huge_valf();
    uint32_t best_chunk = tid;
    for (int c0 = tid; c0 < nchunks; c0 += U * THREADS) {
        LpChunk<T> ch[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = (int64_t)(c0 + u * THREADS) * 8;
            const int64_t left = p.vocab - at;
            ch[u].load(x + at, left < 8 ? (left > 0 ? (int)left : 0) : 8);
        }
        float v[8], top = kLowest;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ch[u].get(v);
            const float q = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
            top = fmaxf(top, q);
            if constexpr (TOP) {
                best_chunk = q > best ? (uint32_t)(c0 + u * THREADS) : best_chunk;
                best = fmaxf(best, q);
            }
        }
        a.move(fmaxf(a.m, top), c);
        float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ch[u].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = v[j] - a.m;
                const float e = __builtin_amdgcn_exp2f(d * c);
                s[j & 1] += e;
                // masked: 0 times a finite number
                if constexpr (ENTROPY) t[j & 1] = __builtin_fmaf(e, fmaxf(d, kLowest), t[j & 1]);
            }
        }
        a.s += s[0] + s[1];
        a.t += t[0] + t[1];
    }
    // the wave's and the row's sums
    a.move(wave_max(a.m), c);
    a.s = wave_sum(a.s);
    if constexpr (ENTROPY) a.t = wave_sum(a.t);
    uint64_t mine = 0;
    if constexpr (TOP) {
        mine = best_chunk < (uint32_t)nchunks ? order_key(best, best_chunk) : 0;
        constexpr int G = THREADS / 64;  // lanes per group
        const uint64_t g = group_max_u64<G>(mine);
        if (tid % G == 0) sh.group[tid / G] = g;
    }
    if constexpr (WAVES > 1) {
        if (lane == 0) sh.wave[wave] = a;
        __syncthreads();
        a = sh.wave[0];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) {
            Sums b = sh.wave[i];
            const float m = fmaxf(a.m, b.m);
            a.move(m, c);
            b.move(m, c);
            a.s += b.s;
            a.t += b.t;
        }
    } else if constexpr (TOP) {
        __syncthreads();
    }
    const bool lost = a.s != a.s, empty = a.s == 0.0f;
    const float log_s = logf(a.s);
    if (tid == 0) {
        const float nan = __builtin_nanf(""), inf = __builtin_huge_valf();
        if (p.stats) {
            p.stats[2 * row] = lost ? nan : empty ? -inf : a.m;
            p.stats[2 * row + 1] = a.s;
        }
        if (p.logprob)
            p.logprob[row] = target < 0                   ? 0.0f
                             : lost || target >= p.vocab ? nan
                             : empty                      ? -inf
                                                          : scaled_diff(xt, a.m, p.scale) - log_s;
        if (p.entropy) p.entropy[row] = empty ? 0.0f : log_s - p.scale * a.t / a.s;
    }
    if constexpr (TOP) lp_top<T, THREADS>(p, x, row, mine, a.m, log_s, lost, sh);
}

template <typename T, int THREADS>
const void* pick_lp(bool entropy, bool top) {
    return entropy ? (top ? (const void*)&lp_kernel<T, THREADS, true, true> : (const void*)&lp_kernel<T, THREADS, true, false>)
                   : (top ? (const void*)&lp_kernel<T, THREADS, false, true>
                          : (const void*)&lp_kernel<T, THREADS, false, false>);
}
template <typename T>
const void* pick_lp(int threads, bool entropy, bool top) {
    return threads == 64    ? pick_lp<T, 64>(entropy, top)
           : threads == 256 ? pick_lp<T, 256>(entropy, top)
                            : pick_lp<T, 1024>(entropy, top);
}

// ---- backward -------------------------------------------------------------------------

constexpr int kLpBwdThreads = 256;
constexpr int kLpBwdChunks = 4;  // per lane

template <typename T, bool ENTROPY>
__global__ __launch_bounds__(kLpBwdThreads) void lp_bwd_kernel(const LpBwdParams p, int64_t group0, int64_t segs) {
    constexpr int U = kLpBwdChunks;
    const int64_t g = group0 + blockIdx.x;
    const int64_t row = g / segs;
    const int base = (int)(g - row * segs) * (kLpBwdThreads * U * 8);
    const T* x = (const T*)p.logits + row * p.ld + base;
    T* dx = (T*)p.dlogits + row * p.dld + base;
    const int cols = p.vocab - base;  // of this segment and what follows
    const float m = p.stats[2 * row], s = p.stats[2 * row + 1];
    const int64_t target = p.targets ? p.targets[row] : -1;
    float dlp = p.dlogprob ? p.dlogprob[row] : 0.0f;
    if (target < 0) dlp = 0.0f;
    else if (p.dlogprob && target >= p.vocab) dlp = __builtin_nanf("");
    // a row without a distribution, or without anything to differentiate, has the gradient 0
    const bool zero = s == 0.0f || (!ENTROPY && (target < 0 || !p.dlogprob));
    const float inv = 1.0f / s, c = p.scale * kLog2e;
    float k = -p.scale * dlp, kd = 0.0f;
    if constexpr (ENTROPY) {
        const float dh = p.dentropy[row];
        k -= p.scale * dh * (p.entropy[row] - logf(s));
        kd = -p.scale * dh * kLn2;
    }
    const int64_t own = target - base;
    LpChunk<T> ch[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = (u * kLpBwdThreads + (int)threadIdx.x) * 8;
        if (!zero) ch[u].load(x + at, cols - at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = (u * kLpBwdThreads + (int)threadIdx.x) * 8;
        float v[8];
        if (zero) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        } else {
            ch[u].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // below 2^-160 the probability is 0 in fp32, and so is its product with a finite number
                const float d = fmaxf((v[j] - m) * c, -160.0f);
                const float e = __builtin_amdgcn_exp2f(d) * inv;
                v[j] = e * (ENTROPY ? __builtin_fmaf(kd, d, k) : k);
                v[j] += at + j == own ? p.scale * dlp : 0.0f;
            }
        }
        store_chunk(dx + at, cols - at, v);
    }
}

}  // namespace

hipError_t launch_lp(const LpParams& p, hipStream_t stream) {
    // At least 64 chunks for each of the groups' lanes, so that the groups bound the best values.
    const int threads = p.vocab <= 2048 ? 64 : p.rows >= 512 || p.vocab < 8192 ? 256 : 1024;
    const bool entropy = p.entropy != nullptr, top = p.top > 0;
    const void* k = p.f32 ? pick_lp<float>(threads, entropy, top) : pick_lp<uint16_t>(threads, entropy, top);
    for (int64_t row0 = 0; row0 < p.rows; row0 += kMaxGrid) {
        const int64_t rows = p.rows - row0 < kMaxGrid ? p.rows - row0 : kMaxGrid;
        void* args[] = {(void*)&p, (void*)&row0};
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)rows), dim3(threads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t launch_lp_bwd(const LpBwdParams& p, hipStream_t stream) {
    constexpr int64_t per = kLpBwdThreads * kLpBwdChunks * 8;
    const int64_t segs = (p.vocab + per - 1) / per, groups = p.rows * segs;
    const bool entropy = p.dentropy != nullptr;
    const void* k = p.f32 ? (entropy ? (const void*)&lp_bwd_kernel<float, true> : (const void*)&lp_bwd_kernel<float, false>)
                          : (entropy ? (const void*)&lp_bwd_kernel<uint16_t, true>
                                     : (const void*)&lp_bwd_kernel<uint16_t, false>);
    for (int64_t g0 = 0; g0 < groups; g0 += kMaxGrid) {
        const int64_t n = groups - g0 < kMaxGrid ? groups - g0 : kMaxGrid;
        void* args[] = {(void*)&p, (void*)&g0, (void*)&segs};
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)n), dim3(kLpBwdThreads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace loco
