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
//
// Forward, a large call is bound by HBM and nearly as much by its 11 instructions per value: 8192 x 32000 in
// bf16 86 us, 6.1 TB/s, with the vector units busy for most of them; in fp32 176 us, 6.0 TB/s.  A few rows are
// bound by latency: a row of 32000 with 8 alternatives takes 6.8 us, 3.5 more than nothing at all, 48 of 131071 with
// 20 take 12.8 and 3.9 for the join; half of their LDS cycles are conflicts of the groups' layout.  The gradient
// reads and writes each value once: 168 us for 8192 x 32000, 6.2 TB/s; in fp32 398 us, 5.3 TB/s.
//
// How a row is cut depends on the number of rows (below), and so do the order of its sums and their last bit.

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

// 16 bytes at any address.  Once: they leave the caches to what is read again.
template <bool ONCE>
__device__ __forceinline__ u32x4 load16_for(const void* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load((const u32x4_any*)p);
    else return load16(p);
}

// The sequence of a row; rows of more than one are fewer than 2^32.
__device__ __forceinline__ int64_t seq_of(const LpSeqs& s, int64_t row) { return s.rows ? (uint32_t)row / s.rows : 0u; }

// Values of a chunk, minus infinity past the row's end.
template <typename T>
struct LpChunk;
template <>
struct LpChunk<uint16_t> {
    u32x4 w;
    template <bool ONCE>
    __device__ __forceinline__ void load(const uint16_t* p, int valid) {
        if (valid >= 8) {
            w = load16_for<ONCE>(p);
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
    template <bool ONCE>
    __device__ __forceinline__ void load(const float* p, int valid) {
        if (valid >= 8) {
            const u32x4 a = load16_for<ONCE>(p), b = load16_for<ONCE>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __uint_as_float(a[i]);
                w[4 + i] = __uint_as_float(b[i]);
            }
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

// Candidates that are ranked at once, and slots (below) that are looked through once more.  A single wave's
// bounds hold all that it can have where fewer lanes than k have a chunk, or where all values are equal.
constexpr int lp_cand(int threads) { return threads == 64 ? 256 : 1024; }
constexpr int lp_hits(int threads) { return threads == 64 ? 256 : 1024; }

// A lane's batches of values, in order, over this many slots: each slot has the largest of its values.
constexpr int lp_slots(int threads) { return threads == 256 ? 16 : threads == 64 ? 4 : 2; }

template <int THREADS>
struct LpShared {
    Sums wave[THREADS / 64];
    uint64_t lane[THREADS];  // each lane's best
    uint64_t group[64];
    uint64_t cand[lp_cand(THREADS) + 8];
    float slot[lp_slots(THREADS)][THREADS];
    uint16_t hit[lp_hits(THREADS)];
    int nhit, ncand;
    uint64_t bound, best;
};

// The sums of all waves, in every lane.  sh.wave is free again after the next barrier.
template <int THREADS>
__device__ __forceinline__ Sums join_waves(Sums a, float c, LpShared<THREADS>& sh) {
    constexpr int WAVES = THREADS / 64;
    const int lane = threadIdx.x & 63;
    a.move(wave_max(a.m), c);
    a.s = wave_sum(a.s);
    a.t = wave_sum(a.t);
    if constexpr (WAVES > 1) {
        if (lane == 0) sh.wave[threadIdx.x >> 6] = a;
        __syncthreads();
        const Sums none = {kLowest, 0.0f, 0.0f};
        a = lane < WAVES ? sh.wave[lane] : none;
        a.move(wave_max(a.m), c);
        a.s = wave_sum(a.s);
        a.t = wave_sum(a.t);
    }
    return a;
}

// The k-th largest of the 64 groups' bests (1 if fewer groups than k have one), in every lane.  A group is every
// 64th lane: where all values are equal and the first ones count, these are in as many groups.  Called by all
// threads after the barrier that follows the writes of sh.lane; ends with one.
template <int THREADS>
__device__ __forceinline__ uint64_t kth_group(int k, LpShared<THREADS>& sh) {
    constexpr int PER = THREADS / 64;  // lanes per group: each compares it with 64 / PER others
    const int g = threadIdx.x / PER, part = threadIdx.x % PER;
    const uint64_t own = group_max_u64<PER>(sh.lane[part * 64 + g]);
    if (part == 0) sh.group[g] = own;
    __syncthreads();
    int above = 0;
#pragma unroll 16
    for (int i = 0; i < 64 / PER; ++i) above += sh.group[part * (64 / PER) + i] > own;
    if constexpr (PER >= 2) above += (int)dpp<0xB1>((uint32_t)above);
    if constexpr (PER >= 4) above += (int)dpp<0x4E>((uint32_t)above);
    if constexpr (PER >= 8) above += (int)dpp<0x141>((uint32_t)above);
    if constexpr (PER >= 16) above += (int)dpp<0x140>((uint32_t)above);
    if (above == k - 1 && own != 0) sh.bound = own;  // one group's lanes: the keys differ
    __syncthreads();
    return sh.bound;
}

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <int THREADS>
__device__ __forceinline__ void add_candidate(uint64_t key, LpShared<THREADS>& sh) {
    const int n = atomicAdd(&sh.ncand, 1);
    if (n < lp_cand(THREADS)) sh.cand[n] = key;
}

// The first k of the n candidates in order: emit(rank, key).
template <int THREADS, typename Emit>
__device__ __forceinline__ void rank_candidates(int n, int k, LpShared<THREADS>& sh, Emit emit) {
    if (threadIdx.x < 8) sh.cand[n + threadIdx.x] = 0;  // the last eight that are read together
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const uint64_t key = sh.cand[i];
        int above = 0;
        for (int j = 0; j < n; j += 8)
#pragma unroll
            for (int q = 0; q < 8; ++q) above += sh.cand[j + q] > key;
        if (above < k) emit(above, key);
    }
}

// One of a row's alternatives.
__device__ __forceinline__ void write_top(const LpParams& p, int64_t row, int i, uint64_t key, float m, float log_s) {
    const float v = key_value(key);
    p.top_ids[row * p.top + i] = (int32_t) ~(uint32_t)key;
    p.top_logprobs[row * p.top + i] = v == -__builtin_huge_valf() ? v : scaled_diff(v, m, p.scale) - log_s;
}

// Alternatives past the vocabulary, or all of them of a row without a distribution.
__device__ __forceinline__ void write_no_top(const LpParams& p, int64_t row, int i, bool lost) {
    p.top_ids[row * p.top + i] = -1;
    p.top_logprobs[row * p.top + i] = lost ? __builtin_nanf("") : -__builtin_huge_valf();
}

// A row's numbers from its sums, by one thread.
__device__ __forceinline__ void write_row(const LpParams& p, int64_t row, const Sums& a, float log_s) {
    const bool lost = a.s != a.s, empty = a.s == 0.0f;
    const float nan = __builtin_nanf(""), inf = __builtin_huge_valf();
    if (p.stats) {
        p.stats[2 * row] = lost ? nan : empty ? -inf : a.m;
        p.stats[2 * row + 1] = a.s;
    }
    if (p.entropy) p.entropy[row] = empty ? 0.0f : log_s - p.scale * a.t / a.s;
}
template <typename T>
__device__ __forceinline__ float target_logit(const LpParams& p, int64_t row, int64_t& target) {
    const int64_t seq = seq_of(p.seqs, row);
    target = p.targets[row + seq * p.seqs.targets];
    if (target < 0 || target >= p.vocab) return 0.0f;
    const T* x = (const T*)p.logits + row * p.ld + seq * p.seqs.logits + target;
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)*x << 16);
    else return *x;
}
__device__ __forceinline__ void write_logprob(const LpParams& p, int64_t row, const Sums& a, float log_s, int64_t target,
                                              float xt) {
    p.logprob[row] = target < 0                         ? 0.0f
                     : a.s != a.s || target >= p.vocab ? __builtin_nanf("")
                     : a.s == 0.0f                      ? -__builtin_huge_valf()
                                                        : scaled_diff(xt, a.m, p.scale) - log_s;
}

// One workgroup per row, or (SPLIT) per piece of p.piece chunks of a row, whose sums and best values go to the
// workspace for lp_join_kernel.
template <typename T, int THREADS, bool ENTROPY, bool TOP, bool SPLIT>
__global__ __launch_bounds__(THREADS) void lp_kernel(const LpParams p, int64_t row0) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // 64 bytes per lane at once
    __shared__ LpShared<THREADS> sh;
    int64_t row = row0 + blockIdx.x;
    int first = 0, last = (p.vocab + 7) / 8;  // chunks
    int64_t part = 0;
    if constexpr (SPLIT) {
        part = row0 + blockIdx.x;
        row = part / p.splits;
        first = (int)(part - row * p.splits) * p.piece;
        last = min(last, first + p.piece);
    }
    const int tid = threadIdx.x;
    const T* x = (const T*)p.logits + row * p.ld + seq_of(p.seqs, row) * p.seqs.logits;
    const float c = p.scale * kLog2e;
    if constexpr (TOP) {
        if (tid == 0) {
            sh.nhit = sh.ncand = 0;
            sh.bound = 1;
        }
    }
    // the given token's logit, on its way beside the row's
    int64_t target = -1;
    float xt = 0.0f;
    if (!SPLIT && tid == 0 && p.logprob) xt = target_logit<T>(p, row, target);
    Sums a = {kLowest, 0.0f, 0.0f};
    float best = -__builtin_huge_valf();
    uint32_t best_chunk = first + tid;
    LpChunk<T> ch[U];
    constexpr int SLOTS = lp_slots(THREADS);
    int turn = 0;
    auto valid_of = [&](int at) { return at < last ? min(p.vocab - at * 8, 8) : 0; };
    for (int c0 = first + tid; c0 < last; c0 += U * THREADS, ++turn) {
#pragma unroll
        for (int u = 0; u < U; ++u) ch[u].template load<!TOP>(x + (int64_t)(c0 + u * THREADS) * 8, valid_of(c0 + u * THREADS));
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
        if constexpr (TOP) {
            float& slot = sh.slot[turn % SLOTS][tid];
            slot = turn < SLOTS ? top : fmaxf(slot, top);
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
    uint64_t mine = 0;
    if constexpr (TOP) {
        mine = best_chunk < (uint32_t)last ? order_key(best, best_chunk) : 0;
        sh.lane[tid] = mine;
    }
    a = join_waves<THREADS>(a, c, sh);
    const float log_s = SPLIT ? 0.0f : logf(a.s);
    const bool lost = a.s != a.s;
    if (tid == 0) {
        if constexpr (SPLIT) {
            p.sums[part] = f32x4{a.m, a.s, a.t, 0.0f};
        } else {
            write_row(p, row, a, log_s);
            if (p.logprob) write_logprob(p, row, a, log_s, target, xt);
        }
    }
    if constexpr (TOP) {
        const int elems = min(p.vocab - first * 8, (last - first) * 8);
        const int k = min(p.top, elems);
        uint64_t* keys = SPLIT ? p.keys + part * p.top : nullptr;
        auto emit = [&](int i, uint64_t key) {
            if constexpr (SPLIT) keys[i] = key;
            else write_top(p, row, i, key, a.m, log_s);
        };
        for (int i = tid; i < p.top; i += THREADS) {
            if (i < k && !lost) continue;
            if constexpr (SPLIT) keys[i] = 0;
            else write_no_top(p, row, i, lost);
        }
        if (lost) return;  // the workgroup
        if constexpr (THREADS == 64) __syncthreads();
        const uint64_t bound = kth_group<THREADS>(k, sh);
        // The values of the slots that reach the bound, once more, one per lane.  (Taken from the registers of
        // the lanes that hold them, they need a branch each: code that runs once is fetched for as long as it
        // runs.)
        const int turns = (last - first + U * THREADS - 1) / (U * THREADS);
        if (mine >= bound) {
            const float least = bound == 1 ? kLowest : key_value(bound);  // minus infinity is in a slot as the lowest number
            for (int i = 0; i < min(turns, SLOTS); ++i)
                if (first + tid + i * U * THREADS < last && sh.slot[i][tid] >= least) {
                    const int n = atomicAdd(&sh.nhit, 1);
                    if (n < lp_hits(THREADS)) sh.hit[n] = (uint16_t)(tid * SLOTS + i);
                }
        }
        __syncthreads();
        const int each = min(U, (last - first + THREADS - 1) / THREADS);  // chunks of a batch
        const int per = (turns + SLOTS - 1) / SLOTS * each * 8, nhit = sh.nhit;
        if (nhit <= lp_hits(THREADS)) {
            for (int job = tid; job < nhit * per; job += THREADS) {
                const int h = job / per, r = job - h * per, lane_of = sh.hit[h] / SLOTS, slot = sh.hit[h] % SLOTS;
                const int at = first + lane_of + ((slot + r / (each * 8) * SLOTS) * U + r / 8 % each) * THREADS;
                const int i = at * 8 + r % 8;
                if (at >= last || i >= p.vocab) continue;
                float v;
                if constexpr (sizeof(T) == 2) v = __uint_as_float((uint32_t)x[i] << 16);
                else v = x[i];
                if (order_key(v, (uint32_t)at) >= bound) add_candidate(order_key(v, (uint32_t)i), sh);
            }
        }
        __syncthreads();
        const int n = sh.ncand;
        if (nhit <= lp_hits(THREADS) && n <= lp_cand(THREADS)) {
            rank_candidates<THREADS>(n, k, sh, emit);
            return;
        }
        // More slots or values than fit, as where few lanes hold all the large ones: one after the other, each
        // the largest below the last.
        uint64_t before = ~(uint64_t)0;
        for (int i = 0; i < k; ++i) {
            uint64_t most = 0;
            for (int j = tid; j < elems; j += THREADS) {
                float v;
                if constexpr (sizeof(T) == 2) v = __uint_as_float((uint32_t)x[first * 8 + j] << 16);
                else v = x[first * 8 + j];
                const uint64_t key = order_key(v, (uint32_t)(first * 8 + j));
                most = key < before && key > most ? key : most;
            }
            most = group_max_u64<64>(most);
            if (tid == 0) sh.best = 0;
            __syncthreads();
            if ((tid & 63) == 0) atomicMax((unsigned long long*)&sh.best, (unsigned long long)most);
            __syncthreads();
            before = sh.best;
            if (tid == 0) emit(i, before);
            __syncthreads();
        }
    }
}

// A row's results from its pieces' sums and best values, in the pieces' order.
template <typename T, bool TOP>
__global__ __launch_bounds__(256) void lp_join_kernel(const LpParams p, int64_t row0) {
    constexpr int THREADS = 256, KEYS = kLpMaxSplits * kLpMaxTop / THREADS;
    static_assert(kLpMaxSplits * kLpMaxTop <= lp_cand(THREADS));
    __shared__ LpShared<THREADS> sh;
    const int64_t row = row0 + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const float c = p.scale * kLog2e;
    if constexpr (TOP) {
        if (tid == 0) {
            sh.ncand = 0;
            sh.bound = 1;
        }
    }
    int64_t target = -1;
    float xt = 0.0f;
    if (tid == 0 && p.logprob) xt = target_logit<T>(p, row, target);
    uint64_t key[KEYS], mine = 0;
    if constexpr (TOP) {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int at = i * THREADS + tid;
            key[i] = at < p.splits * p.top ? p.keys[row * p.splits * p.top + at] : 0;
            mine = key[i] > mine ? key[i] : mine;
        }
    }
    Sums a = {kLowest, 0.0f, 0.0f};
    if (lane < p.splits) {
        const f32x4 q = p.sums[row * p.splits + lane];
        a = {q.x, q.y, q.z};
    }
    a.move(wave_max(a.m), c);
    a.s = wave_sum(a.s);
    a.t = wave_sum(a.t);
    const float log_s = logf(a.s);
    const bool lost = a.s != a.s;
    if (tid == 0) {
        write_row(p, row, a, log_s);
        if (p.logprob) write_logprob(p, row, a, log_s, target, xt);
    }
    if constexpr (TOP) {
        const int k = min(p.top, p.vocab);
        for (int i = tid; i < p.top; i += THREADS)
            if (i >= k || lost) write_no_top(p, row, i, lost);
        if (lost) return;
        sh.lane[tid] = mine;
        __syncthreads();
        const uint64_t bound = kth_group<THREADS>(k, sh);
#pragma unroll
        for (int i = 0; i < KEYS; ++i)
            if (key[i] >= bound) add_candidate(key[i], sh);
        __syncthreads();
        rank_candidates<THREADS>(sh.ncand, k, sh, [&](int i, uint64_t q) { write_top(p, row, i, q, a.m, log_s); });
    }
}

template <typename T, int THREADS, bool SPLIT>
const void* pick_lp(bool entropy, bool top) {
    return entropy ? (top ? (const void*)&lp_kernel<T, THREADS, true, true, SPLIT>
                          : (const void*)&lp_kernel<T, THREADS, true, false, SPLIT>)
                   : (top ? (const void*)&lp_kernel<T, THREADS, false, true, SPLIT>
                          : (const void*)&lp_kernel<T, THREADS, false, false, SPLIT>);
}
template <typename T>
const void* pick_lp(int threads, bool split, bool entropy, bool top) {
    return split            ? pick_lp<T, 256, true>(entropy, top)
           : threads == 64  ? pick_lp<T, 64, false>(entropy, top)
           : threads == 256 ? pick_lp<T, 256, false>(entropy, top)
                            : pick_lp<T, 1024, false>(entropy, top);
}
template <typename T>
const void* pick_lp_join(bool top) {
    return top ? (const void*)&lp_join_kernel<T, true> : (const void*)&lp_join_kernel<T, false>;
}

// ---- backward -------------------------------------------------------------------------

// One wave takes 1024 elements of a row; runs of 128 of them are on one XCD.  The stores stream past the
// caches.  8192 x 32000 in bf16 / 333 x 50001 in fp32 (133 MB, whose half the caches hold), us in one run: 169 / 25;
// four waves of 2048 elements each in dispatch order 192 / 25, with streaming stores 184 / 27, with streaming
// loads too 180 / 32; this with streaming loads too 165 / 29, with 1536 elements 175 / 26.
constexpr int kLpBwdChunks = 2;  // per lane
constexpr int kLpBwdTile = 64 * kLpBwdChunks * 8;

__device__ __forceinline__ void store_once(uint16_t* p, int valid, const float (&v)[8]) {
    if (valid >= 8) stream16(p, pack_bf16x8(v));
    else store_chunk(p, valid, v);
}
__device__ __forceinline__ void store_once(float* p, int valid, const float (&v)[8]) {
    if (valid >= 8) {
        stream16(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
        stream16(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else {
        store_chunk(p, valid, v);
    }
}

// segs: tiles per row.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(64) void lp_bwd_kernel(const LpBwdParams p, int64_t row0, uint32_t segs) {
    constexpr int U = kLpBwdChunks;
    const uint32_t g = (uint32_t)xcd_remap<kXcds, 128>(blockIdx.x, gridDim.x), r = g / segs;
    const int64_t row = row0 + r;
    const int base = (int)(g - r * segs) * kLpBwdTile;
    const int64_t seq = seq_of(p.seqs, row);
    const T* x = (const T*)p.logits + row * p.ld + seq * p.seqs.logits + base;
    T* dx = (T*)p.dlogits + row * p.dld + seq * p.seqs.dlogits + base;
    const int cols = p.vocab - base;  // of this segment and what follows
    const float m = p.stats[2 * row], s = p.stats[2 * row + 1];
    const int64_t target = p.targets ? p.targets[row + seq * p.seqs.targets] : -1;
    float dlp = p.dlogprob ? p.dlogprob[row] : 0.0f;
    if (target < 0) dlp = 0.0f;
    const bool past = p.dlogprob && target >= p.vocab;
    if (past) dlp = __builtin_nanf("");
    // a row without a distribution, or without anything to differentiate, has the gradient 0
    const bool zero = (s == 0.0f && !past) || (!ENTROPY && (target < 0 || !p.dlogprob));
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
        const int at = (u * 64 + (int)threadIdx.x) * 8;
        if (!zero) ch[u].template load<false>(x + at, cols - at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = (u * 64 + (int)threadIdx.x) * 8;
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
        store_once(dx + at, cols - at, v);
    }
}

}  // namespace

// Pieces of a row (1: one workgroup takes it whole).  With few rows a workgroup's arithmetic bounds it, a
// batch of its lanes taking 1.5 us, so rows of more than one batch of 1024 lanes are cut into batches of 256
// where four workgroups per compute unit are not there without; the second launch costs 2.5 us.  us without /
// with 20 alternatives: 1 x 131071 4.9 / 9.9, whole 12.6 / 17.5; 1 x 32000 4.6 / 10.0, whole 4.2 / 6.8; 48 x
// 131071 9.6 / 16.2, in pieces twice as large 10.3 / 16.6, in 5 of them 11.9 / 18.1, whole 16.7 / 21.9; 200 x
// 131071 20 / 27, whole 20 / 23.
int lp_splits(int64_t rows, int64_t vocab) {
    if (rows <= 0 || rows >= 512 || vocab <= 32768) return 1;
    const int64_t most = (vocab + 8191) / 8192, wanted = 1024 / rows;
    const int64_t n = wanted < most ? wanted : most;
    return (int)(n < 1 ? 1 : n < kLpMaxSplits ? n : kLpMaxSplits);
}

hipError_t launch_lp(const LpParams& params, hipStream_t stream) {
    LpParams p = params;
    const bool entropy = p.entropy != nullptr, top = p.top > 0;
    p.splits = lp_splits(p.rows, p.vocab);
    p.piece = ((p.vocab + 7) / 8 + p.splits - 1) / p.splits;
    // At least one chunk for each of the groups' lanes, so that the groups bound the best values; few rows in
    // large workgroups, many short ones in single waves (8192 x 2056: 15 us, 26 in four; 1024 x 4096 the
    // same in both, with 20 alternatives 13 and 10).
    const int threads = p.vocab <= 2048 || (p.rows >= 2048 && p.vocab <= 4096) ? 64
                        : p.rows >= 512 || p.vocab < 8192                      ? 256
                                                                               : 1024;
    const bool split = p.splits > 1;
    const void* k = p.f32 ? pick_lp<float>(threads, split, entropy, top) : pick_lp<uint16_t>(threads, split, entropy, top);
    const int64_t groups = p.rows * p.splits;
    for (int64_t g0 = 0; g0 < groups; g0 += kMaxGrid) {
        const int64_t n = groups - g0 < kMaxGrid ? groups - g0 : kMaxGrid;
        void* args[] = {(void*)&p, (void*)&g0};
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)n), dim3(split ? 256 : threads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    if (!split) return hipSuccess;
    int64_t row0 = 0;  // fewer rows than a grid holds are split
    void* args[] = {(void*)&p, (void*)&row0};
    return hipLaunchKernel(p.f32 ? pick_lp_join<float>(top) : pick_lp_join<uint16_t>(top), dim3((unsigned)p.rows), dim3(256),
                           args, 0, stream);
}

hipError_t launch_lp_bwd(const LpBwdParams& p, hipStream_t stream) {
    const uint32_t segs = (uint32_t)((p.vocab + kLpBwdTile - 1) / kLpBwdTile);
    const int64_t rows = kMaxGrid / segs;  // of one launch
    const bool entropy = p.dentropy != nullptr;
    const void* k = p.f32 ? (entropy ? (const void*)&lp_bwd_kernel<float, true> : (const void*)&lp_bwd_kernel<float, false>)
                          : (entropy ? (const void*)&lp_bwd_kernel<uint16_t, true>
                                     : (const void*)&lp_bwd_kernel<uint16_t, false>);
    for (int64_t row0 = 0; row0 < p.rows; row0 += rows) {
        const int64_t n = p.rows - row0 < rows ? p.rows - row0 : rows;
        void* args[] = {(void*)&p, (void*)&row0, (void*)&segs};
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)(n * segs)), dim3(64), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace loco
