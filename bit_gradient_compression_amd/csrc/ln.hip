// Layer norm, forward and backward.
//
// Forward, per row: mu = mean x, r = 1/sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b.
// Backward: xh = (x - mu) r, g = dy w, dx = r (g - mean g - xh mean(g xh)) [+ residual],
// dw = sum over rows of dy xh, db = sum over rows of dy.
//
// Both are bound by HBM: each element is read once and written once.  A row stays in
// registers between the statistics and the output: forward one wave holds up to 1024 columns,
// four or eight waves together a wider row.  All sums are fp32; the
// variance is the mean of squared differences from the mean, not a difference of squares.
// Measured at 16384 x 4096 in bf16: forward 51 us (5.2 TB/s, as torch's copy of the same
// bytes), 67 with a checkpoint of y; backward with a residual 110 (5.0 TB/s).  In fp32: forward
// 100 us (5.4 TB/s), backward without a residual 167 (4.8).  The smallest calls take one launch's
// 4 us.

#include "loco_layer.hpp"
#include "loco_layer_internal.hpp"

namespace loco {

namespace {

// Sum over the WPR waves of a row; every lane gets it.  `slot` alternates between calls so
// that one barrier per call is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red, int slot) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[slot * WPR + wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += red[slot * WPR + i];
    }
    return v;
}

__device__ __forceinline__ int chunk_valid(int cols, int c) { return cols - c < 8 ? cols - c : 8; }

// ---- forward --------------------------------------------------------------------------

// WPR waves per row, NP chunks of eight per lane.  The grid is not persistent: what hides the
// latencies of a row is the other rows on the compute unit, so registers are spent on as many
// waves as fit and not on the next row's loads.
template <typename T, int WPR, int NP>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void ln_kernel(const LnParams p, int64_t row0) {
    __shared__ float red[2 * WPR];
    constexpr int RPW = WPR == 1 ? 4 : 1;  // rows per workgroup
    constexpr int LANES = WPR * 64;
    const int64_t row = row0 + (int64_t)blockIdx.x * RPW + (WPR == 1 ? uniform(threadIdx.x >> 6) : 0);
    if (row >= p.rows) return;  // whole waves (WPR == 1: no barrier follows)
    const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int cols = p.cols;
    const float inv_cols = 1.0f / (float)cols;
    const T* x = (const T*)p.x + row * cols;
    RawChunk<T> raw[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = (i * LANES + lane) * 8;
        raw[i].load(x + c, chunk_valid(cols, c));
    }
    float v[8], sum = 0.0f, sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[j];
    }
    const float mean = row_sum<WPR>(sum, red, 0) * inv_cols;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int valid = chunk_valid(cols, (i * LANES + lane) * 8);
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v[j] - mean;
            sq = j < valid ? __builtin_fmaf(d, d, sq) : sq;
        }
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<WPR>(sq, red, 1) * inv_cols + p.eps);
    if (lane == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    T* y = (T*)p.y + row * cols;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = (i * LANES + lane) * 8;
        const int valid = chunk_valid(cols, c);
        float w[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 1.0f;
            b[j] = 0.0f;
        }
        if (p.w) load_chunk_any(p.w, p.param_f32, c, valid, w);
        if (p.b) load_chunk_any(p.b, p.param_f32, c, valid, b);
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < valid ? __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]) : 0.0f;
        store_chunk(y + c, valid, v);
        if (p.ckpt.codes) {
            // of y in fp32, before its rounding to the output's type
            const uint32_t e = ckpt_exp(block_top(v, p.ckpt.block64));
            store_codes(p.ckpt.codes + row * cols + c, valid, ckpt_codes(v, e));
            const int per = p.ckpt.block64 ? 8 : 4;
            if ((lane & (per - 1)) == 0 && valid > 0)
                p.ckpt.exps[row * p.ckpt.nblocks + c / (8 * per)] = (uint8_t)e;
        }
    }
}

struct LnShape {
    int wpr, np;
};
// 32 to 64 bytes per lane up to 8192 columns: fewer leave too little in flight, more leave room
// for too few waves (16384 x 4096 in bf16: 51 us with 32 bytes, 59 with 16, 62 with 128).
LnShape ln_shape(bool f32, int64_t cols) {
    if (cols <= 512) return {1, 1};
    if (cols <= 1024) return {1, 2};
    if (cols <= 2048) return {4, 1};
    if (cols <= 4096) return f32 ? LnShape{8, 1} : LnShape{4, 2};
    if (cols <= 6144 && !f32) return {4, 3};
    if (cols <= 8192) return f32 ? LnShape{8, 2} : LnShape{4, 4};
    if (cols <= 12288) return {8, 3};
    return {8, 4};
}
template <typename T>
const void* pick_ln(LnShape s) {
    switch (s.wpr * 16 + s.np) {
        case 16 + 1: return (const void*)&ln_kernel<T, 1, 1>;
        case 16 + 2: return (const void*)&ln_kernel<T, 1, 2>;
        case 64 + 1: return (const void*)&ln_kernel<T, 4, 1>;
        case 128 + 3: return (const void*)&ln_kernel<T, 8, 3>;
        case 128 + 4: return (const void*)&ln_kernel<T, 8, 4>;
    }
    if constexpr (sizeof(T) == 4) {
        return s.np == 1 ? (const void*)&ln_kernel<T, 8, 1> : (const void*)&ln_kernel<T, 8, 2>;
    } else {
        return s.np == 2   ? (const void*)&ln_kernel<T, 4, 2>
               : s.np == 3 ? (const void*)&ln_kernel<T, 4, 3>
                           : (const void*)&ln_kernel<T, 4, 4>;
    }
}

// ---- backward -------------------------------------------------------------------------
//
// A workgroup of WAVES waves works TEAMS = WAVES / WPR rows at a time and keeps the sums of dw
// and db over all its rows in registers; at the end the teams' sums meet in LDS and one
// partial sum per workgroup goes to memory, to be joined by a second kernel.  Large workgroups
// keep those few: at 16384 x 4096 1024 workgroups of one row wrote and read 66 MB of them beside
// 403 MB of work, 256 of four rows a quarter.  With few rows they weigh more: 1023 x 2047 in fp32
// leaves 8.4 MB of them, as much as x, and takes 11 us here (30 % of the LDS cycles are conflicts
// of the teams' join) and 5 in the join.

template <typename T, int WPR, int NP, int WAVES>
__global__ __launch_bounds__(WAVES * 64, NP == 1 ? 6 : NP == 2 ? 4 : 2) void ln_bwd_kernel(const LnBwdParams p) {
    constexpr int TEAMS = WAVES / WPR;
    constexpr int LANES = WPR * 64;
    constexpr int COLS = NP * LANES * 8;
    // the residual is loaded with x and dy where that costs no workgroup its place
    constexpr bool EARLY = NP >= 3 || (NP == 2 && (WPR == 1 || (WPR == 4 && sizeof(T) == 2)));
    __shared__ float red[2][2][WAVES];
    __shared__ float join[TEAMS > 1 ? TEAMS * COLS : 1];
    const int wave = uniform(threadIdx.x >> 6), team = wave / WPR;
    const int lane = threadIdx.x - team * LANES;
    const int cols = p.cols;
    const float inv_cols = 1.0f / (float)cols;
    float dw[NP][8], db[NP][8];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
    RawChunk<T> x[NP], dy[NP], res[NP];
    // every team takes part in every turn's barrier, with or without a row
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t row = (int64_t)blockIdx.x * TEAMS + team;
    for (int flip = 0; row - team < p.rows; row += step, flip ^= 1) {
        const bool here = row < p.rows;
        const void* weight = p.w;
        // w is read again for each row where keeping it would cost another workgroup its registers
        if (NP == 2) asm("" : "+s"(weight));
        const float mean = here ? p.mean[row] : 0.0f, rstd = here ? p.rstd[row] : 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            const int valid = here ? chunk_valid(cols, c) : 0;
            x[i].load((const T*)p.x + row * cols + c, valid);
            dy[i].load((const T*)p.dy + row * cols + c, valid);
            if (EARLY && p.residual) res[i].load((const T*)p.residual + row * cols + c, valid);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float w[8], v[8], g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            const int c = (i * LANES + lane) * 8;
            const int valid = chunk_valid(cols, c);
            if (weight) load_chunk_any(weight, p.param_f32, c, valid, w);
            x[i].get(v);
            dy[i].get(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // Past the row's end dy is 0, and xh has to be finite for its products with it to count
                // for nothing: -mean * rstd may overflow.
                const float xh = j < valid ? (v[j] - mean) * rstd : 0.0f;
                dw[i][j] = __builtin_fmaf(g[j], xh, dw[i][j]);
                db[i][j] += g[j];
                const float gw = g[j] * w[j];
                s1 += gw;
                s2 = __builtin_fmaf(gw, xh, s2);
            }
        }
        // two sums through one barrier; the slots alternate from turn to turn
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0) {
                red[flip][0][wave] = s1;
                red[flip][1][wave] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                s1 += red[flip][0][team * WPR + i];
                s2 += red[flip][1][team * WPR + i];
            }
        }
        if (!here) continue;
        s1 *= inv_cols;
        s2 *= inv_cols;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            const int valid = chunk_valid(cols, c);
            float w[8], v[8], g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            if (weight) load_chunk_any(weight, p.param_f32, c, valid, w);
            x[i].get(v);
            dy[i].get(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // the sums' expression, so that its value is kept: another one takes 14 registers more
                const float xh = j < valid ? (v[j] - mean) * rstd : 0.0f;
                g[j] = (g[j] * w[j] - s1 - xh * s2) * rstd;
            }
            if (p.residual) {
                if (!EARLY) res[i].load((const T*)p.residual + row * cols + c, valid);
                res[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] += v[j];
            }
            store_chunk((T*)p.dx + row * cols + c, valid, g);
        }
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if constexpr (TEAMS > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            if constexpr (TEAMS > 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) join[team * COLS + c + j] = which ? db[i][j] : dw[i][j];
            } else if (which) {
                store_chunk(part + cols + c, chunk_valid(cols, c), db[i]);
            } else {
                store_chunk(part + c, chunk_valid(cols, c), dw[i]);
            }
        }
        if constexpr (TEAMS > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += WAVES * 64) {
                float s = 0.0f;
#pragma unroll
                for (int t = 0; t < TEAMS; ++t) s += join[t * COLS + c];
                part[which * cols + c] = s;
            }
        }
    }
}

// dw[c] and db[c] from the groups' partial sums: 32 columns per workgroup, 32 threads down
// the groups, joined in LDS in a fixed order.
__global__ __launch_bounds__(1024) void ln_bwd_join_kernel(const LnBwdParams p, int64_t groups) {
    __shared__ float s[2][32][33];
    const int cl = threadIdx.x & 31, g0 = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    float dw = 0.0f, db = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t g = g0; g < groups; g += 32) {
            dw += p.part[(g * 2 + 0) * p.cols + c];
            db += p.part[(g * 2 + 1) * p.cols + c];
        }
    }
    s[0][g0][cl] = dw;
    s[1][g0][cl] = db;
    __syncthreads();
    if (threadIdx.x < 64) {
        const int which = threadIdx.x >> 5;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s[which][i][cl];
        void* out = which ? p.db : p.dw;
        if (out && c < p.cols) {
            if (p.grad_f32) ((float*)out)[c] = v;
            else ((uint16_t*)out)[c] = bf16_rne(v);
        }
    }
}

struct LnBwdShape {
    int wpr, np, waves, groups;  // groups: the workgroups that are at work at once
};
LnBwdShape ln_bwd_shape(int64_t cols) {
    if (cols <= 512) return {1, 1, 8, 768};
    if (cols <= 1024) return {1, 2, 16, 256};
    if (cols <= 2048) return {4, 1, 8, 768};
    if (cols <= 4096) return {4, 2, 16, 256};
    if (cols <= 8192) return {8, 2, 16, 256};
    if (cols <= 12288) return {8, 3, 8, 256};
    return {8, 4, 8, 256};
}
template <typename T>
const void* pick_ln_bwd(LnBwdShape s) {
    switch (s.wpr * 16 + s.np) {
        case 16 + 1: return (const void*)&ln_bwd_kernel<T, 1, 1, 8>;
        case 16 + 2: return (const void*)&ln_bwd_kernel<T, 1, 2, 16>;
        case 64 + 1: return (const void*)&ln_bwd_kernel<T, 4, 1, 8>;
        case 64 + 2: return (const void*)&ln_bwd_kernel<T, 4, 2, 16>;
        case 128 + 2: return (const void*)&ln_bwd_kernel<T, 8, 2, 16>;
        case 128 + 3: return (const void*)&ln_bwd_kernel<T, 8, 3, 8>;
    }
    return (const void*)&ln_bwd_kernel<T, 8, 4, 8>;
}

}  // namespace

hipError_t launch_ln(const LnParams& p, hipStream_t stream) {
    const LnShape s = ln_shape(p.f32, p.cols);
    const int rpw = s.wpr == 1 ? 4 : 1, threads = s.wpr == 1 ? 256 : s.wpr * 64;
    const void* k = p.f32 ? pick_ln<float>(s) : pick_ln<uint16_t>(s);
    for (int64_t row0 = 0; row0 < p.rows; row0 += kMaxGrid * rpw) {
        const int64_t rows = p.rows - row0 < kMaxGrid * rpw ? p.rows - row0 : kMaxGrid * rpw;
        void* args[] = {(void*)&p, (void*)&row0};
        const hipError_t err =
            hipLaunchKernel(k, dim3((unsigned)((rows + rpw - 1) / rpw)), dim3(threads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

int64_t ln_bwd_groups(int64_t rows, int64_t cols) {
    const LnBwdShape s = ln_bwd_shape(cols);
    const int64_t teams = s.waves / s.wpr, wanted = (rows + teams - 1) / teams;
    return wanted < 1 ? 1 : wanted < s.groups ? wanted : s.groups;
}

hipError_t launch_ln_bwd(const LnBwdParams& p, hipStream_t stream) {
    const LnBwdShape s = ln_bwd_shape(p.cols);
    const int64_t groups = ln_bwd_groups(p.rows, p.cols);
    const void* k = p.f32 ? pick_ln_bwd<float>(s) : pick_ln_bwd<uint16_t>(s);
    void* args[] = {(void*)&p};
    hipError_t err = hipLaunchKernel(k, dim3((unsigned)groups), dim3(s.waves * 64), args, 0, stream);
    if (err != hipSuccess || !p.part) return err;
    void* jargs[] = {(void*)&p, (void*)&groups};
    return hipLaunchKernel((const void*)&ln_bwd_join_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), jargs, 0,
                           stream);
}

}  // namespace loco
