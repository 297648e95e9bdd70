// Layer norm, forward and backward.
//
// Forward, per row: mu = mean x, r = 1/sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b.
// Backward: xh = (x - mu) r, g = dy w, dx = r (g - mean g - xh mean(g xh)) [+ residual],
// dw = sum over rows of dy xh, db = sum over rows of dy.
//
// Both are bound by HBM: each element is read once and written once.  A row stays in
// registers between the statistics and the output: one wave holds up to 4096 columns in
// the forward pass, a workgroup of four or eight waves wider rows.  All sums are fp32; the
// variance is the mean of squared differences from the mean, not a difference of squares.

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

template <typename T, int WPR, int NP>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void ln_kernel(const LnParams p, int64_t row0) {
    __shared__ float red[2 * (WPR > 1 ? WPR : 1)];
    constexpr int RPW = WPR == 1 ? 4 : 1;  // rows per workgroup
    constexpr int LANES = WPR * 64;
    const int64_t row = row0 + (int64_t)blockIdx.x * RPW + (WPR == 1 ? uniform(threadIdx.x >> 6) : 0);
    if (row >= p.rows) return;  // whole waves (WPR == 1: no barrier follows)
    const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int cols = p.cols;
    const T* x = (const T*)p.x + row * cols;
    float v[NP][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = (i * LANES + lane) * 8;
        load_chunk(x + c, chunk_valid(cols, c), v[i]);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[i][j];
    const float mean = row_sum<WPR>(sum, red, 0) / (float)cols;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int valid = chunk_valid(cols, (i * LANES + lane) * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] -= mean;
            sq = j < valid ? __builtin_fmaf(v[i][j], v[i][j], sq) : sq;
        }
    }
    const float var = row_sum<WPR>(sq, red, 1) / (float)cols;
    const float rstd = 1.0f / __builtin_sqrtf(var + p.eps);
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
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = j < valid ? __builtin_fmaf(v[i][j] * rstd, w[j], b[j]) : 0.0f;
        store_chunk(y + c, valid, v[i]);
        if (p.ckpt.codes) {
            // of y in fp32, before its rounding to the output's type
            const uint32_t e = ckpt_exp(block_top(v[i], p.ckpt.block64));
            store_codes(p.ckpt.codes + row * cols + c, valid, ckpt_codes(v[i], e));
            const int per = p.ckpt.block64 ? 8 : 4;
            if ((lane & (per - 1)) == 0 && valid > 0)
                p.ckpt.exps[row * p.ckpt.nblocks + c / (8 * per)] = (uint8_t)e;
        }
    }
}

template <typename T>
const void* pick_ln(int cols) {
    if (cols <= 512) return (const void*)&ln_kernel<T, 1, 1>;
    if (cols <= 1024) return (const void*)&ln_kernel<T, 1, 2>;
    if (cols <= 2048) return (const void*)&ln_kernel<T, 4, 1>;
    if (cols <= 4096) return (const void*)&ln_kernel<T, 4, 2>;
    if (cols <= 8192) return (const void*)&ln_kernel<T, 4, 4>;
    return (const void*)&ln_kernel<T, 8, 4>;
}

// ---- backward -------------------------------------------------------------------------

template <typename T, int WPR, int NP>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void ln_bwd_kernel(const LnBwdParams p) {
    constexpr int RPW = WPR == 1 ? 4 : 1;
    constexpr int LANES = WPR * 64;
    constexpr int COLS = NP * LANES * 8;
    __shared__ float red[4 * (WPR > 1 ? WPR : 1)];
    __shared__ float join[WPR == 1 ? 4 * COLS : 1];
    const int wave = uniform(threadIdx.x >> 6);
    const int lane = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int cols = p.cols;
    const float inv_cols = 1.0f / (float)cols;
    float w[NP][8], dw[NP][8], db[NP][8];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = (i * LANES + lane) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[i][j] = 1.0f;
            dw[i][j] = 0.0f;
            db[i][j] = 0.0f;
        }
        if (p.w) load_chunk_any(p.w, p.param_f32, c, chunk_valid(cols, c), w[i]);
    }
    const int64_t step = (int64_t)gridDim.x * RPW;
    int flip = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPW + (WPR == 1 ? wave : 0); row < p.rows; row += step) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float g[NP][8], xh[NP][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            const int valid = chunk_valid(cols, c);
            load_chunk((const T*)p.x + row * cols + c, valid, xh[i]);
            load_chunk((const T*)p.dy + row * cols + c, valid, g[i]);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // past the row's end g is 0, so whatever xh is there counts for nothing
                xh[i][j] = (xh[i][j] - mean) * rstd;
                dw[i][j] = __builtin_fmaf(g[i][j], xh[i][j], dw[i][j]);
                db[i][j] += g[i][j];
                g[i][j] *= w[i][j];
                s1 += g[i][j];
                s2 = __builtin_fmaf(g[i][j], xh[i][j], s2);
            }
        // two sums through one barrier; the slots alternate from row to row
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0) {
                red[(flip * 2 + 0) * WPR + wave] = s1;
                red[(flip * 2 + 1) * WPR + wave] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                s1 += red[(flip * 2 + 0) * WPR + i];
                s2 += red[(flip * 2 + 1) * WPR + i];
            }
            flip ^= 1;
        }
        s1 *= inv_cols;
        s2 *= inv_cols;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            const int valid = chunk_valid(cols, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = (g[i][j] - s1 - xh[i][j] * s2) * rstd;
            if (p.residual) {
                float r[8];
                load_chunk((const T*)p.residual + row * cols + c, valid, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] += r[j];
            }
            store_chunk((T*)p.dx + row * cols + c, valid, g[i]);
        }
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = (i * LANES + lane) * 8;
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = which ? db[i][j] : dw[i][j];
            if constexpr (WPR == 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) join[wave * COLS + c + j] = s[j];
            } else {
                store_chunk(part + which * cols + c, chunk_valid(cols, c), s);
            }
        }
        if constexpr (WPR == 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += 256)
                part[which * cols + c] = (join[c] + join[COLS + c]) + (join[2 * COLS + c] + join[3 * COLS + c]);
            __syncthreads();
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
    int wpr, np;
};
LnBwdShape ln_bwd_shape(int64_t cols) {
    if (cols <= 512) return {1, 1};
    if (cols <= 1024) return {1, 2};
    if (cols <= 2048) return {4, 1};
    if (cols <= 4096) return {4, 2};
    if (cols <= 8192) return {8, 2};
    return {8, 4};
}
template <typename T>
const void* pick_ln_bwd(LnBwdShape s) {
    if (s.wpr == 1) return s.np == 1 ? (const void*)&ln_bwd_kernel<T, 1, 1> : (const void*)&ln_bwd_kernel<T, 1, 2>;
    if (s.wpr == 4) return s.np == 1 ? (const void*)&ln_bwd_kernel<T, 4, 1> : (const void*)&ln_bwd_kernel<T, 4, 2>;
    return s.np == 2 ? (const void*)&ln_bwd_kernel<T, 8, 2> : (const void*)&ln_bwd_kernel<T, 8, 4>;
}

}  // namespace

hipError_t launch_ln(const LnParams& p, hipStream_t stream) {
    const int wpr = p.cols <= 1024 ? 1 : p.cols <= 8192 ? 4 : 8;
    const int rpw = wpr == 1 ? 4 : 1, threads = wpr == 1 ? 256 : wpr * 64;
    const void* k = p.f32 ? pick_ln<float>(p.cols) : pick_ln<uint16_t>(p.cols);
    for (int64_t row0 = 0; row0 < p.rows; row0 += kMaxGrid * rpw) {
        const int64_t rows = p.rows - row0 < kMaxGrid * rpw ? p.rows - row0 : kMaxGrid * rpw;
        void* args[] = {(void*)&p, (void*)&row0};
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)((rows + rpw - 1) / rpw)), dim3(threads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

int64_t ln_bwd_groups(int64_t rows, int64_t cols) {
    const int64_t wanted = ln_bwd_shape(cols).wpr == 1 ? (rows + 3) / 4 : rows;
    const int64_t most = 1024;
    return wanted < 1 ? 1 : wanted < most ? wanted : most;
}

hipError_t launch_ln_bwd(const LnBwdParams& p, hipStream_t stream) {
    const LnBwdShape s = ln_bwd_shape(p.cols);
    const int64_t groups = ln_bwd_groups(p.rows, p.cols);
    const void* k = p.f32 ? pick_ln_bwd<float>(s) : pick_ln_bwd<uint16_t>(s);
    void* args[] = {(void*)&p};
    hipError_t err = hipLaunchKernel(k, dim3((unsigned)groups), dim3(s.wpr == 1 ? 256 : s.wpr * 64), args, 0, stream);
    if (err != hipSuccess || !p.part) return err;
    void* jargs[] = {(void*)&p, (void*)&groups};
    return hipLaunchKernel((const void*)&ln_bwd_join_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), jargs, 0,
                           stream);
}

}  // namespace loco
