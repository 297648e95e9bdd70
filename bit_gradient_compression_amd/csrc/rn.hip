// The norms around a transformer block, fused with its gate and residual, forward and backward.
//
// Forward, per row: rp = 1/sqrt(mean y^2 + eps), u = y rp wp (or u = y); h = residual + s g u;
// r = 1/sqrt(mean h^2 + eps), out = h r w.  Backward, with xh = h r and yh = y rp:
//   dh' = dh + r (dout w - xh mean(dout w xh))            the gradient of h, and of the residual
//   dy  = rp (t - yh mean(t yh)),  t = s g dh' wp         (or dy = s g dh')
//   dw = sum over rows of dout xh,  dwp = sum of s g dh' yh,  dg = s dh' u, summed for a gate of columns
//
// Both are bound by HBM: each element is read once and written once, but for fp32 rows past 8192 columns
// backward, which read h, dout and y again for the phase that needs them.  A row stays in registers from
// its loads to its stores, through both of its sums; all sums are fp32.
//
// Times here are of calls one after another whose matrices change from call to call, unless they say "the same
// buffers": then the caches hold some of them.  16384 x 4096 in bf16 with a gate of columns: forward 97 us
// (5.5 TB/s), 108 with the checkpoint (5.6 TB/s); backward 152 us (5.4 TB/s), 5 of them for the join.  Past 8192
// columns they are further from the copy's 6.4 TB/s: 4096 x 11008 takes 81 us forward (4.4 TB/s: a third of
// the lanes' chunks is empty) and 154 backward (3.5 TB/s: a row waits for its own loads).

#include "loco_layer.hpp"
#include "loco_step_internal.hpp"

namespace loco {

namespace {

// Sum over the LPT lanes of a row; every lane gets it.  `slot` alternates between calls so that one
// barrier per call is enough.
template <int LPT>
__device__ __forceinline__ float row_sum(float v, float* red, int slot) {
    v = lanes_sum<LPT < 64 ? LPT : 64>(v);
    if constexpr (LPT > 64) {
        constexpr int WPR = LPT / 64;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[slot * WPR + wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += red[slot * WPR + i];
    }
    return v;
}

__device__ __forceinline__ void fill(float (&v)[8], float x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x;
}

// ---- forward --------------------------------------------------------------------------

// Where a lane's chunk lies in a row: `valid` elements, 0 to 8, from column c on.  WHOLE: all of a chunk or
// nothing.  Else a chunk of which less than all exists is read as the row's last eight elements (`at`), of which
// `shift` are dropped when they are there: element by element, or in parts that are put together where they are
// loaded, one matrix waited for the one before it (16384 x 4095 in bf16 with a checkpoint, the same buffers, 236
// and 176 us, so 149; 8192 x 4095 in fp32 109, 114 and 107; only a last chunk alone in its wave is slower, 4097
// in fp32 116, 117 and 136).
struct Place {
    int c, at, valid, shift;
};
template <bool WHOLE>
__device__ __forceinline__ Place place_of(int c, int cols, bool here) {
    const int valid = !here || c >= cols ? 0 : WHOLE || cols - c >= 8 ? 8 : cols - c;
    const int at = WHOLE || valid == 8 || cols < 8 ? c : cols - 8;
    return {c, at, valid, WHOLE || valid == 0 ? 0 : c - at};
}

// A chunk as it lies in memory; elements that do not exist are 0 after `fix`.
template <typename T, bool WHOLE>
struct RowChunk;
template <bool WHOLE>
struct RowChunk<uint16_t, WHOLE> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t* row, int cols, const Place& q) {
        w = u32x4{0u, 0u, 0u, 0u};
        if (!WHOLE && cols < 8) {
            if (q.valid)
                for (int j = 0; j < cols; ++j) {
                    const uint32_t x = (uint32_t)row[j] << (16 * (j & 1));
                    w.x |= j < 2 ? x : 0u;
                    w.y |= j >> 1 == 1 ? x : 0u;
                    w.z |= j >> 1 == 2 ? x : 0u;
                    w.w |= j >> 1 == 3 ? x : 0u;
                }
        } else if (q.valid) {
            w = load16(row + q.at);
        }
    }
    __device__ __forceinline__ void fix(const Place& q) {
        if (!WHOLE && q.shift) {
            if (q.shift & 4) w = u32x4{w.z, w.w, 0u, 0u};
            if (q.shift & 2) w = u32x4{w.y, w.z, w.w, 0u};
            if (q.shift & 1)
                w = u32x4{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_bf16x8(w, v); }
    static __device__ __forceinline__ void store(uint16_t* row, const Place& q, const float (&v)[8], bool once) {
        uint16_t* p = row + q.c;
        const u32x4 x = pack_bf16x8(v);
        if (q.valid == 8) {
            if (once) stream16(p, x);
            else store16(p, x);
        } else if (!WHOLE && q.valid > 0) {
            const uint32_t r0 = q.valid & 4 ? x[2] : x[0], r1 = q.valid & 4 ? x[3] : x[1];
            const u32x2 four = {x[0], x[1]};
            if (q.valid & 4) __builtin_memcpy(p, &four, 8);
            if (q.valid & 2) __builtin_memcpy(p + (q.valid & 4), &r0, 4);
            if (q.valid & 1) p[q.valid & 6] = (uint16_t)(q.valid & 2 ? r1 : r0);
        }
    }
};
template <bool WHOLE>
struct RowChunk<float, WHOLE> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* row, int cols, const Place& q) {
        a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!WHOLE && cols < 8) {
            if (q.valid)
                for (int j = 0; j < cols; ++j) {
                    const float x = row[j];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        a[k] = j == k ? x : a[k];
                        b[k] = j == 4 + k ? x : b[k];
                    }
                }
        } else if (q.valid) {
            __builtin_memcpy(&a, row + q.at, 16);
            __builtin_memcpy(&b, row + q.at + 4, 16);
        }
    }
    __device__ __forceinline__ void fix(const Place& q) {
        if (!WHOLE && q.shift) {
            if (q.shift & 4) {
                a = b;
                b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            if (q.shift & 2) {
                a = f32x4{a[2], a[3], b[0], b[1]};
                b = f32x4{b[2], b[3], 0.0f, 0.0f};
            }
            if (q.shift & 1) {
                a = f32x4{a[1], a[2], a[3], b[0]};
                b = f32x4{b[1], b[2], b[3], 0.0f};
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    }
    static __device__ __forceinline__ void store(float* row, const Place& q, const float (&v)[8], bool once) {
        float* p = row + q.c;
        const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        if (q.valid == 8) {
            if (once) {
                stream16(p, __builtin_bit_cast(u32x4, a));
                stream16(p + 4, __builtin_bit_cast(u32x4, b));
            } else {
                __builtin_memcpy(p, &a, 16);
                __builtin_memcpy(p + 4, &b, 16);
            }
        } else if (!WHOLE && q.valid > 0) {
            const f32x4 r = q.valid & 4 ? b : a;
            const float two[2] = {r[0], r[1]};
            if (q.valid & 4) __builtin_memcpy(p, &a, 16);
            if (q.valid & 2) __builtin_memcpy(p + (q.valid & 4), two, 8);
            if (q.valid & 1) p[q.valid & 6] = q.valid & 2 ? r[2] : r[0];
        }
    }
};
// The same of a parameter vector, whose type is known at run time only.
template <bool WHOLE>
__device__ __forceinline__ void get_chunk(const void* base, bool f32, int cols, const Place& q, float (&v)[8]) {
    if (f32) {
        RowChunk<float, WHOLE> x;
        x.load((const float*)base, cols, q);
        x.fix(q);
        x.get(v);
    } else {
        RowChunk<uint16_t, WHOLE> x;
        x.load((const uint16_t*)base, cols, q);
        x.fix(q);
        x.get(v);
    }
}
template <bool WHOLE>
__device__ __forceinline__ void store_row_codes(int8_t* p, int valid, u32x2 w) {
    if (valid == 8) {
        stream8(p, w);
    } else if (!WHOLE && valid > 0) {
        const uint32_t four = w.x, r = valid & 4 ? w.y : w.x;
        const uint16_t two = (uint16_t)r;
        if (valid & 4) __builtin_memcpy(p, &four, 4);
        if (valid & 2) __builtin_memcpy(p + (valid & 4), &two, 2);
        if (valid & 1) p[valid & 6] = (int8_t)(valid & 2 ? r >> 16 : r);
    }
}

// 1 / sqrt(x), within an ulp as the hardware's is.  That takes normal numbers only.
__device__ __forceinline__ float inv_root(float x) {
    const bool small = x < 0x1p-96f;
    return __builtin_amdgcn_rsqf(small ? x * 0x1p64f : x) * (small ? 0x1p32f : 1.0f);
}

// LPT lanes per row, NP chunks of eight per lane.  WHOLE: rows are whole chunks, and a lane has all of a
// chunk or nothing.  Past a row's end every value is 0 and stays it: a norm's factor, which may be infinite,
// is made 0 there.
template <typename T, int LPT, int NP, bool WHOLE>
__global__ __launch_bounds__(LPT <= 64 ? 256 : LPT) void rn_kernel(const RnParams p, int64_t row0, bool once) {
    __shared__ float red[LPT <= 64 ? 1 : 2 * LPT / 64];
    constexpr int LANES = LPT;
    constexpr int RPW = LPT <= 64 ? 256 / LPT : 1;  // rows per workgroup
    int64_t row = row0 + (int64_t)blockIdx.x * RPW;
    if constexpr (LPT == 64) row += uniform(threadIdx.x >> 6);
    else row += threadIdx.x / LPT;
    if (LPT >= 64 && row >= p.rows) return;  // whole waves (LPT == 64: no barrier follows)
    // rows of part of a wave: the others go on, with nothing to read or write
    const bool here = row < p.rows;
    const int lane = threadIdx.x % LPT;
    const int cols = p.cols;
    const float inv_cols = 1.0f / (float)cols;
    const auto place = [&](int i) { return place_of<WHOLE>((i * LANES + lane) * 8, cols, here); };
    using Chunk = RowChunk<T, WHOLE>;
    Chunk y[NP], res[NP], gate[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const Place q = place(i);
        if (p.y) y[i].load((const T*)p.y + row * cols, cols, q);
        if (p.residual) res[i].load((const T*)p.residual + row * cols, cols, q);
        if (p.gate_kind == kGateElement) gate[i].load((const T*)p.gate + row * cols, cols, q);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const Place q = place(i);
        if (p.y) y[i].fix(q);
        if (p.residual) res[i].fix(q);
        if (p.gate_kind == kGateElement) gate[i].fix(q);
    }
    float v[8], h[NP][8];
    float rp = 1.0f;
    if (p.post_rstd) {
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            y[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[j], v[j], sq);
        }
        rp = inv_root(row_sum<LPT>(sq, red, 0) * inv_cols + p.eps);
        if (lane == 0 && here) p.post_rstd[row] = rp;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const Place q = place(i);
        fill(h[i], 0.0f);
        if (p.residual) res[i].get(h[i]);
        if (p.y) {
            float k[8], w[8];
            fill(k, p.scale);
            if (p.gate_kind != kGateNone) {
                if (p.gate_kind == kGateElement) gate[i].get(w);
                else get_chunk<WHOLE>(p.gate, p.param_f32, cols, q, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] *= w[j];
            }
            y[i].get(v);
            if (p.post_rstd) {
                fill(w, 1.0f);
                if (p.post_weight) get_chunk<WHOLE>(p.post_weight, p.param_f32, cols, q, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * (WHOLE ? q.valid ? rp : 0.0f : j < q.valid ? rp : 0.0f) * w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = __builtin_fmaf(k[j], v[j], h[i][j]);
        }
        if (p.h) Chunk::store((T*)p.h + row * cols, q, h[i], once);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(h[i][j], h[i][j], sq);
    }
    if (!p.out) return;  // the whole grid
    const float r = inv_root(row_sum<LPT>(sq, red, 1) * inv_cols + p.eps);
    if (lane == 0 && here) p.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const Place q = place(i);
        float w[8];
        fill(w, 1.0f);
        if (p.weight) get_chunk<WHOLE>(p.weight, p.param_f32, cols, q, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[i][j] * (WHOLE ? q.valid ? r : 0.0f : j < q.valid ? r : 0.0f) * w[j];
        Chunk::store((T*)p.out + row * cols, q, v, once);
        if (p.ckpt.codes) {
            // of the fp32 values, before their rounding to the output's type
            const uint32_t e = ckpt_exp(block_top(v, p.ckpt.block64));
            store_row_codes<WHOLE>(p.ckpt.codes + row * cols + q.c, q.valid, ckpt_codes(v, e));
            const int per = p.ckpt.block64 ? 8 : 4;
            if ((lane & (per - 1)) == 0 && q.valid > 0)
                p.ckpt.exps[row * p.ckpt.nblocks + q.c / (8 * per)] = (uint8_t)e;
        }
    }
}

struct RnShape {
    int lpt, np;
};
// 16 to 32 bytes of each matrix per lane.  The shape does not depend on the rows, so that a token's bits do
// not depend on what else is in its batch.  us: 16384 x 4096 in bf16 from y and residual / of the residual
// alone 98 / 53 with 512 lanes, 99 / 44 with 256, 110 / 51 with 128; one row 3.7, 4.7, 6.6; 8192 x 4096 in fp32
// 100, 108, 114; 8192 x 8192 in bf16 102 with 1024, 99 with 512, 107 with 256; 4096 x 8192 in fp32 102, 106, 113.
RnShape rn_shape(int64_t cols, bool f32, bool alone) {
    if (cols <= 128) return {16, 1};
    if (cols <= 256) return {32, 1};
    if (cols <= 512) return {64, 1};
    if (cols <= 1024) return {64, 2};
    if (cols <= 2048) return {256, 1};
    if (cols <= 4096) return f32 || !alone ? RnShape{512, 1} : RnShape{256, 2};
    if (cols <= 8192) return f32 ? RnShape{1024, 1} : RnShape{512, 2};
    return {512, 4};
}
template <typename T, bool WHOLE>
const void* pick_rn(RnShape s) {
    switch (s.lpt * 8 + s.np) {
        case 16 * 8 + 1: return (const void*)&rn_kernel<T, 16, 1, WHOLE>;
        case 32 * 8 + 1: return (const void*)&rn_kernel<T, 32, 1, WHOLE>;
        case 64 * 8 + 1: return (const void*)&rn_kernel<T, 64, 1, WHOLE>;
        case 64 * 8 + 2: return (const void*)&rn_kernel<T, 64, 2, WHOLE>;
        case 256 * 8 + 1: return (const void*)&rn_kernel<T, 256, 1, WHOLE>;
        case 512 * 8 + 1: return (const void*)&rn_kernel<T, 512, 1, WHOLE>;
    }
    if constexpr (sizeof(T) == 4) {
        if (s.lpt == 1024) return (const void*)&rn_kernel<T, 1024, 1, WHOLE>;
    } else {
        if (s.np == 2) return s.lpt == 256 ? (const void*)&rn_kernel<T, 256, 2, WHOLE> : (const void*)&rn_kernel<T, 512, 2, WHOLE>;
    }
    return (const void*)&rn_kernel<T, 512, 4, WHOLE>;
}

// ---- backward -------------------------------------------------------------------------
//
// A workgroup of WAVES waves works TEAMS = WAVES / WPR rows at a time and keeps the column sums over
// all its rows: dweight's in registers, the other two in LDS, where each lane has its own columns
// (all three in registers leave room for too few rows at a time).  At the end the teams' sums meet in
// LDS and one partial sum per workgroup goes to memory, to be joined by a second kernel in a fixed
// order.
//
// A lane holds NP whole chunks of eight columns and, in the first lanes of a team, one of the up to
// seven columns past the last whole chunk.  All of them are moved through buffer resources over the
// row's whole chunks, or over its tail: the address is a scalar base and a 32-bit lane offset, and what
// lies past the row's end reads as 0 and is not written, without a branch.  Branches for the columns
// of a partial chunk and 64-bit lane addresses of each matrix took more registers than the values.

typedef __amdgpu_buffer_rsrc_t Rsrc;

// `count` elements of a matrix or a vector of T from element `at` on.
template <typename T>
__device__ __forceinline__ Rsrc span_of(const void* p, int64_t at, uint32_t count) {
    return buffer_rsrc((const T*)p + at, count * (uint32_t)sizeof(T));
}

// W consecutive elements, the first of them element i of a span, as they lie in memory.
template <typename T, int W>
struct Piece;
template <>
struct Piece<uint16_t, 8> {
    u32x4 w;
    template <bool ONCE = false>
    __device__ __forceinline__ void load(Rsrc r, uint32_t i) {
        w = __builtin_amdgcn_raw_buffer_load_b128(r, i * 2, 0, ONCE ? kLoadNt : 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack_bf16x8(w, v); }
    // Makes the compiler unpack the values again, instead of keeping them from one phase of a row to the
    // next in registers of their own.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(w)); }
    static __device__ __forceinline__ void store(Rsrc r, uint32_t i, const float (&v)[8]) {
        __builtin_amdgcn_raw_buffer_store_b128(pack_bf16x8(v), r, i * 2, 0, 0);
    }
};
template <>
struct Piece<float, 8> {
    u32x4 a, b;
    template <bool ONCE = false>
    __device__ __forceinline__ void load(Rsrc r, uint32_t i) {
        a = __builtin_amdgcn_raw_buffer_load_b128(r, i * 4, 0, ONCE ? kLoadNt : 0);
        b = __builtin_amdgcn_raw_buffer_load_b128(r, i * 4 + 16, 0, ONCE ? kLoadNt : 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(a[j]);
            v[4 + j] = __uint_as_float(b[j]);
        }
    }
    __device__ __forceinline__ void forget() {}
    static __device__ __forceinline__ void store(Rsrc r, uint32_t i, const float (&v)[8]) {
        u32x4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __float_as_uint(v[j]);
            b[j] = __float_as_uint(v[4 + j]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(a, r, i * 4, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(b, r, i * 4 + 16, 0, 0);
    }
};
template <>
struct Piece<uint16_t, 1> {
    uint32_t w;
    template <bool = false>
    __device__ __forceinline__ void load(Rsrc r, uint32_t i) { w = __builtin_amdgcn_raw_buffer_load_b16(r, i * 2, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __uint_as_float(w << 16); }
    __device__ __forceinline__ void forget() {}
    static __device__ __forceinline__ void store(Rsrc r, uint32_t i, const float (&v)[1]) {
        __builtin_amdgcn_raw_buffer_store_b16(bf16_rne(v[0]), r, i * 2, 0, 0);
    }
};
template <>
struct Piece<float, 1> {
    uint32_t w;
    template <bool = false>
    __device__ __forceinline__ void load(Rsrc r, uint32_t i) { w = __builtin_amdgcn_raw_buffer_load_b32(r, i * 4, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __uint_as_float(w); }
    __device__ __forceinline__ void forget() {}
    static __device__ __forceinline__ void store(Rsrc r, uint32_t i, const float (&v)[1]) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, i * 4, 0, 0);
    }
};

// Elements i .. of a parameter vector from column c0 on, `count` of them; null: ones.
template <int W>
__device__ __forceinline__ void get_param(const void* p, bool f32, uint32_t c0, uint32_t count, uint32_t i, float (&v)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = 1.0f;
    if (!p) return;
    if (f32) {
        Piece<float, W> x;
        x.load(span_of<float>(p, c0, count), i);
        x.get(v);
    } else {
        Piece<uint16_t, W> x;
        x.load(span_of<uint16_t>(p, c0, count), i);
        x.get(v);
    }
}

// Where a lane's piece lies: element i of a span of `live` elements from `at` on in each matrix (past its
// end if the piece is not there), element ip of `count` from column c0 on in the parameters.
struct RowPart {
    int64_t at;
    uint32_t live, i;
    uint32_t c0, count, ip;
    bool in;
};
constexpr uint32_t kNowhere = 1u << 28;  // past the end of any span

// What the pass reads of a row's W columns, as it lies in memory.
template <typename T, int W, bool POST, int GATE, bool STREAM>
struct RnRaw {
    using P = Piece<T, W>;
    P h, dout, y, dh, gate;

    // A matrix that is not there is loaded as a span of no elements: values kept from the last row in
    // its place would need registers of their own.
    __device__ __forceinline__ void load_first(const RnBwdParams& p, const RowPart& q) {
        const uint32_t live = p.dout ? q.live : 0u;
        h.template load<STREAM>(span_of<T>(p.h, q.at, live), q.i);
        dout.template load<STREAM>(span_of<T>(p.dout, q.at, live), q.i);
    }
    __device__ __forceinline__ void load_y(const RnBwdParams& p, const RowPart& q) {
        if constexpr (POST || GATE != kGateNone) y.template load<STREAM>(span_of<T>(p.y, q.at, q.live), q.i);
    }
    __device__ __forceinline__ void load_rest(const RnBwdParams& p, const RowPart& q) {
        load_y(p, q);
        dh.template load<STREAM>(span_of<T>(p.dh, q.at, p.dh ? q.live : 0u), q.i);
        if constexpr (GATE == kGateElement) gate.template load<STREAM>(span_of<T>(p.gate, q.at, q.live), q.i);
    }
};

// W columns of a row through the three phases of the pass.  KEEP: the parameters stay in registers.
template <typename T, int W, bool POST, int GATE, bool STREAM, bool KEEP>
struct RnBwdPiece {
    using P = Piece<T, W>;
    using Raw = RnRaw<T, W, POST, GATE, STREAM>;
    float dw[W];  // dweight's sum over the rows
    float t[W];   // the gradient of the normed y
    float kept[3][KEEP ? W : 1];

    __device__ __forceinline__ void keep(const RnBwdParams& p, const RowPart& q) {
        get_param(p.dout ? p.weight : nullptr, p.param_f32, q.c0, q.count, q.ip, kept[0]);
        if constexpr (POST) get_param(p.post_weight, p.param_f32, q.c0, q.count, q.ip, kept[1]);
        if constexpr (GATE == kGateColumn) get_param(p.gate, p.param_f32, q.c0, q.count, q.ip, kept[2]);
    }
    template <int WHICH>
    __device__ __forceinline__ void param(const void* v, const RnBwdParams& p, const RowPart& q, float (&w)[W]) {
        if constexpr (KEEP) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j] = kept[WHICH][j];
        } else {
            get_param(v, p.param_f32, q.c0, q.count, q.ip, w);
        }
    }
    // The sum of dout weight xh.  Outside the row the values are 0, and so has to be r, which may be
    // infinite.
    __device__ __forceinline__ void first(Raw& x, const RnBwdParams& p, const RowPart& q, float r, float& s) {
        float w[W], v[W], g[W];
        param<0>(p.weight, p, q, w);
        x.h.get(v);
        x.dout.get(g);
        const float rc = q.in ? r : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float gx = g[j] * (v[j] * rc);
            dw[j] += gx;
            s = __builtin_fmaf(gx, w[j], s);
        }
        x.h.forget();
        x.dout.forget();
    }
    // dresidual and what follows from it; the sums over the rows of the gate's and the post-norm's
    // gradients are added by `add`.  Outside the row all values are 0, and the row's factors are made so.
    template <typename Add>
    __device__ __forceinline__ void second(Raw& x, const RnBwdParams& p, const RowPart& q, float r, float s, float rp,
                                           float& s2, Add add) {
        float w[W], v[W], g[W];
        const float rc = q.in ? r : 0.0f, rs = q.in ? r * s : 0.0f;
        param<0>(p.dout ? p.weight : nullptr, p, q, w);
        x.h.get(v);
        x.dout.get(g);
#pragma unroll
        for (int j = 0; j < W; ++j) g[j] = __builtin_fmaf(-v[j], rs, g[j] * w[j]);
        x.dh.get(v);
#pragma unroll
        for (int j = 0; j < W; ++j) g[j] = __builtin_fmaf(g[j], rc, v[j]);  // dh without dout, whose r is 0
        if (p.dresidual) P::store(span_of<T>(p.dresidual, q.at, q.live), q.i, g);
#pragma unroll
        for (int j = 0; j < W; ++j) t[j] = g[j] * p.scale;
        if constexpr (POST || GATE != kGateNone) {
            float k[W];
            if constexpr (GATE == kGateElement) x.gate.get(k);
            if constexpr (GATE == kGateColumn) param<2>(p.gate, p, q, k);
            if constexpr (POST) param<1>(p.post_weight, p, q, w);
            x.y.get(v);
            const float yc = q.in ? rp : 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) g[j] = t[j] * (v[j] * yc);  // times yh
            if constexpr (GATE != kGateNone) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    v[j] = POST ? g[j] * w[j] : g[j];
                    t[j] *= k[j];
                    g[j] *= k[j];
                }
                if constexpr (GATE == kGateColumn) add(1, v);
                else if (p.dgate_rows) P::store(span_of<T>(p.dgate_rows, q.at, q.live), q.i, v);
            }
            if constexpr (POST) {
                add(0, g);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    s2 = __builtin_fmaf(g[j], w[j], s2);
                    t[j] *= w[j];
                }
                x.y.forget();
            }
        }
    }
    __device__ __forceinline__ void third(const Raw& x, const RnBwdParams& p, const RowPart& q, float rp, float s2) {
        if constexpr (POST) {
            float y[W];
            x.y.get(y);
            const float ys = rp * s2;
#pragma unroll
            for (int j = 0; j < W; ++j) t[j] = __builtin_fmaf(-y[j], ys, t[j]) * rp;
        }
        P::store(span_of<T>(p.dy, q.at, q.live), q.i, t);
    }
};

// LPT lanes per row (a team), NP pieces of W columns per lane.  Teams smaller than a wave have consecutive
// rows, which are one span.
//
// In bf16 the next row is on its way while one is worked on.  Loads return in order, so none may follow
// it: the parameters are kept in registers.  In fp32 those registers would cost a workgroup its place.
template <typename T, int LPT, int W, int NP, int WAVES, bool POST, int GATE, bool STREAM>
__global__ __launch_bounds__(WAVES * 64, LPT < 64 ? 3 : 4) void rn_bwd_kernel(const RnBwdParams p) {
    constexpr int TEAMS = WAVES * 64 / LPT;
    constexpr int LANES = LPT;
    constexpr int SUB = LPT < 64 ? 64 / LPT : 1;   // teams of a wave
    constexpr int WPR = LPT < 64 ? 1 : LPT / 64;   // waves of a team
    constexpr int COLS = NP * LANES * W;
    constexpr int Q = W / 4;  // fours of columns per piece
    // Two pieces of fp32 per lane do not fit: h, dout and y are read again for the phase that needs them, from
    // the caches.
    constexpr bool ONCE = NP == 1 || sizeof(T) == 2;
    constexpr bool AHEAD = NP == 1 && sizeof(T) == 2;
    constexpr int LSUMS = POST || GATE == kGateColumn ? 2 : 1;  // the join needs one
    __shared__ float red[2][2][WAVES];
    __shared__ float ltail[3][TEAMS][8];
    // [which][team][COLS], a lane's four columns together: column W (i LANES + lane) + 4 q + j at
    // ((Q i + q) LANES + lane) 4 + j, free of bank conflicts
    __shared__ f32x4 lsum[LSUMS * TEAMS * COLS / 4];
    const int wave = uniform(threadIdx.x >> 6);
    const int first_team = wave * SUB / WPR;  // of the wave
    const uint32_t sub = SUB > 1 ? (threadIdx.x & 63) / LPT : 0;
    const int team = first_team + (int)sub;
    const int lane = threadIdx.x - team * LANES;
    const uint32_t cols = p.cols, whole = cols & ~(W - 1u);
    const float inv_cols = 1.0f / (float)p.cols;
    f32x4* mine = lsum + team * (COLS / 4) + lane;
    RnBwdPiece<T, W, POST, GATE, STREAM, AHEAD> pc[NP];
    RnBwdPiece<T, 1, POST, GATE, STREAM, AHEAD> tail;
    const bool tailed = (uint32_t)lane < cols - whole;
    float tsum[2] = {0.0f, 0.0f};
    tail.dw[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) pc[i].dw[j] = 0.0f;
    if (LSUMS == 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < Q * NP; ++i) mine[k * (TEAMS * COLS / 4) + i * LANES] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Sum over the row's waves; the two slots of a turn and the turns' flip keep one barrier enough.
    auto team_sum = [&](float v, int flip, int slot) {
        v = lanes_sum<LPT < 64 ? LPT : 64>(v);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0) red[flip][slot][wave] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) v += red[flip][slot][team * WPR + i];
        }
        return v * inv_cols;
    };
    // Of the wave's first row `row`.
    auto rows_here = [&](int64_t row) {
        const int64_t left = p.rows - row;
        return left <= 0 ? 0u : left < SUB ? (uint32_t)left : (uint32_t)SUB;
    };
    auto part = [&](int64_t row, int i) {
        const uint32_t n = rows_here(row), c = (uint32_t)(i * LANES + lane) * W;
        const bool in = sub < n && c < whole;
        if constexpr (SUB > 1) return RowPart{row * cols, n * cols, in ? sub * cols + c : kNowhere, 0, whole, c, in};
        else return RowPart{row * cols, n * whole, c, 0, whole, c, in};
    };
    auto rest = [&](int64_t row) {
        const uint32_t n = rows_here(row), tail_cols = cols - whole;
        const bool in = sub < n && tailed;
        if constexpr (SUB > 1)
            return RowPart{row * cols, n * cols, in ? sub * cols + whole + lane : kNowhere, whole, tail_cols, (uint32_t)lane, in};
        else return RowPart{row * cols + whole, n * tail_cols, (uint32_t)lane, whole, tail_cols, (uint32_t)lane, in};
    };
    // What a row brings with it.
    struct Row {
        RnRaw<T, W, POST, GATE, STREAM> x[NP];
        RnRaw<T, 1, POST, GATE, STREAM> tail;
        float r, rp;
    };
    auto load_row = [&](Row& o, int64_t row) {
        const bool here = sub < rows_here(row);
        o.r = here && p.dout ? p.rstd[row + sub] : 0.0f;
        o.rp = !POST ? 1.0f : here ? p.post_rstd[row + sub] : 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            o.x[i].load_first(p, part(row, i));
            if (ONCE) o.x[i].load_rest(p, part(row, i));
        }
        if (whole != cols) {
            o.tail.load_first(p, rest(row));
            if (ONCE) o.tail.load_rest(p, rest(row));
        }
    };
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t row = (int64_t)blockIdx.x * TEAMS + first_team;
    Row cur;
    if constexpr (AHEAD) {
        pc[0].keep(p, part(0, 0));
        if (whole != cols) tail.keep(p, rest(0));
        load_row(cur, row);
    }
    // every team takes part in every turn's barriers, with or without a row
    for (int flip = 0; row - first_team < p.rows; row += step, flip ^= 1) {
        Row next;
        if constexpr (AHEAD) load_row(next, row + step);
        else load_row(cur, row);
        const float r = cur.r, rp = cur.rp;
        float s = 0.0f, s2 = 0.0f;
        if (p.dout) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (!ONCE) __builtin_amdgcn_sched_barrier(0);
                pc[i].first(cur.x[i], p, part(row, i), r, s);
            }
            if (whole != cols) tail.first(cur.tail, p, rest(row), r, s);
            s = team_sum(s, flip, 0);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            RowPart q = part(row, i);
            if (!ONCE) {
                __builtin_amdgcn_sched_barrier(0);  // one chunk after the other
                asm volatile("" : "+v"(q.i));       // loads of their own, not the first phase's kept
                cur.x[i].load_first(p, q);
                cur.x[i].load_rest(p, q);
            }
            pc[i].second(cur.x[i], p, q, r, s, rp, s2, [&](int which, const float(&v)[W]) {
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    mine[which * (TEAMS * COLS / 4) + (Q * i + k) * LANES] +=
                        f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
            });
        }
        if (whole != cols) {
            RowPart q = rest(row);
            if (!ONCE) {
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("" : "+v"(q.i));
                cur.tail.load_first(p, q);
                cur.tail.load_rest(p, q);
            }
            tail.second(cur.tail, p, q, r, s, rp, s2, [&](int which, const float(&v)[1]) { tsum[which] += v[0]; });
        }
        if constexpr (POST) s2 = team_sum(s2, flip, 1);
        if (p.dy) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                RowPart q = part(row, i);
                if (!ONCE) {
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("" : "+v"(q.i));
                    cur.x[i].load_y(p, q);
                }
                pc[i].third(cur.x[i], p, q, rp, s2);
            }
            if (whole != cols) {
                RowPart q = rest(row);
                if (!ONCE) {
                    asm volatile("" : "+v"(q.i));
                    cur.tail.load_y(p, q);
                }
                tail.third(cur.tail, p, q, rp, s2);
            }
        }
        if constexpr (AHEAD) cur = next;
    }
    if (!p.part) return;
    if (tailed) {
        ltail[0][team][lane] = tail.dw[0];
        ltail[1][team][lane] = tsum[0];
        ltail[2][team][lane] = tsum[1];
    }
    // What LDS holds first, then dweight's sums through the first's place.
    auto join = [&](int which, const f32x4* teams) {
        float* out = p.part + ((int64_t)blockIdx.x * 3 + which) * cols;
        __syncthreads();
        for (uint32_t q = threadIdx.x; q < COLS / 4; q += WAVES * 64) {
            const uint32_t c = (q / (Q * LANES) * LANES + q % LANES) * W + q / LANES % Q * 4;
            if (c >= whole) continue;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < TEAMS; ++k) v += teams[k * (COLS / 4) + q];
#pragma unroll
            for (int j = 0; j < 4; ++j) out[c + j] = v[j];
        }
        if (threadIdx.x < cols - whole) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < TEAMS; ++k) v += ltail[which][k][threadIdx.x];
            out[whole + threadIdx.x] = v;
        }
    };
    if constexpr (LSUMS == 2) {
        if (p.sums[1]) join(1, lsum);
        if (p.sums[2]) join(2, lsum + TEAMS * COLS / 4);
    }
    if (p.sums[0]) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const float(&d)[W] = pc[i].dw;
                mine[(Q * i + k) * LANES] = f32x4{d[4 * k], d[4 * k + 1], d[4 * k + 2], d[4 * k + 3]};
            }
        join(0, lsum);
    }
}

// The column sums from the groups' partial ones: 32 columns per workgroup, 32 threads down the
// groups, joined in LDS in a fixed order.  blockIdx.y: which sum.
__global__ __launch_bounds__(1024) void rn_bwd_join_kernel(const RnBwdParams p, int64_t groups) {
    __shared__ float s[32][33];
    const int which = blockIdx.y;
    void* out = p.sums[which];
    if (!out) return;
    const int cl = threadIdx.x & 31, g0 = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    float v = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t g = g0; g < groups; g += 32) v += p.part[(g * 3 + which) * p.cols + c];
    }
    s[g0][cl] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s[i][cl];
        if (c < p.cols) {
            if (p.grad_f32) ((float*)out)[c] = v;
            else ((uint16_t*)out)[c] = bf16_rne(v);
        }
    }
}

struct RnBwdShape {
    int lpt, waves, groups;  // groups: the workgroups that are at work at once
};
// Two rows a workgroup from 2049 to 4096 columns.  Without streaming, 16384 x 4096 in bf16 with a gate of columns, without one, with
// one of elements, the norm alone, and 1024 rows, us: in one row of eight waves, 512 at once, 163, 161, 218, 81
// and 22.9; in two, 256 at once, 155, 154, 205, 78 and 20.3.
RnBwdShape rn_bwd_shape(int64_t cols) {
    if (cols <= 128) return {16, 4, 768};
    if (cols <= 256) return {32, 4, 768};
    if (cols <= 512) return {64, 8, 512};
    if (cols <= 1024) return {128, 8, 512};
    if (cols <= 2048) return {256, 8, 512};
    if (cols <= 4096) return {512, 16, 256};
    return {1024, 16, 256};
}
template <typename T, bool POST, int GATE, bool STREAM>
const void* pick_rn_bwd_shape(int64_t cols) {
    switch (rn_bwd_shape(cols).lpt) {
        case 16: return (const void*)&rn_bwd_kernel<T, 16, 8, 1, 4, POST, GATE, STREAM>;
        case 32: return (const void*)&rn_bwd_kernel<T, 32, 8, 1, 4, POST, GATE, STREAM>;
        case 64: return (const void*)&rn_bwd_kernel<T, 64, 8, 1, 8, POST, GATE, STREAM>;
        case 128: return (const void*)&rn_bwd_kernel<T, 128, 8, 1, 8, POST, GATE, STREAM>;
        case 256: return (const void*)&rn_bwd_kernel<T, 256, 8, 1, 8, POST, GATE, STREAM>;
        case 512: return (const void*)&rn_bwd_kernel<T, 512, 8, 1, 16, POST, GATE, STREAM>;
    }
    return cols <= 8192 ? (const void*)&rn_bwd_kernel<T, 1024, 8, 1, 16, POST, GATE, STREAM>
                        : (const void*)&rn_bwd_kernel<T, 1024, 8, 2, 16, POST, GATE, STREAM>;
}
template <typename T, bool POST, bool STREAM>
const void* pick_rn_bwd_gate(int64_t s, int gate) {
    return gate == kGateNone     ? pick_rn_bwd_shape<T, POST, kGateNone, STREAM>(s)
           : gate == kGateColumn ? pick_rn_bwd_shape<T, POST, kGateColumn, STREAM>(s)
                                 : pick_rn_bwd_shape<T, POST, kGateElement, STREAM>(s);
}
template <typename T>
const void* pick_rn_bwd(int64_t s, bool post, int gate, bool stream) {
    if constexpr (sizeof(T) == 2) {
        if (stream) return post ? pick_rn_bwd_gate<T, true, true>(s, gate) : pick_rn_bwd_gate<T, false, true>(s, gate);
    }
    return post ? pick_rn_bwd_gate<T, true, false>(s, gate) : pick_rn_bwd_gate<T, false, false>(s, gate);
}

// What the matrices of one pass have to come to for it to stream them past the caches: the last-level cache's
// bytes, past which nothing of the last pass is left in it, nor anything of this one for the next.
constexpr int64_t kStreamBytes = 256 << 20;

}  // namespace

hipError_t launch_rn(const RnParams& p, hipStream_t stream) {
    const RnShape s = rn_shape(p.cols, p.f32, !p.y);
    const int rpw = s.lpt <= 64 ? 256 / s.lpt : 1, threads = s.lpt <= 64 ? 256 : s.lpt;
    const void* k = p.cols % 8 == 0 ? (p.f32 ? pick_rn<float, true>(s) : pick_rn<uint16_t, true>(s))
                                    : (p.f32 ? pick_rn<float, false>(s) : pick_rn<uint16_t, false>(s));
    // What is written.  us without / with, both norms and a gate of columns in bf16: 16384 x 4096 98 / 97, with the
    // checkpoint 109 / 108, 8192 x 8192 101 / 96; the same buffers 110 / 88, 115 / 97 and 101 / 80.  Smaller
    // outputs the caches hold for what reads them next.
    const bool once = p.rows * p.cols * ((p.h ? 1 : 0) + (p.out ? 1 : 0)) * (p.f32 ? 4 : 2) >= kStreamBytes;
    for (int64_t row0 = 0; row0 < p.rows; row0 += kMaxGrid * rpw) {
        const int64_t rows = p.rows - row0 < kMaxGrid * rpw ? p.rows - row0 : kMaxGrid * rpw;
        void* args[] = {(void*)&p, (void*)&row0, (void*)&once};
        const hipError_t err =
            hipLaunchKernel(k, dim3((unsigned)((rows + rpw - 1) / rpw)), dim3(threads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

int64_t rn_bwd_groups(int64_t rows, int64_t cols) {
    const RnBwdShape s = rn_bwd_shape(cols);
    const int64_t teams = s.waves * 64 / s.lpt, wanted = (rows + teams - 1) / teams;
    return wanted < 1 ? 1 : wanted < s.groups ? wanted : s.groups;
}

hipError_t launch_rn_bwd(const RnBwdParams& p, hipStream_t stream) {
    const RnBwdShape s = rn_bwd_shape(p.cols);
    const int64_t groups = rn_bwd_groups(p.rows, p.cols);
    const bool post = p.post_rstd || p.sums[1];  // without rows the sum is there without rstd
    // What is read, in bf16.  Rows of 4096, us without / with, with a gate of columns, without one: 8192 rows 86 / 82
    // and 84 / 80, 16384 155 / 152 and 155 / 147.  The same buffers: 4096 rows 40 / 49 and 37 / 43, 6144 62 / 64
    // and 57 / 57, 8192 86 / 80 and 85 / 71, 16384 155 / 140 and 155 / 128.  In fp32, which reads each row when it is
    // its turn, 8192 rows 165 / 174.
    const int matrices = (p.dout ? 2 : 0) + (p.dh ? 1 : 0) + (post || p.gate_kind != kGateNone ? 1 : 0) +
                         (p.gate_kind == kGateElement ? 1 : 0);
    const bool once = !p.f32 && p.rows * p.cols * matrices * 2 >= kStreamBytes;
    const void* k = p.f32 ? pick_rn_bwd<float>(p.cols, post, p.gate_kind, once)
                          : pick_rn_bwd<uint16_t>(p.cols, post, p.gate_kind, once);
    void* args[] = {(void*)&p};
    hipError_t err = hipLaunchKernel(k, dim3((unsigned)groups), dim3(s.waves * 64), args, 0, stream);
    if (err != hipSuccess || !p.part) return err;
    void* jargs[] = {(void*)&p, (void*)&groups};
    return hipLaunchKernel((const void*)&rn_bwd_join_kernel, dim3((unsigned)((p.cols + 31) / 32), 3), dim3(1024), jargs,
                           0, stream);
}

}  // namespace loco
