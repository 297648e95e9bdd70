// Activation checkpoints in 8 bits: written from bf16 or fp32, read back through an
// activation.  The format is described in loco_layer.hpp.
//
// Both kernels are bound by HBM (3 bytes per bf16 element): 8192 x 11008 is written in 38 - 50 us
// and read through GELU in 44 - 48 (5.4 TB/s and more; a streaming copy reaches 6.4).  A lane takes
// a chunk of eight elements, 16 bytes of bf16; a block is an aligned group of four or eight
// lanes, so its largest value meets in two or three lane exchanges.

#include "loco_layer.hpp"
#include "loco_layer_internal.hpp"

namespace loco {

namespace {

constexpr int kAcThreads = 256;
constexpr int kAcChunks = 2;  // per thread, all loaded before the first is worked
constexpr int64_t kAcTile = kAcThreads * kAcChunks;

// Chunk t of the tensor: rows are padded to whole blocks, so that a block never spans two
// rows and its lanes stay together.  Rows that are whole blocks lie end to end and need no
// division (FLAT: one row).
struct ChunkAt {
    int64_t row, col;
    int valid;
};
template <bool FLAT>
__device__ __forceinline__ ChunkAt chunk_at(int64_t t, int64_t rows, int64_t cols, int64_t per_row) {
    ChunkAt a;
    if constexpr (FLAT) a.row = 0;
    else if (rows * per_row < (int64_t)1 << 31) a.row = (uint32_t)t / (uint32_t)per_row;
    else a.row = t / per_row;
    a.col = (t - a.row * per_row) * 8;
    const int64_t left = cols - a.col;
    a.valid = a.row >= rows || left <= 0 ? 0 : left < 8 ? (int)left : 8;
    return a;
}

template <typename T, bool FLAT>
__global__ __launch_bounds__(kAcThreads) void ckpt_write_kernel(const T* x, CkptDev ck, int64_t rows, int64_t cols,
                                                                int64_t per_row, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * kAcTile + threadIdx.x;
    ChunkAt a[kAcChunks];
    RawChunk<T> raw[kAcChunks];
#pragma unroll
    for (int u = 0; u < kAcChunks; ++u) {
        a[u] = chunk_at<FLAT>(t + u * kAcThreads, rows, cols, per_row);
        raw[u].load(x + a[u].row * cols + a[u].col, a[u].valid);
    }
    const int per = ck.block64 ? 8 : 4, shift = ck.block64 ? 6 : 5;
#pragma unroll
    for (int u = 0; u < kAcChunks; ++u) {
        float v[8];
        raw[u].get(v);
        const uint32_t e = ckpt_exp(block_top(v, ck.block64));
        store_codes(ck.codes + a[u].row * cols + a[u].col, a[u].valid, ckpt_codes(v, e));
        if ((threadIdx.x & (per - 1)) == 0 && a[u].valid > 0)
            ck.exps[a[u].row * ck.nblocks + (a[u].col >> shift)] = (uint8_t)e;
    }
}

// What the rounding of v to bf16 leaves, 0 where that is an infinity; a NaN stays one.
__device__ __forceinline__ void rest_chunk(float (&v)[8]) {
    float h[8];
    unpack_bf16x8(pack_bf16x8(v), h);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fabsf(h[i]) == __builtin_inff() ? 0.0f : v[i] - h[i];
}

template <typename T, int ACT, bool FLAT, bool REST = false>
__global__ __launch_bounds__(kAcThreads) void ckpt_read_kernel(CkptDev ck, T* out, int64_t rows, int64_t cols,
                                                               int64_t per_row, int64_t t0, int64_t ld, int stream) {
    const int64_t t = t0 + (int64_t)blockIdx.x * kAcTile + threadIdx.x;
    const int shift = ck.block64 ? 6 : 5;
    ChunkAt a[kAcChunks];
    u32x2 codes[kAcChunks];
    uint32_t e[kAcChunks];
#pragma unroll
    for (int u = 0; u < kAcChunks; ++u) {
        a[u] = chunk_at<FLAT>(t + u * kAcThreads, rows, cols, per_row);
        codes[u] = load_codes(ck.codes + a[u].row * cols + a[u].col, a[u].valid);
        e[u] = a[u].valid > 0 ? ck.exps[a[u].row * ck.nblocks + (a[u].col >> shift)] : 0u;
    }
#pragma unroll
    for (int u = 0; u < kAcChunks; ++u) {
        float v[8];
        decode_codes(codes[u], e[u], v);
        act_chunk<ACT>(v);
        if constexpr (REST) rest_chunk(v);
        T* to = out + a[u].row * ld + a[u].col;
        if constexpr (sizeof(T) == 2) {
            if (stream && a[u].valid >= 8) {
                stream16(to, pack_bf16x8(v));
                continue;
            }
        }
        store_chunk(to, a[u].valid, v);
    }
}

template <typename T, bool FLAT>
const void* pick_act(int act) {
    switch (act) {
        case 1: return (const void*)&ckpt_read_kernel<T, 1, FLAT>;
        case 2: return (const void*)&ckpt_read_kernel<T, 2, FLAT>;
        case 3: return (const void*)&ckpt_read_kernel<T, 3, FLAT>;
    }
    return (const void*)&ckpt_read_kernel<T, 0, FLAT>;
}
template <typename T>
const void* pick_read(int act, bool flat) {
    return flat ? pick_act<T, true>(act) : pick_act<T, false>(act);
}
template <bool FLAT>
const void* pick_rest(int act) {
    return act == 2 ? (const void*)&ckpt_read_kernel<uint16_t, 2, FLAT, true>
                    : (const void*)&ckpt_read_kernel<uint16_t, 3, FLAT, true>;
}
template <typename T>
const void* pick_write(bool flat) {
    return flat ? (const void*)&ckpt_write_kernel<T, true> : (const void*)&ckpt_write_kernel<T, false>;
}

// Launches over all chunks, at most kMaxGrid workgroups at a time; args[5] points at t0.
hipError_t launch_chunks(const void* k, void** args, int64_t* t0, int64_t chunks, hipStream_t stream) {
    for (*t0 = 0; *t0 < chunks; *t0 += kMaxGrid * kAcTile) {
        const int64_t left = chunks - *t0;
        const int64_t blocks = left < kMaxGrid * kAcTile ? (left + kAcTile - 1) / kAcTile : kMaxGrid;
        const hipError_t err = hipLaunchKernel(k, dim3((unsigned)blocks), dim3(kAcThreads), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// Rows that are whole blocks long lie end to end: one long row, no division per chunk's row.
void flatten(int64_t& rows, int64_t& cols, CkptDev& c) {
    const int64_t block = c.block64 ? 64 : 32;
    if (cols % block == 0) {
        cols *= rows;
        rows = 1;
        c.nblocks = cols / block;
    }
}

int64_t chunks_per_row(int64_t cols, const CkptDev& c) { return ((cols + (c.block64 ? 63 : 31)) / (c.block64 ? 64 : 32)) * (c.block64 ? 8 : 4); }

}  // namespace

hipError_t launch_ckpt_write(const void* x, bool f32, int64_t rows, int64_t cols, const CkptDev& ck,
                             hipStream_t stream) {
    CkptDev c = ck;
    flatten(rows, cols, c);
    int64_t per_row = chunks_per_row(cols, c), t0 = 0;
    void* args[] = {(void*)&x, (void*)&c, (void*)&rows, (void*)&cols, (void*)&per_row, (void*)&t0};
    const void* k = f32 ? pick_write<float>(rows == 1) : pick_write<uint16_t>(rows == 1);
    return launch_chunks(k, args, &t0, rows * per_row, stream);
}

hipError_t launch_ckpt_read(const CkptDev& ck, int64_t rows, int64_t cols, int act, void* out, int64_t ld, bool f32,
                            bool rest, hipStream_t hip_stream) {
    CkptDev c = ck;
    if (ld == cols) {
        flatten(rows, cols, c);
        ld = cols;
    }
    int64_t per_row = chunks_per_row(cols, c), t0 = 0;
    // An output that the 256 MB Infinity Cache could not keep beside the rest goes past it: 134 MB
    // of bf16 take 29 us streamed and 36 cached.  Smaller ones stay for their reader (67 MB:
    // streaming costs a layer norm that follows 4 us).  fp32 chunks are two stores of half a
    // sector each, which streaming would not merge (46 us against 37).
    int stream = !f32 && rows * ld * 2 >= (int64_t)128 << 20;
    void* args[] = {(void*)&c, (void*)&out, (void*)&rows, (void*)&cols, (void*)&per_row, (void*)&t0, (void*)&ld,
                    (void*)&stream};
    const bool flat = rows == 1;
    const void* k = rest  ? (flat ? pick_rest<true>(act) : pick_rest<false>(act))
                    : f32 ? pick_read<float>(act, flat)
                          : pick_read<uint16_t>(act, flat);
    return launch_chunks(k, args, &t0, rows * per_row, hip_stream);
}

}  // namespace loco
