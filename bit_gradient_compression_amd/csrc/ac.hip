// Activation checkpoints in 8 bits: written from bf16 or fp32, read back through an
// activation.  The format is described in loco_layer.hpp.
//
// Both kernels are bound by HBM (3 bytes per bf16 element).  A lane takes a chunk of eight
// elements; a block is an aligned group of four or eight lanes.

#include "loco_layer.hpp"
#include "loco_layer_internal.hpp"

namespace loco {

namespace {

constexpr int kAcThreads = 256;

// Chunk t of the tensor: rows are padded to whole blocks, so that a block never spans two
// rows and its lanes stay together.
struct ChunkAt {
    int64_t row;
    int64_t col;
    int valid;
};
__device__ __forceinline__ ChunkAt chunk_at(int64_t t, int64_t rows, int64_t cols, int64_t per_row) {
    ChunkAt a;
    a.row = t / per_row;
    a.col = (t - a.row * per_row) * 8;
    const int64_t left = cols - a.col;
    a.valid = a.row >= rows || left <= 0 ? 0 : left < 8 ? (int)left : 8;
    return a;
}

template <typename T>
__global__ __launch_bounds__(kAcThreads) void ckpt_write_kernel(const T* x, CkptDev ck, int64_t rows, int64_t cols,
                                                                int64_t per_row, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * kAcThreads + threadIdx.x;
    const ChunkAt a = chunk_at(t, rows, cols, per_row);
    float v[8];
    load_chunk(x + a.row * cols + a.col, a.valid, v);
    const uint32_t e = ckpt_exp(block_top(v, ck.block64));
    store_codes(ck.codes + a.row * cols + a.col, a.valid, ckpt_codes(v, e));
    const int per = ck.block64 ? 8 : 4;
    if ((threadIdx.x & (per - 1)) == 0 && a.valid > 0)
        ck.exps[a.row * ck.nblocks + a.col / (8 * per)] = (uint8_t)e;
}

template <typename T, int ACT>
__global__ __launch_bounds__(kAcThreads) void ckpt_read_kernel(CkptDev ck, T* out, int64_t rows, int64_t cols,
                                                               int64_t per_row, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * kAcThreads + threadIdx.x;
    const ChunkAt a = chunk_at(t, rows, cols, per_row);
    if (a.valid <= 0) return;
    const uint32_t e = ck.exps[a.row * ck.nblocks + a.col / (ck.block64 ? 64 : 32)];
    float v[8];
    decode_codes(load_codes(ck.codes + a.row * cols + a.col, a.valid), e, v);
    act_chunk<ACT>(v);
    store_chunk(out + a.row * cols + a.col, a.valid, v);
}

template <typename T>
const void* pick_read(int act) {
    switch (act) {
        case 1: return (const void*)&ckpt_read_kernel<T, 1>;
        case 2: return (const void*)&ckpt_read_kernel<T, 2>;
        case 3: return (const void*)&ckpt_read_kernel<T, 3>;
    }
    return (const void*)&ckpt_read_kernel<T, 0>;
}

// Launches over all chunks, at most kMaxGrid workgroups at a time; args[5] points at t0.
hipError_t launch_chunks(const void* k, void** args, int64_t* t0, int64_t chunks, hipStream_t stream) {
    for (*t0 = 0; *t0 < chunks; *t0 += kMaxGrid * kAcThreads) {
        const int64_t left = chunks - *t0;
        const int64_t blocks = left < kMaxGrid * kAcThreads ? (left + kAcThreads - 1) / kAcThreads : kMaxGrid;
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
    const void* k = f32 ? (const void*)&ckpt_write_kernel<float> : (const void*)&ckpt_write_kernel<uint16_t>;
    return launch_chunks(k, args, &t0, rows * per_row, stream);
}

hipError_t launch_ckpt_read(const CkptDev& ck, int64_t rows, int64_t cols, int act, void* out, bool f32,
                            hipStream_t stream) {
    CkptDev c = ck;
    flatten(rows, cols, c);
    int64_t per_row = chunks_per_row(cols, c), t0 = 0;
    void* args[] = {(void*)&c, (void*)&out, (void*)&rows, (void*)&cols, (void*)&per_row, (void*)&t0};
    return launch_chunks(f32 ? pick_read<float>(act) : pick_read<uint16_t>(act), args, &t0, rows * per_row, stream);
}

}  // namespace loco
