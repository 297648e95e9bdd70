// Host-side interface between the C ABI of the layer operators (abi.hip) and their
// kernel launchers.
#pragma once

#include "loco_internal.hpp"

namespace loco {

// An 8-bit checkpoint [rows, cols] on the device; codes null: none.
struct CkptDev {
    int8_t* codes;
    uint8_t* exps;
    int block64;  // blocks of 64 elements (else 32)
    int64_t nblocks;  // per row
};

// ---- layer norm --------------------------------------------------------------------

constexpr int64_t kLnMaxCols = 16384;  // a row stays in one workgroup's registers

struct LnParams {
    const void* x;
    const void* w;  // may be null: ones
    const void* b;  // may be null: zeros
    void* y;
    float* mean;
    float* rstd;
    CkptDev ckpt;
    int64_t rows;
    int cols;
    float eps;
    int f32, param_f32;
};
hipError_t launch_ln(const LnParams& p, hipStream_t stream);

struct LnBwdParams {
    const void* dy;
    const void* x;
    const void* w;  // may be null: ones
    const float* mean;
    const float* rstd;
    const void* residual;  // may be null
    void* dx;
    void* dw;     // may be null
    void* db;     // may be null
    float* part;  // [groups][2][cols] partial sums of dw and db
    int64_t rows;
    int cols;
    int f32, param_f32, grad_f32;
};
// Workgroups of the row pass, each of which leaves one partial sum of dw and db.
int64_t ln_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_ln_bwd(const LnBwdParams& p, hipStream_t stream);

// ---- activation checkpoints ----------------------------------------------------------

hipError_t launch_ckpt_write(const void* x, bool f32, int64_t rows, int64_t cols, const CkptDev& c, hipStream_t stream);
// out: rows of `ld` elements, of which cols are written.  rest (GELU or SiLU, bf16): not the
// activation, but what its rounding to bf16 leaves.
hipError_t launch_ckpt_read(const CkptDev& c, int64_t rows, int64_t cols, int act, void* out, int64_t ld, bool f32,
                            bool rest, hipStream_t stream);

// ---- matrix products -----------------------------------------------------------------

// Features are bounded so that a tile's byte offsets fit 32 bits.
constexpr int64_t kMmMaxFeatures = (int64_t)1 << 20;

// What happens to a product's sums v on their way out, in this order.
struct MmEpilogue {
    const uint16_t* bias;      // v += bias[col] (null: none)
    CkptDev ckpt;              // 8-bit checkpoint of v (codes null: none)
    CkptDev slope;             // v *= act'(checkpointed value) (codes null: none)
    int act;                   // else v = act(v)
    const uint16_t* residual;  // v += residual[row, col] (null: none)
    int accumulate;            // v += out[row, col]
    void* out;
    int out_f32;
};

// C[m, n] = sum over k of A B, with A [m, k] (a_kmajor) or [k, m], B [n, k] (b_kmajor) or
// [k, n], row-major bf16.
struct MmParams {
    const uint16_t* a;
    const uint16_t* b;
    int64_t m, n, k;
    int64_t b_ld;  // elements per row of B; 0: as many as it has columns
    int a_kmajor, b_kmajor;
    MmEpilogue ep;
    void* workspace;  // mm_workspace bytes
};
// with_ckpt: whether the call writes a checkpoint, which few rows' kernel does not.
int64_t mm_workspace(const MmParams& p, bool with_ckpt);
hipError_t launch_mm(const MmParams& p, hipStream_t stream);
// The row length at which an operand need not be copied.
int64_t mm_padded(int64_t n);

// out[n] = sum over the rows of x [rows, n]; part [col_sum_groups][n].
int64_t col_sum_groups(int64_t rows, int64_t n);
hipError_t launch_col_sum(const uint16_t* x, int64_t rows, int64_t n, float* part, void* out, bool f32, bool accumulate,
                          hipStream_t stream);

}  // namespace loco
