// Host-side interface between the C ABI of the operators around a layer's products
// (abi_step.hpp) and their kernel launchers: AdamW over many tensors, the norms around a block,
// log probabilities of tokens.
#pragma once

#include "loco_layer_internal.hpp"

namespace loco {

// ---- AdamW over many tensors ---------------------------------------------------------

constexpr int kAwTile = 512;        // elements per wave of a step
constexpr int kAwStateTile = 2048;  // elements per wave that reads or writes states, which moves 3 to 5 bytes of each

// One tensor (or one 8-bit state with its values) as its table in device memory describes it.  A table of
// n is n of AwSegDev after the n first tiles, each in the call's tile space.
struct AwSegDev {
    void* param;  // or the values of a state
    const void* grad;
    void* m;  // fp32, or 8-bit codes with mexp
    void* v;
    uint8_t* mexp;
    uint8_t* vexp;
    uint16_t* copy;  // may be null
    int64_t n;
    double weight_decay;
    int64_t second;  // of a state: the second moment's
};
inline int64_t aw_table_bytes(int64_t n) { return ((n * 8 + 15) / 16 * 16) + n * (int64_t)sizeof(AwSegDev); }

// Kernel arguments that carry descriptions into a table: a launch takes 4 KB of them.
constexpr int kAwFill = 40;
struct AwFillParams {
    AwSegDev seg[kAwFill];
    int64_t tile0[kAwFill];
    void* table;
    int64_t n, first;
    int count;
};
hipError_t launch_aw_fill(const AwFillParams& p, hipStream_t stream);

struct AwParams {
    const void* table;
    int64_t n, ntiles;
    const float* grad_scale;  // may be null: 1
    double lr;
    float beta1, omb1, beta2, omb2;
    float step_size;  // lr / (1 - beta1^step)
    float root;       // 1 / sqrt(1 - beta2^step)
    float eps;
    uint64_t key;            // of random rounding: aw_mix(key + *counter) is the call's
    const int64_t* counter;  // may be null: 0
};
// 64 bits of which each depends on all of x's.
__host__ __device__ inline uint64_t aw_mix(uint64_t x) {
    x = (x ^ (x >> 32)) * 0x9E3779B97F4A7C15u;
    x = (x ^ (x >> 29)) * 0xB504F333F9DE6485u;
    return x ^ (x >> 32);
}
// block: 0 for states in fp32, else the elements of one block of 8-bit states, rounded at random or to nearest.
hipError_t launch_aw(const AwParams& p, bool param_f32, bool grad_f32, int block, bool random, hipStream_t stream);
hipError_t launch_aw_state(const void* table, int64_t n, int64_t ntiles, int block, bool f32, bool write,
                           hipStream_t stream);

// ---- the norms around a block ----------------------------------------------------------

enum : int { kGateNone = 0, kGateColumn = 1, kGateElement = 2 };

struct RnParams {
    const void* y;            // may be null: only the residual
    const void* residual;     // may be null: 0
    const void* gate;         // [cols] of the parameters' type, or [rows, cols]
    const void* weight;       // may be null: ones
    const void* post_weight;  // may be null: ones
    void* h;                  // may be null
    void* out;                // may be null
    float* rstd;              // with out
    float* post_rstd;         // null: y is not normed
    CkptDev ckpt;
    int64_t rows;
    int cols;
    float scale, eps;
    int gate_kind;
    int f32, param_f32;
};
hipError_t launch_rn(const RnParams& p, hipStream_t stream);

struct RnBwdParams {
    const void* dout;  // may be null: 0
    const void* dh;    // may be null: 0
    const void* h;     // with dout
    const void* y;     // where post_rstd, dgate or dpost_weight need it
    const void* gate;
    const void* weight;
    const void* post_weight;
    const float* rstd;
    const float* post_rstd;
    void* dresidual;  // may be null
    void* dy;         // may be null
    void* dgate_rows; // gradient of a gate of elements; may be null
    void* sums[3];    // dweight, dpost_weight, a column gate's gradient; each may be null
    float* part;      // [groups][3][cols] partial sums; null: no sums
    int64_t rows;
    int cols;
    float scale;
    int gate_kind;
    int f32, param_f32, grad_f32;
};
int64_t rn_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_rn_bwd(const RnBwdParams& p, hipStream_t stream);

// ---- log probabilities of tokens ---------------------------------------------------------

typedef float f32x4_t __attribute__((ext_vector_type(4)));
constexpr int kLpMaxTop = 32;
constexpr int64_t kLpMaxVocab = (int64_t)1 << 24;

// Sequences of rows: what a row's place in a buffer has beyond row times the step from row to row.
struct LpSeqs {
    uint32_t rows;  // of a sequence; 0: there is one
    int64_t logits, dlogits, targets;  // elements between a sequence's end and the next one
};

struct LpParams {
    const void* logits;
    int64_t rows, ld;
    int vocab;
    const int64_t* targets;  // may be null
    float scale;
    float* logprob;  // may be null
    float* entropy;  // may be null
    float* stats;    // [rows][2]; may be null
    int32_t* top_ids;
    float* top_logprobs;
    int top;
    int f32;
    f32x4_t* sums;   // [rows][splits] of a row's pieces: maximum and sums
    uint64_t* keys;  // [rows][splits][top]: their best values
    LpSeqs seqs;
    int splits, piece;  // set by launch_lp: pieces per row, chunks of eight per piece
};
// Pieces of a row that a call works on apart and joins in a second launch; 1: none.
constexpr int kLpMaxSplits = 32;
int lp_splits(int64_t rows, int64_t vocab);
hipError_t launch_lp(const LpParams& p, hipStream_t stream);

struct LpBwdParams {
    const void* logits;
    void* dlogits;
    int64_t rows, ld, dld;
    int vocab;
    const int64_t* targets;
    const float* stats;
    const float* entropy;
    const float* dlogprob;  // may be null: 0
    const float* dentropy;  // may be null: 0
    float scale;
    int f32;
    LpSeqs seqs;
};
hipError_t launch_lp_bwd(const LpBwdParams& p, hipStream_t stream);

}  // namespace loco
