// Host-side interface between the C ABI of the operators around a layer's products
// (abi_step.hpp) and their kernel launchers: AdamW over many tensors, the norms around a block,
// log probabilities of tokens.
#pragma once

#include "loco_layer_internal.hpp"

namespace loco {

// ---- AdamW over many tensors ---------------------------------------------------------

// Tensors per launch: their descriptions are kernel arguments, of which a launch takes 4 KB.
constexpr int kAwMaxSeg = 48;
constexpr int kAwTile = 512;  // elements per wave

struct AwSegDev {
    void* param;
    const void* grad;
    void* m;  // fp32, or 8-bit codes with mexp
    void* v;
    uint8_t* mexp;
    uint8_t* vexp;
    uint16_t* copy;  // may be null
    int64_t n;
};

struct AwParams {
    AwSegDev seg[kAwMaxSeg];
    int64_t tile0[kAwMaxSeg];  // first tile of each tensor in the launch's tile space
    float decay[kAwMaxSeg];    // 1 - lr * weight decay
    int nseg;
    int64_t ntiles;
    const float* grad_scale;  // may be null: 1
    float beta1, omb1, beta2, omb2;
    float step_size;  // lr / (1 - beta1^step)
    float root;       // 1 / sqrt(1 - beta2^step)
    float eps;
};
// block: 0 for states in fp32, else the elements of one block of 8-bit states.
hipError_t launch_aw(const AwParams& p, bool param_f32, bool grad_f32, int block, hipStream_t stream);

struct AwStateDev {
    uint8_t* codes;
    uint8_t* exps;
    void* values;
    int64_t n;
};
constexpr int kAwMaxStates = 64;
struct AwStateParams {
    AwStateDev st[kAwMaxStates];
    int64_t tile0[kAwMaxStates];
    uint64_t second;  // bit i: state i is a second moment
    int nst;
    int64_t ntiles;
};
hipError_t launch_aw_state(const AwStateParams& p, int block, bool f32, bool write, hipStream_t stream);

}  // namespace loco
