// C ABI of the operators around a layer's products (a part of abi.hip): AdamW over many tensors,
// the norms around a block, log probabilities of tokens.
#pragma once

#include <new>

#include "loco_checks.hpp"
#include "loco_step_internal.hpp"

using namespace loco;

// ---- AdamW ----------------------------------------------------------------------------------

namespace {

int check_state_block(int block) {
    if (block <= 0) return LOCO_ERR_INVALID;
    return block_ok(block) ? LOCO_OK : LOCO_ERR_UNSUPPORTED;
}

// The tiles of the tensors before index i in one launch; `add` describes tensor i there.
template <typename Add, typename Size, typename Launch>
int launch_batches(int count, int most, Size size, Add add, Launch launch) {
    int i = 0;
    while (i < count) {
        int used = 0;
        int64_t tiles = 0;
        for (; i < count && used < most; ++i) {
            const int64_t n = size(i);
            if (n == 0) continue;
            add(used++, i, tiles);
            tiles += (n + kAwTile - 1) / kAwTile;
        }
        if (used > 0 && launch(used, tiles) != hipSuccess) return LOCO_ERR_HIP;
    }
    return LOCO_OK;
}

int check_adamw_tensors(const loco_adamw_tensor_t* ts, int nt, int param_dtype, int grad_dtype, int bits, int block,
                        double lr, const float* grad_scale) {
    const int ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype), ss = bits == 8 ? 1 : 4;
    for (int i = 0; i < nt; ++i) {
        const loco_adamw_tensor_t& t = ts[i];
        if (t.n < 0 || t.n > kMaxElems || !isfinite((float)(1.0 - lr * t.weight_decay))) return LOCO_ERR_INVALID;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (bits == 8 && (!t.m_exps || !t.v_exps))) return LOCO_ERR_INVALID;
        if (t.param_bf16 && param_dtype != LOCO_F32) return LOCO_ERR_INVALID;
    }
    for (int i = 0; i < nt; ++i) {
        const loco_adamw_tensor_t& t = ts[i];
        if (t.n == 0) continue;
        uintptr_t bits_of = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.m | (uintptr_t)t.v |
                            (uintptr_t)t.param_bf16;
        if (bits == 8) bits_of |= (uintptr_t)t.m_exps | (uintptr_t)t.v_exps;
        if (bits_of & 15u) return LOCO_ERR_ALIGN;
    }
    if (grad_scale && !aligned16(grad_scale)) return LOCO_ERR_ALIGN;
    std::vector<Span> spans;
    spans.reserve(7 * (size_t)nt + 1);
    for (int i = 0; i < nt; ++i) {
        const loco_adamw_tensor_t& t = ts[i];
        if (t.n == 0) continue;
        spans.push_back({range_of(t.param, t.n * ps), true});
        spans.push_back({range_of(t.grad, t.n * gs), false});
        spans.push_back({range_of(t.m, t.n * ss), true});
        spans.push_back({range_of(t.v, t.n * ss), true});
        if (bits == 8) {
            spans.push_back({range_of(t.m_exps, nblocks(t.n, block)), true});
            spans.push_back({range_of(t.v_exps, nblocks(t.n, block)), true});
        }
        if (t.param_bf16) spans.push_back({range_of(t.param_bf16, t.n * 2), true});
    }
    if (grad_scale) spans.push_back({range_of(grad_scale, 4), false});
    return any_write_overlap(spans) ? LOCO_ERR_INVALID : LOCO_OK;
}

}  // namespace

LOCO_API int loco_adamw(const loco_adamw_tensor_t* tensors, int ntensors, loco_dtype_t param_dtype,
                        loco_dtype_t grad_dtype, int state_bits, int block, const loco_adamw_t* options,
                        const float* grad_scale, void* stream) {
    if (ntensors < 0 || (ntensors > 0 && !tensors) || !options) return LOCO_ERR_INVALID;
    if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    if (state_bits != 8 && state_bits != 32) return LOCO_ERR_INVALID;
    if (state_bits == 8) {
        const int st = check_state_block(block);
        if (st != LOCO_OK) return st;
    }
    const loco_adamw_t& o = *options;
    if (!isfinite(o.lr) || !isfinite(o.eps) || !((float)o.eps > 0.0f) || !isfinite((float)o.eps)) return LOCO_ERR_INVALID;
    if (!(o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0) || o.step < 1) return LOCO_ERR_INVALID;
    const double bias1 = 1.0 - pow(o.beta1, (double)o.step), bias2 = 1.0 - pow(o.beta2, (double)o.step);
    AwParams p;
    memset(&p, 0, sizeof(p));
    p.grad_scale = grad_scale;
    p.beta1 = (float)o.beta1;
    p.omb1 = (float)(1.0 - o.beta1);
    p.beta2 = (float)o.beta2;
    p.omb2 = (float)(1.0 - o.beta2);
    p.step_size = (float)(o.lr / bias1);
    p.root = (float)(1.0 / sqrt(bias2));
    p.eps = (float)o.eps;
    if (!isfinite(p.step_size)) return LOCO_ERR_INVALID;
    try {
        const int st = check_adamw_tensors(tensors, ntensors, param_dtype, grad_dtype, state_bits, block, o.lr,
                                           grad_scale);
        if (st != LOCO_OK) return st;
    } catch (const std::bad_alloc&) {
        return LOCO_ERR_INVALID;  // more tensors than the host has memory to check
    }
    return launch_batches(
        ntensors, kAwMaxSeg, [&](int i) { return tensors[i].n; },
        [&](int at, int i, int64_t tile0) {
            const loco_adamw_tensor_t& t = tensors[i];
            p.seg[at] = {t.param, t.grad, t.m, t.v, t.m_exps, t.v_exps, t.param_bf16, t.n};
            p.tile0[at] = tile0;
            p.decay[at] = (float)(1.0 - o.lr * t.weight_decay);
        },
        [&](int used, int64_t tiles) {
            p.nseg = used;
            p.ntiles = tiles;
            return launch_aw(p, param_dtype == LOCO_F32, grad_dtype == LOCO_F32, state_bits == 8 ? block : 0,
                             (hipStream_t)stream);
        });
}

namespace {

int adamw_states(const loco_adamw_state_t* states, int nstates, int block, int dtype, bool write, void* stream) {
    if (nstates < 0 || (nstates > 0 && !states) || !dtype_ok(dtype)) return LOCO_ERR_INVALID;
    int st = check_state_block(block);
    if (st != LOCO_OK) return st;
    for (int i = 0; i < nstates; ++i) {
        const loco_adamw_state_t& s = states[i];
        if (s.n < 0 || s.n > kMaxElems || (s.moment != 1 && s.moment != 2)) return LOCO_ERR_INVALID;
        if (s.n > 0 && (!s.codes || !s.exps || !s.values)) return LOCO_ERR_INVALID;
    }
    for (int i = 0; i < nstates; ++i) {
        const loco_adamw_state_t& s = states[i];
        if (s.n > 0 && (!aligned16(s.codes) || !aligned16(s.exps) || !aligned16(s.values))) return LOCO_ERR_ALIGN;
    }
    try {
        std::vector<Span> spans;
        spans.reserve(3 * (size_t)nstates);
        for (int i = 0; i < nstates; ++i) {
            const loco_adamw_state_t& s = states[i];
            if (s.n == 0) continue;
            spans.push_back({range_of(s.codes, s.n), write});
            spans.push_back({range_of(s.exps, nblocks(s.n, block)), write});
            spans.push_back({range_of(s.values, s.n * dtype_size(dtype)), !write});
        }
        if (any_write_overlap(spans)) return LOCO_ERR_INVALID;
    } catch (const std::bad_alloc&) {
        return LOCO_ERR_INVALID;
    }
    AwStateParams p;
    memset(&p, 0, sizeof(p));
    return launch_batches(
        nstates, kAwMaxStates, [&](int i) { return states[i].n; },
        [&](int at, int i, int64_t tile0) {
            const loco_adamw_state_t& s = states[i];
            p.st[at] = {s.codes, s.exps, s.values, s.n};
            p.tile0[at] = tile0;
            p.second = (at == 0 ? 0u : p.second) | ((uint64_t)(s.moment == 2) << at);
        },
        [&](int used, int64_t tiles) {
            p.nst = used;
            p.ntiles = tiles;
            return launch_aw_state(p, block, dtype == LOCO_F32, write, (hipStream_t)stream);
        });
}

}  // namespace

LOCO_API int loco_adamw_state_read(const loco_adamw_state_t* states, int nstates, int block, loco_dtype_t dtype,
                                   void* stream) {
    return adamw_states(states, nstates, block, dtype, false, stream);
}
LOCO_API int loco_adamw_state_write(const loco_adamw_state_t* states, int nstates, int block, loco_dtype_t dtype,
                                    void* stream) {
    return adamw_states(states, nstates, block, dtype, true, stream);
}
