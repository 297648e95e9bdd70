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

// Fills a table of the `count` segments that are not empty; describe(d, i) describes segment i.
template <typename Size, typename Describe>
int fill_table(int count, int64_t live, int tile, Size size, Describe describe, void* table, int64_t& tiles,
               hipStream_t st) {
    AwFillParams p;
    memset(&p, 0, sizeof(p));
    p.table = table;
    p.n = live;
    tiles = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t n = size(i);
        if (n > 0) {
            memset(&p.seg[p.count], 0, sizeof(AwSegDev));
            describe(p.seg[p.count], i);
            p.seg[p.count].n = n;
            p.tile0[p.count++] = tiles;
            tiles += (n + tile - 1) / tile;
        }
        if (p.count == kAwFill || (i == count - 1 && p.count > 0)) {
            if (launch_aw_fill(p, st) != hipSuccess) return LOCO_ERR_HIP;
            p.first += p.count;
            p.count = 0;
        }
    }
    return LOCO_OK;
}

constexpr int kAdamwPlan = 0x61647721, kStatePlan = 0x61647722;  // what a plan was made for

int check_adamw_tensors(const loco_adamw_tensor_t* ts, int nt, int param_dtype, int grad_dtype, int bits, int block,
                        const void* table, int64_t& live) {
    const int ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype), ss = bits == 8 ? 1 : 4;
    for (int i = 0; i < nt; ++i) {
        const loco_adamw_tensor_t& t = ts[i];
        if (t.n < 0 || t.n > kMaxElems || !isfinite(t.weight_decay)) return LOCO_ERR_INVALID;
        if (t.n == 0) continue;
        ++live;
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
    if (live > 0 && !table) return LOCO_ERR_INVALID;
    if (live > 0 && !aligned16(table)) return LOCO_ERR_ALIGN;
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
    spans.push_back({range_of(table, live > 0 ? aw_table_bytes(live) : 0), true});
    return any_write_overlap(spans) ? LOCO_ERR_INVALID : LOCO_OK;
}

}  // namespace

LOCO_API int64_t loco_adamw_table_bytes(int n) { return n > 0 ? aw_table_bytes(n) : 0; }

LOCO_API int loco_adamw_plan(const loco_adamw_tensor_t* tensors, int ntensors, loco_dtype_t param_dtype,
                             loco_dtype_t grad_dtype, int state_bits, int block, void* table, int64_t table_bytes,
                             loco_adamw_plan_t* plan, void* stream) {
    if (ntensors < 0 || (ntensors > 0 && !tensors) || !plan) return LOCO_ERR_INVALID;
    if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    if (state_bits != 8 && state_bits != 32) return LOCO_ERR_INVALID;
    if (state_bits == 8) {
        const int st = check_state_block(block);
        if (st != LOCO_OK) return st;
    }
    if (table_bytes < loco_adamw_table_bytes(ntensors)) return LOCO_ERR_INVALID;
    int64_t live = 0, tiles = 0;
    try {
        const int st = check_adamw_tensors(tensors, ntensors, param_dtype, grad_dtype, state_bits, block, table, live);
        if (st != LOCO_OK) return st;
    } catch (const std::bad_alloc&) {
        return LOCO_ERR_INVALID;  // more tensors than the host has memory to check
    }
    const int st = fill_table(
        ntensors, live, kAwTile, [&](int i) { return tensors[i].n; },
        [&](AwSegDev& d, int i) {
            const loco_adamw_tensor_t& t = tensors[i];
            d = {t.param, t.grad, t.m, t.v, t.m_exps, t.v_exps, t.param_bf16, t.n, t.weight_decay, 0};
        },
        table, tiles, (hipStream_t)stream);
    if (st != LOCO_OK) return st;
    *plan = {kAdamwPlan, ntensors, live, tiles, table, tensors, param_dtype, grad_dtype, state_bits, block};
    return LOCO_OK;
}

LOCO_API int loco_adamw_ex(const loco_adamw_plan_t* plan, const loco_adamw_t* options, const float* grad_scale,
                           const loco_adamw_rounding_t* rounding, void* stream) {
    if (!plan || plan->kind != kAdamwPlan || !options) return LOCO_ERR_INVALID;
    const loco_adamw_t& o = *options;
    if (!isfinite(o.lr) || !isfinite(o.eps) || !((float)o.eps > 0.0f) || !isfinite((float)o.eps)) return LOCO_ERR_INVALID;
    if (!(o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0) || o.step < 1) return LOCO_ERR_INVALID;
    const double bias1 = 1.0 - pow(o.beta1, (double)o.step), bias2 = 1.0 - pow(o.beta2, (double)o.step);
    const int64_t* counter = rounding ? rounding->counter : nullptr;
    AwParams p;
    memset(&p, 0, sizeof(p));
    p.table = plan->table;
    p.n = plan->live;
    p.ntiles = plan->tiles;
    p.grad_scale = grad_scale;
    p.lr = o.lr;
    p.beta1 = (float)o.beta1;
    p.omb1 = (float)(1.0 - o.beta1);
    p.beta2 = (float)o.beta2;
    p.omb2 = (float)(1.0 - o.beta2);
    p.step_size = (float)(o.lr / bias1);
    p.root = (float)(1.0 / sqrt(bias2));
    p.eps = (float)o.eps;
    if (rounding) p.key = aw_mix(rounding->seed + (uint64_t)o.step * 0x9E3779B97F4A7C15u);
    p.counter = counter;
    if (!isfinite(p.step_size)) return LOCO_ERR_INVALID;
    const int ps = dtype_size(plan->param_dtype), ss = plan->state_bits == 8 ? 1 : 4;
    const Range scalars[2] = {range_of(grad_scale, grad_scale ? 4 : 0), range_of(counter, counter ? 8 : 0)};
    for (int i = 0; i < plan->ntensors; ++i) {
        const loco_adamw_tensor_t& t = plan->tensors[i];
        if (!isfinite((float)(1.0 - o.lr * t.weight_decay))) return LOCO_ERR_INVALID;
        if ((!grad_scale && !counter) || t.n == 0) continue;
        const int64_t nb = plan->state_bits == 8 ? nblocks(t.n, plan->block) : 0;
        for (const Range& r : scalars)
            if (overlap(r, range_of(t.param, t.n * ps)) || overlap(r, range_of(t.m, t.n * ss)) ||
                overlap(r, range_of(t.v, t.n * ss)) || overlap(r, range_of(t.m_exps, nb)) ||
                overlap(r, range_of(t.v_exps, nb)) || overlap(r, range_of(t.param_bf16, t.param_bf16 ? t.n * 2 : 0)))
                return LOCO_ERR_INVALID;
    }
    if ((grad_scale && !aligned16(grad_scale)) || (counter && !aligned16(counter))) return LOCO_ERR_ALIGN;
    if (p.ntiles == 0) return LOCO_OK;
    return hip_status(launch_aw(p, plan->param_dtype == LOCO_F32, plan->grad_dtype == LOCO_F32,
                                plan->state_bits == 8 ? plan->block : 0, rounding != nullptr, (hipStream_t)stream));
}

LOCO_API int loco_adamw(const loco_adamw_plan_t* plan, const loco_adamw_t* options, const float* grad_scale, void* stream) {
    return loco_adamw_ex(plan, options, grad_scale, nullptr, stream);
}

LOCO_API int loco_adamw_state_plan(const loco_adamw_state_t* states, int nstates, int block, loco_dtype_t dtype,
                                   void* table, int64_t table_bytes, loco_adamw_plan_t* plan, void* stream) {
    if (nstates < 0 || (nstates > 0 && !states) || !dtype_ok(dtype) || !plan) return LOCO_ERR_INVALID;
    int st = check_state_block(block);
    if (st != LOCO_OK) return st;
    if (table_bytes < loco_adamw_table_bytes(nstates)) return LOCO_ERR_INVALID;
    int64_t live = 0, tiles = 0;
    for (int i = 0; i < nstates; ++i) {
        const loco_adamw_state_t& s = states[i];
        if (s.n < 0 || s.n > kMaxElems || (s.moment != 1 && s.moment != 2)) return LOCO_ERR_INVALID;
        if (s.n > 0 && (!s.codes || !s.exps || !s.values)) return LOCO_ERR_INVALID;
        live += s.n > 0;
    }
    if (live > 0 && !table) return LOCO_ERR_INVALID;
    for (int i = 0; i < nstates; ++i) {
        const loco_adamw_state_t& s = states[i];
        if (s.n > 0 && (!aligned16(s.codes) || !aligned16(s.exps) || !aligned16(s.values))) return LOCO_ERR_ALIGN;
    }
    if (live > 0 && !aligned16(table)) return LOCO_ERR_ALIGN;
    try {
        // each may be written, the states by one call and the values by the other
        std::vector<Span> spans;
        spans.reserve(3 * (size_t)nstates + 1);
        for (int i = 0; i < nstates; ++i) {
            const loco_adamw_state_t& s = states[i];
            if (s.n == 0) continue;
            spans.push_back({range_of(s.codes, s.n), true});
            spans.push_back({range_of(s.exps, nblocks(s.n, block)), true});
            spans.push_back({range_of(s.values, s.n * dtype_size(dtype)), true});
        }
        spans.push_back({range_of(table, live > 0 ? aw_table_bytes(live) : 0), true});
        if (any_write_overlap(spans)) return LOCO_ERR_INVALID;
    } catch (const std::bad_alloc&) {
        return LOCO_ERR_INVALID;
    }
    st = fill_table(
        nstates, live, kAwStateTile, [&](int i) { return states[i].n; },
        [&](AwSegDev& d, int i) {
            const loco_adamw_state_t& s = states[i];
            d.param = s.values;
            d.m = s.codes;
            d.mexp = s.exps;
            d.second = s.moment == 2;
        },
        table, tiles, (hipStream_t)stream);
    if (st != LOCO_OK) return st;
    *plan = {kStatePlan, nstates, live, tiles, table, nullptr, dtype, dtype, 8, block};
    return LOCO_OK;
}

namespace {

int adamw_states(const loco_adamw_plan_t* plan, bool write, void* stream) {
    if (!plan || plan->kind != kStatePlan) return LOCO_ERR_INVALID;
    if (plan->tiles == 0) return LOCO_OK;
    return hip_status(launch_aw_state(plan->table, plan->live, plan->tiles, plan->block, plan->param_dtype == LOCO_F32,
                                      write, (hipStream_t)stream));
}

}  // namespace

LOCO_API int loco_adamw_state_read(const loco_adamw_plan_t* plan, void* stream) { return adamw_states(plan, false, stream); }
LOCO_API int loco_adamw_state_write(const loco_adamw_plan_t* plan, void* stream) { return adamw_states(plan, true, stream); }

// ---- the norms around a block -----------------------------------------------------------------

namespace {

bool gate_ok(int kind, const void* gate) {
    return kind >= LOCO_GATE_NONE && kind <= LOCO_GATE_ELEMENT && (kind == LOCO_GATE_NONE) == (gate == nullptr);
}

}  // namespace

LOCO_API int loco_residual_norm(const void* y, const void* residual, loco_dtype_t dtype, const void* gate,
                                loco_gate_t gate_kind, const void* post_weight, const void* weight,
                                loco_dtype_t param_dtype, int64_t rows, int64_t cols, float scale, float eps, void* h,
                                void* out, float* post_rstd, float* rstd, const loco_checkpoint_t* ckpt, void* stream) {
    if (!sizes_ok(rows, cols) || cols < 1) return LOCO_ERR_INVALID;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return LOCO_ERR_INVALID;
    if (!isfinite(eps) || eps < 0.0f || !isfinite(scale)) return LOCO_ERR_INVALID;
    if (ckpt) {
        const int st = check_ckpt(*ckpt);
        if (st != LOCO_OK) return st;
    }
    if (cols > kLnMaxCols) return LOCO_ERR_UNSUPPORTED;
    if (gate_kind < LOCO_GATE_NONE || gate_kind > LOCO_GATE_ELEMENT) return LOCO_ERR_INVALID;
    if (rows == 0) return LOCO_OK;
    if (!gate_ok(gate_kind, gate)) return LOCO_ERR_INVALID;
    if ((!y && !residual) || (!h && !out)) return LOCO_ERR_INVALID;
    if (!y && (gate || post_rstd || post_weight)) return LOCO_ERR_INVALID;
    if (post_weight && !post_rstd) return LOCO_ERR_INVALID;
    if (out ? !rstd : rstd || ckpt || weight) return LOCO_ERR_INVALID;
    const int64_t s = dtype_size(dtype), ps = dtype_size(param_dtype);
    const int st = check_bufs({{y, rows * cols * s, false, false},
                               {residual, rows * cols * s, false, false},
                               {gate, gate_kind == LOCO_GATE_ELEMENT ? rows * cols * s : cols * ps, false, false},
                               {post_weight, cols * ps, false, false},
                               {weight, cols * ps, false, false},
                               {h, rows * cols * s, true, false},
                               {out, rows * cols * s, true, false},
                               {post_rstd, rows * 4, true, false},
                               {rstd, rows * 4, true, false},
                               codes_buf(ckpt, rows, cols, true),
                               exps_buf(ckpt, rows, cols, true)});
    if (st != LOCO_OK) return st;
    const RnParams p = {y, residual, gate, weight, post_weight, h, out, rstd, post_rstd, ckpt_dev(ckpt, cols), rows,
                        (int)cols, scale, eps, gate_kind, dtype == LOCO_F32, param_dtype == LOCO_F32};
    return hip_status(launch_rn(p, (hipStream_t)stream));
}

LOCO_API int64_t loco_residual_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (!sizes_ok(rows, cols) || cols < 1 || cols > kLnMaxCols) return 0;
    return rn_bwd_groups(rows, cols) * 3 * cols * 4;
}

LOCO_API int loco_residual_norm_backward(const void* dout, const void* dh, const void* h, const void* y,
                                         loco_dtype_t dtype, const void* gate, loco_gate_t gate_kind,
                                         const void* post_weight, const void* weight, loco_dtype_t param_dtype,
                                         const float* post_rstd, const float* rstd, int64_t rows, int64_t cols,
                                         float scale, void* dresidual, void* dy, void* dgate, void* dpost_weight,
                                         void* dweight, loco_dtype_t grad_dtype, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
    if (!sizes_ok(rows, cols) || cols < 1) return LOCO_ERR_INVALID;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    if (!isfinite(scale)) return LOCO_ERR_INVALID;
    if (cols > kLnMaxCols) return LOCO_ERR_UNSUPPORTED;
    if (gate_kind < LOCO_GATE_NONE || gate_kind > LOCO_GATE_ELEMENT) return LOCO_ERR_INVALID;
    const bool elements = gate_kind == LOCO_GATE_ELEMENT;
    void* sums[3] = {dweight, dpost_weight, elements ? nullptr : dgate};
    const bool any_sum = sums[0] || sums[1] || sums[2];
    if (rows > 0) {
        if (!gate_ok(gate_kind, gate) || (!dout && !dh)) return LOCO_ERR_INVALID;
        if (dout ? (!h || !rstd) : (dweight != nullptr)) return LOCO_ERR_INVALID;
        if (post_weight && !post_rstd) return LOCO_ERR_INVALID;
        if ((post_rstd || gate) && !y) return LOCO_ERR_INVALID;
        if (dpost_weight && !post_rstd) return LOCO_ERR_INVALID;
        if (!dresidual && !dy && !dgate && !any_sum) return LOCO_ERR_INVALID;
    }
    if (dgate && gate_kind == LOCO_GATE_NONE) return LOCO_ERR_INVALID;
    const int64_t need = any_sum ? loco_residual_norm_backward_workspace(rows, cols) : 0;
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    if (rows == 0 && !any_sum) return LOCO_OK;
    const int64_t s = dtype_size(dtype), ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype);
    const int st = check_bufs({{dout, rows * cols * s, false, false},
                               {dh, rows * cols * s, false, false},
                               {h, rows * cols * s, false, false},
                               {y, rows * cols * s, false, false},
                               {gate, elements ? rows * cols * s : cols * ps, false, false},
                               {post_weight, cols * ps, false, false},
                               {weight, cols * ps, false, false},
                               {post_rstd, rows * 4, false, false},
                               {rstd, rows * 4, false, false},
                               {dresidual, rows * cols * s, true, false},
                               {dy, rows * cols * s, true, false},
                               {dgate, elements ? rows * cols * s : cols * gs, true, false},
                               {dpost_weight, cols * gs, true, false},
                               {dweight, cols * gs, true, false},
                               {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    const RnBwdParams p = {dout, dh, h, y, gate, weight, post_weight, rstd, post_rstd, dresidual, dy,
                           elements ? dgate : nullptr, {sums[0], sums[1], sums[2]}, any_sum ? (float*)workspace : nullptr,
                           rows, (int)cols, scale, gate_kind, dtype == LOCO_F32, param_dtype == LOCO_F32,
                           grad_dtype == LOCO_F32};
    return hip_status(launch_rn_bwd(p, (hipStream_t)stream));
}

// ---- log probabilities of tokens -----------------------------------------------------------------

namespace {

// Sequences of rows of logits as a call gives them.
struct Rows {
    int64_t seqs, rows, vocab;
    int64_t total() const { return seqs * rows; }
    // the elements, from the first to the last, of `width` each, `ld` from row to row and `seq_ld` from sequence to sequence
    int64_t span(int64_t ld, int64_t seq_ld, int64_t width) const {
        return total() > 0 ? (seqs > 1 ? (seqs - 1) * seq_ld : 0) + (rows - 1) * ld + width : 0;
    }
    int64_t gap(int64_t ld, int64_t seq_ld) const { return seqs > 1 ? seq_ld - rows * ld : 0; }
    bool steps_ok(int64_t ld, int64_t seq_ld, int64_t width) const {
        if (ld < width || !sizes_ok(rows, ld)) return false;
        return seqs <= 1 || rows == 0 || (seq_ld >= (rows - 1) * ld + width && sizes_ok(seqs, seq_ld));
    }
};

int check_logits(const Rows& r, int64_t ld, int64_t seq_ld, int64_t target_ld, int dtype, float scale) {
    if (r.seqs < 0 || r.rows < 0 || r.vocab < 1 || !sizes_ok(r.seqs, r.rows) || !r.steps_ok(ld, seq_ld, r.vocab))
        return LOCO_ERR_INVALID;
    if (!r.steps_ok(1, target_ld, 1) || !dtype_ok(dtype)) return LOCO_ERR_INVALID;
    if (!(scale >= 1e-6f && scale <= 1e6f)) return LOCO_ERR_INVALID;
    return r.vocab > kLpMaxVocab || (r.seqs > 1 && r.total() > UINT32_MAX) ? LOCO_ERR_UNSUPPORTED : LOCO_OK;
}

LpSeqs seqs_dev(const Rows& r, int64_t ld, int64_t seq_ld, int64_t dld, int64_t dseq_ld, int64_t target_ld) {
    return {r.seqs > 1 ? (uint32_t)r.rows : 0u, r.gap(ld, seq_ld), r.gap(dld, dseq_ld), r.gap(1, target_ld)};
}

// align: least alignment of all buffers.
int token_logprobs(const void* logits, int dtype, const Rows& r, int64_t ld, int64_t seq_ld, const int64_t* targets,
                   int64_t target_ld, float scale, float* logprob, float* entropy, float* stats, int top,
                   int32_t* top_ids, float* top_logprobs, void* workspace, int64_t workspace_bytes, unsigned align,
                   void* stream) {
    int st = check_logits(r, ld, seq_ld, target_ld, dtype, scale);
    if (st != LOCO_OK) return st;
    if (top < 0) return LOCO_ERR_INVALID;
    if (top > kLpMaxTop) return LOCO_ERR_UNSUPPORTED;
    const int64_t rows = r.total(), need = loco_token_logprobs_workspace(rows, r.vocab, top);
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    if (rows == 0) return LOCO_OK;
    if (!logits || (logprob && !targets) || (!logprob && !entropy && !stats && top == 0)) return LOCO_ERR_INVALID;
    const unsigned size = (unsigned)dtype_size(dtype), a4 = std::max(align, 4u);
    st = check_bufs({{logits, r.span(ld, seq_ld, r.vocab) * size, false, true, std::max(align, size)},
                     {targets, r.span(1, target_ld, 1) * 8, false, false, std::max(align, 8u)},
                     {logprob, rows * 4, true, false, a4},
                     {entropy, rows * 4, true, false, a4},
                     {stats, rows * 8, true, false, a4},
                     {top_ids, rows * top * 4, true, true, a4},
                     {top_logprobs, rows * top * 4, true, true, a4},
                     {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    const int64_t parts = need > 0 ? rows * lp_splits(rows, r.vocab) : 0;
    const LpParams p = {logits, rows, ld, (int)r.vocab, targets, scale, logprob, entropy, stats, top_ids, top_logprobs, top,
                        dtype == LOCO_F32, (f32x4_t*)workspace, (uint64_t*)((char*)workspace + parts * 16),
                        seqs_dev(r, ld, seq_ld, ld, seq_ld, target_ld), 0, 0};
    return hip_status(launch_lp(p, (hipStream_t)stream));
}

int token_logprobs_backward(const void* logits, int dtype, const Rows& r, int64_t ld, int64_t seq_ld,
                            const int64_t* targets, int64_t target_ld, float scale, const float* stats,
                            const float* entropy, const float* dlogprob, const float* dentropy, void* dlogits,
                            int64_t dld, int64_t dseq_ld, unsigned align, void* stream) {
    int st = check_logits(r, ld, seq_ld, target_ld, dtype, scale);
    if (st != LOCO_OK) return st;
    if (!r.steps_ok(dld, dseq_ld, r.vocab)) return LOCO_ERR_INVALID;
    const int64_t rows = r.total();
    if (rows == 0) return LOCO_OK;
    if (!logits || !stats || !dlogits || (!dlogprob && !dentropy)) return LOCO_ERR_INVALID;
    if ((dlogprob && !targets) || (dentropy && !entropy)) return LOCO_ERR_INVALID;
    // in place: each element is read by the lane that then writes it
    const bool in_place = dlogits == logits && dld == ld && (r.seqs == 1 || dseq_ld == seq_ld);
    const unsigned size = (unsigned)dtype_size(dtype), a4 = std::max(align, 4u);
    st = check_bufs({{logits, in_place ? 0 : r.span(ld, seq_ld, r.vocab) * size, false, true, std::max(align, size)},
                     {targets, r.span(1, target_ld, 1) * 8, false, false, std::max(align, 8u)},
                     {stats, rows * 8, false, true, a4},
                     {entropy, rows * 4, false, false, a4},
                     {dlogprob, rows * 4, false, false, a4},
                     {dentropy, rows * 4, false, false, a4},
                     {dlogits, r.span(dld, dseq_ld, r.vocab) * size, true, true, std::max(align, size)}});
    if (st != LOCO_OK) return st;
    const LpBwdParams p = {logits, dlogits, rows, ld, dld, (int)r.vocab, targets, stats, entropy, dlogprob, dentropy, scale,
                           dtype == LOCO_F32, seqs_dev(r, ld, seq_ld, dld, dseq_ld, target_ld)};
    return hip_status(launch_lp_bwd(p, (hipStream_t)stream));
}

}  // namespace

LOCO_API int64_t loco_token_logprobs_workspace(int64_t rows, int64_t vocab, int top) {
    if (rows < 0 || vocab < 1 || vocab > kLpMaxVocab || !sizes_ok(rows, vocab) || top < 0 || top > kLpMaxTop) return 0;
    const int64_t splits = lp_splits(rows, vocab);
    return splits > 1 ? rows * splits * (16 + top * 8) : 0;
}

LOCO_API int loco_token_logprobs(const void* logits, loco_dtype_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                 const int64_t* targets, float scale, float* logprob, float* entropy, float* stats,
                                 int top, int32_t* top_ids, float* top_logprobs, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    return token_logprobs(logits, dtype, {1, rows, vocab}, ld, 0, targets, 0, scale, logprob, entropy, stats, top, top_ids,
                          top_logprobs, workspace, workspace_bytes, 16, stream);
}

LOCO_API int loco_token_logprobs_ex(const void* logits, loco_dtype_t dtype, int64_t seqs, int64_t rows, int64_t vocab,
                                    int64_t ld, int64_t seq_ld, const int64_t* targets, int64_t target_ld, float scale,
                                    float* logprob, float* entropy, float* stats, int top, int32_t* top_ids,
                                    float* top_logprobs, void* workspace, int64_t workspace_bytes, void* stream) {
    return token_logprobs(logits, dtype, {seqs, rows, vocab}, ld, seq_ld, targets, target_ld, scale, logprob, entropy,
                          stats, top, top_ids, top_logprobs, workspace, workspace_bytes, 1, stream);
}

LOCO_API int loco_token_logprobs_backward(const void* logits, loco_dtype_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                          const int64_t* targets, float scale, const float* stats, const float* entropy,
                                          const float* dlogprob, const float* dentropy, void* dlogits, int64_t dld,
                                          void* stream) {
    return token_logprobs_backward(logits, dtype, {1, rows, vocab}, ld, 0, targets, 0, scale, stats, entropy, dlogprob,
                                   dentropy, dlogits, dld, 0, 16, stream);
}

LOCO_API int loco_token_logprobs_backward_ex(const void* logits, loco_dtype_t dtype, int64_t seqs, int64_t rows,
                                             int64_t vocab, int64_t ld, int64_t seq_ld, const int64_t* targets,
                                             int64_t target_ld, float scale, const float* stats, const float* entropy,
                                             const float* dlogprob, const float* dentropy, void* dlogits, int64_t dld,
                                             int64_t dseq_ld, void* stream) {
    return token_logprobs_backward(logits, dtype, {seqs, rows, vocab}, ld, seq_ld, targets, target_ld, scale, stats,
                                   entropy, dlogprob, dentropy, dlogits, dld, dseq_ld, 1, stream);
}
