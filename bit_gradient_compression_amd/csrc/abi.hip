// C ABI of the library: argument validation on the host, then one launch per call on
// the caller's stream.  Validation runs before any HIP call, so an error status means
// nothing was launched and nothing was written.

#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <vector>

#include "loco.h"
#include "loco_internal.hpp"
#include "loco_layer_internal.hpp"

#define LOCO_API extern "C" __attribute__((visibility("default")))

namespace loco {

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool bits_ok(int bits) { return bits == 2 || bits == 4 || bits == 8; }
bool block_ok(int block) { return block == 64 || block == 128 || block == 256 || block == 512; }
bool dtype_ok(int d) { return d == LOCO_F32 || d == LOCO_BF16; }
int dtype_size(int d) { return d == LOCO_I8 ? 1 : (d == LOCO_BF16 ? 2 : 4); }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
Range range_of(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// True if some written range overlaps any other range (written or read); read-only
// ranges may overlap each other.  Empty ranges never overlap.  Sorted by start, a range
// overlaps an earlier one exactly when it starts before the largest end seen so far.
struct Span {
    Range r;
    bool written;
};
bool any_write_overlap(std::vector<Span>& v) {
    std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.r.lo < b.r.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Span& s : v) {
        if (s.r.lo >= s.r.hi) continue;
        if (s.r.lo < (s.written ? end_any : end_written)) return true;
        end_any = std::max(end_any, s.r.hi);
        if (s.written) end_written = std::max(end_written, s.r.hi);
    }
    return false;
}

int64_t code_bytes(int64_t n, int bits) { return (n * bits + 7) / 8; }
int64_t nblocks(int64_t n, int block) { return (n + block - 1) / block; }

// Sizes beyond this are refused: far above any device memory, and safe from overflow in
// the byte arithmetic above.
constexpr int64_t kMaxElems = (int64_t)1 << 52;

}  // namespace
}  // namespace loco

using namespace loco;

LOCO_API int loco_version(void) { return 10200; }

LOCO_API const char* loco_status_string(int status) {
    switch (status) {
        case LOCO_OK: return "LOCO_OK";
        case LOCO_ERR_INVALID: return "LOCO_ERR_INVALID: invalid argument";
        case LOCO_ERR_ALIGN: return "LOCO_ERR_ALIGN: device pointer not 16-byte aligned";
        case LOCO_ERR_UNSUPPORTED: return "LOCO_ERR_UNSUPPORTED: valid but not built";
        case LOCO_ERR_HIP: return "LOCO_ERR_HIP: kernel launch failed";
    }
    return "unknown status";
}

namespace {

// Shared body of both compensate-quantize entry points.
int compensate_quantize(const loco_cq_segment_t* segs, int nseg, int grad_dtype, int err_dtype,
                        const loco_cq_options_t& o, hipStream_t st) {
    if (nseg < 0 || (nseg > 0 && !segs)) return LOCO_ERR_INVALID;
    if (!dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    if (!dtype_ok(err_dtype) && err_dtype != LOCO_I8) return LOCO_ERR_INVALID;
    const int bits = o.bits, block = o.block;
    if (bits < 1 || bits > 8) return LOCO_ERR_INVALID;
    if (!bits_ok(bits)) return LOCO_ERR_UNSUPPORTED;
    if (!isfinite(o.beta) || o.beta < 0.0f || o.beta > 1.0f) return LOCO_ERR_INVALID;
    if (!isfinite(o.fixed_scale) || o.fixed_scale < 0.0f) return LOCO_ERR_INVALID;
    float err_step = 0.0f;
    if (err_dtype == LOCO_I8) {
        // s_e > 0 and 256/s_e finite: the decode e8*fl(1/s_e) and its biased form stay finite.
        if (!isfinite(o.err_scale) || !(o.err_scale > 0.0f)) return LOCO_ERR_INVALID;
        err_step = 1.0f / o.err_scale;
        if (!isfinite(256.0f * err_step)) return LOCO_ERR_INVALID;
    }
    const bool fixed = o.fixed_scale > 0.0f;
    if (!fixed) {
        if (block <= 0) return LOCO_ERR_INVALID;
        if (!block_ok(block)) return LOCO_ERR_UNSUPPORTED;
    }
    const int gs = dtype_size(grad_dtype), es = dtype_size(err_dtype);
    int64_t live = 0;
    for (int i = 0; i < nseg; ++i) {
        const loco_cq_segment_t& s = segs[i];
        if (s.n < 0 || s.n > kMaxElems) return LOCO_ERR_INVALID;
        if (s.n == 0) continue;
        if (!s.grad || !s.err || !s.codes || (!fixed && !s.absmax)) return LOCO_ERR_INVALID;
        if (!aligned16(s.grad) || !aligned16(s.err) || !aligned16(s.codes) || (!fixed && !aligned16(s.absmax)))
            return LOCO_ERR_ALIGN;
        Range r[4] = {range_of(s.grad, s.n * gs), range_of(s.err, s.n * es),
                      range_of(s.codes, code_bytes(s.n, bits)),
                      range_of(s.absmax, fixed ? 0 : nblocks(s.n, block) * 4)};
        for (int a = 0; a < 4; ++a)
            for (int b = a + 1; b < 4; ++b)
                if (overlap(r[a], r[b])) return LOCO_ERR_INVALID;
        ++live;
    }
    if (live == 0) return LOCO_OK;
    // across segments: no buffer the call writes (any segment's err, codes, absmax) may overlap another
    // buffer of the call; gradients are only read and may overlap each other
    std::vector<Span> spans;
    spans.reserve(4 * live);
    for (int i = 0; i < nseg; ++i) {
        const loco_cq_segment_t& s = segs[i];
        if (s.n == 0) continue;
        spans.push_back({range_of(s.grad, s.n * gs), false});
        spans.push_back({range_of(s.err, s.n * es), true});
        spans.push_back({range_of(s.codes, code_bytes(s.n, bits)), true});
        if (!fixed) spans.push_back({range_of(s.absmax, nblocks(s.n, block) * 4), true});
    }
    if (any_write_overlap(spans)) return LOCO_ERR_INVALID;

    CqParams p;
    memset(&p, 0, sizeof(p));
    p.beta = o.beta;
    p.omega = 1.0f - o.beta;
    if (fixed) {
        p.fixed_inv = o.fixed_scale;
        p.fixed_step = 1.0f / o.fixed_scale;
    }
    if (err_dtype == LOCO_I8) {
        p.err_scale = o.err_scale;
        p.err_step = err_step;
    }
    p.reset = o.reset_error != 0;
    const int64_t tile = cq_tile_elems(err_dtype);
    int i = 0;
    while (i < nseg) {
        p.nseg = 0;
        p.ntiles = 0;
        for (; i < nseg && p.nseg < kCqMaxSeg; ++i) {
            const loco_cq_segment_t& s = segs[i];
            if (s.n == 0) continue;
            CqSegDev& d = p.seg[p.nseg++];
            d.g = s.grad;
            d.e = s.err;
            d.codes = s.codes;
            d.absmax = s.absmax;
            d.n = s.n;
            d.tile0 = p.ntiles;
            p.ntiles += (s.n + tile - 1) / tile;
        }
        if (p.nseg == 0) break;
        if (launch_cq(p, grad_dtype, err_dtype, bits, block, fixed, st) != hipSuccess) return LOCO_ERR_HIP;
    }
    return LOCO_OK;
}

}  // namespace

LOCO_API int loco_compensate_quantize(const loco_cq_segment_t* segs, int nseg,
                                      loco_dtype_t grad_dtype, loco_dtype_t err_dtype,
                                      int bits, int block, float beta, float fixed_scale,
                                      void* stream) {
    if (err_dtype == LOCO_I8) return LOCO_ERR_INVALID;  // needs s_e: use the _ex entry point
    loco_cq_options_t o;
    memset(&o, 0, sizeof(o));
    o.bits = bits;
    o.block = block;
    o.beta = beta;
    o.fixed_scale = fixed_scale;
    return compensate_quantize(segs, nseg, grad_dtype, err_dtype, o, (hipStream_t)stream);
}

LOCO_API int loco_compensate_quantize_ex(const loco_cq_segment_t* segs, int nseg,
                                         loco_dtype_t grad_dtype, loco_dtype_t err_dtype,
                                         const loco_cq_options_t* opt, void* stream) {
    if (!opt) return LOCO_ERR_INVALID;
    return compensate_quantize(segs, nseg, grad_dtype, err_dtype, *opt, (hipStream_t)stream);
}

namespace {

// Checks shared by both dequant-reduce entry points; fills the payload part of p.
int dr_setup(const loco_payload_t* peers, int npeers, int64_t n, int bits, int block, float fixed_scale,
             float out_scale, DrParams& p, bool& fixed) {
    if (n < 0 || n > kMaxElems) return LOCO_ERR_INVALID;
    if (npeers < 1 || !peers) return LOCO_ERR_INVALID;
    if (npeers > kDrMaxPeers) return LOCO_ERR_UNSUPPORTED;
    if (bits < 1 || bits > 8) return LOCO_ERR_INVALID;
    if (!bits_ok(bits)) return LOCO_ERR_UNSUPPORTED;
    if (!isfinite(fixed_scale) || fixed_scale < 0.0f) return LOCO_ERR_INVALID;
    if (!isfinite(out_scale)) return LOCO_ERR_INVALID;
    fixed = fixed_scale > 0.0f;
    if (!fixed) {
        if (block <= 0) return LOCO_ERR_INVALID;
        if (!block_ok(block)) return LOCO_ERR_UNSUPPORTED;
    }
    memset(&p, 0, sizeof(p));
    for (int i = 0; i < npeers; ++i) {
        if (!peers[i].codes || (!fixed && !peers[i].absmax)) return LOCO_ERR_INVALID;
        if (!aligned16(peers[i].codes) || (!fixed && !aligned16(peers[i].absmax))) return LOCO_ERR_ALIGN;
        p.peer[i].codes = peers[i].codes;
        p.peer[i].absmax = peers[i].absmax;
    }
    for (int i = npeers; i < npeers + kDrPeerBatch; ++i) p.peer[i] = p.peer[npeers - 1];
    p.npeers = npeers;
    p.n = n;
    p.fixed_step = fixed ? 1.0f / fixed_scale : 0.0f;
    p.out_scale = out_scale;
    return LOCO_OK;
}

// An output range must not overlap any peer's payload.
bool overlaps_payloads(const loco_payload_t* peers, int npeers, int64_t n, int bits, int block, bool fixed, Range r) {
    for (int i = 0; i < npeers; ++i) {
        if (overlap(r, range_of(peers[i].codes, code_bytes(n, bits)))) return true;
        if (!fixed && overlap(r, range_of(peers[i].absmax, nblocks(n, block) * 4))) return true;
    }
    return false;
}

}  // namespace

LOCO_API int loco_dequant_reduce(const loco_payload_t* peers, int npeers, int64_t n, int bits,
                                 int block, float fixed_scale, float out_scale, void* out,
                                 loco_dtype_t out_dtype, void* stream) {
    DrParams p;
    bool fixed = false;
    const int st = dr_setup(peers, npeers, n, bits, block, fixed_scale, out_scale, p, fixed);
    if (st != LOCO_OK) return st;
    if (!dtype_ok(out_dtype)) return LOCO_ERR_INVALID;
    if (n == 0) return LOCO_OK;
    if (!out) return LOCO_ERR_INVALID;
    if (!aligned16(out)) return LOCO_ERR_ALIGN;
    if (overlaps_payloads(peers, npeers, n, bits, block, fixed, range_of(out, n * dtype_size(out_dtype))))
        return LOCO_ERR_INVALID;
    const int mode = out_dtype == LOCO_BF16 ? kDrOutBf16 : kDrOutF32;
    p.ntiles = (n + dr_tile_elems(mode) - 1) / dr_tile_elems(mode);
    p.out = out;
    if (launch_dr(p, bits, block, fixed, mode, (hipStream_t)stream) != hipSuccess) return LOCO_ERR_HIP;
    return LOCO_OK;
}

LOCO_API int loco_dequant_reduce_adam(const loco_payload_t* peers, int npeers, int64_t n, int bits, int block,
                                      float fixed_scale, float out_scale, const loco_adam_t* adam, float* param,
                                      float* m, float* v, uint16_t* param_bf16, void* stream) {
    DrParams p;
    bool fixed = false;
    const int st = dr_setup(peers, npeers, n, bits, block, fixed_scale, out_scale, p, fixed);
    if (st != LOCO_OK) return st;
    if (!adam) return LOCO_ERR_INVALID;
    const loco_adam_t& a = *adam;
    if (!isfinite(a.lr) || !isfinite(a.beta1) || !isfinite(a.beta2) || !isfinite(a.delta)) return LOCO_ERR_INVALID;
    if (a.beta1 < 0.0f || a.beta1 > 1.0f || a.beta2 < 0.0f || a.beta2 > 1.0f || !(a.delta > 0.0f))
        return LOCO_ERR_INVALID;
    if (n == 0) return LOCO_OK;
    if (!param || !m || !v) return LOCO_ERR_INVALID;
    if (!aligned16(param) || !aligned16(m) || !aligned16(v) || (param_bf16 && !aligned16(param_bf16)))
        return LOCO_ERR_ALIGN;
    Range r[4] = {range_of(param, n * 4), range_of(m, n * 4), range_of(v, n * 4),
                  range_of(param_bf16, param_bf16 ? n * 2 : 0)};
    for (int x = 0; x < 4; ++x) {
        for (int y = x + 1; y < 4; ++y)
            if (overlap(r[x], r[y])) return LOCO_ERR_INVALID;
        if (overlaps_payloads(peers, npeers, n, bits, block, fixed, r[x])) return LOCO_ERR_INVALID;
    }
    p.ntiles = (n + dr_tile_elems(kDrOutAdam) - 1) / dr_tile_elems(kDrOutAdam);
    p.theta = param;
    p.m = m;
    p.v = v;
    p.theta_bf16 = param_bf16;
    p.lr = a.lr;
    p.beta1 = a.beta1;
    p.omb1 = 1.0f - a.beta1;
    p.beta2 = a.beta2;
    p.omb2 = 1.0f - a.beta2;
    p.delta = a.delta;
    if (launch_dr(p, bits, block, fixed, kDrOutAdam, (hipStream_t)stream) != hipSuccess) return LOCO_ERR_HIP;
    return LOCO_OK;
}

LOCO_API int loco_topk_quantize(const float* grad, float* err, int64_t n, int chunk, int k, int bits,
                                float ef_decay, uint16_t* idx, uint8_t* codes, float* absmax,
                                void* stream) {
    if (n < 0 || n > kMaxElems) return LOCO_ERR_INVALID;
    if (chunk <= 0 || chunk > 65536) return LOCO_ERR_INVALID;
    if (k < 1 || k > chunk) return LOCO_ERR_INVALID;
    if (bits < 1 || bits > 8) return LOCO_ERR_INVALID;
    if (!isfinite(ef_decay) || ef_decay < 0.0f || ef_decay > 1.0f) return LOCO_ERR_INVALID;
    if (!bits_ok(bits)) return LOCO_ERR_UNSUPPORTED;
    if (chunk != 256 && chunk != 512 && chunk != 1024 && chunk != 2048 && chunk != 4096)
        return LOCO_ERR_UNSUPPORTED;
    if (n == 0) return LOCO_OK;
    if (!grad || !err || !idx || !codes || !absmax) return LOCO_ERR_INVALID;
    if (!aligned16(grad) || !aligned16(err) || !aligned16(idx) || !aligned16(codes) || !aligned16(absmax))
        return LOCO_ERR_ALIGN;
    const int64_t chunks = (n + chunk - 1) / chunk;
    Range r[5] = {range_of(grad, n * 4), range_of(err, n * 4), range_of(idx, chunks * k * 2),
                  range_of(codes, chunks * code_bytes(k, bits)), range_of(absmax, chunks * 4)};
    for (int a = 0; a < 5; ++a)
        for (int b = a + 1; b < 5; ++b)
            if (overlap(r[a], r[b])) return LOCO_ERR_INVALID;
    TkParams p;
    p.g = grad;
    p.e = err;
    p.n = n;
    p.k = k;
    p.decay = ef_decay;
    p.idx = idx;
    p.codes = codes;
    p.absmax = absmax;
    if (launch_tk(p, chunk, bits, (hipStream_t)stream) != hipSuccess) return LOCO_ERR_HIP;
    return LOCO_OK;
}

LOCO_API int loco_sparse_aggregate(const loco_sparse_payload_t* peers, int npeers, int64_t n, int chunk, int k,
                                   int bits, float out_scale, void* out, loco_dtype_t out_dtype, void* stream) {
    if (n < 0 || n > kMaxElems) return LOCO_ERR_INVALID;
    if (npeers < 1 || !peers) return LOCO_ERR_INVALID;
    if (npeers > kDrMaxPeers) return LOCO_ERR_UNSUPPORTED;
    if (chunk <= 0 || chunk > 65536) return LOCO_ERR_INVALID;
    if (k < 1 || k > chunk) return LOCO_ERR_INVALID;
    if (bits < 1 || bits > 8) return LOCO_ERR_INVALID;
    if (!bits_ok(bits)) return LOCO_ERR_UNSUPPORTED;
    if (chunk != 256 && chunk != 512 && chunk != 1024 && chunk != 2048 && chunk != 4096)
        return LOCO_ERR_UNSUPPORTED;
    if (!isfinite(out_scale)) return LOCO_ERR_INVALID;
    if (!dtype_ok(out_dtype)) return LOCO_ERR_INVALID;
    if (n == 0) return LOCO_OK;
    if (!out) return LOCO_ERR_INVALID;
    if (!aligned16(out)) return LOCO_ERR_ALIGN;
    const int64_t chunks = (n + chunk - 1) / chunk;
    const Range ro = range_of(out, n * dtype_size(out_dtype));
    for (int i = 0; i < npeers; ++i) {
        const loco_sparse_payload_t& pe = peers[i];
        if (!pe.idx || !pe.codes || !pe.absmax) return LOCO_ERR_INVALID;
        if (!aligned16(pe.idx) || !aligned16(pe.codes) || !aligned16(pe.absmax)) return LOCO_ERR_ALIGN;
        if (overlap(ro, range_of(pe.idx, chunks * k * 2)) || overlap(ro, range_of(pe.codes, chunks * code_bytes(k, bits))) ||
            overlap(ro, range_of(pe.absmax, chunks * 4)))
            return LOCO_ERR_INVALID;
    }
    SaParams p;
    memset(&p, 0, sizeof(p));
    for (int i = 0; i < npeers; ++i) {
        p.peer[i].idx = peers[i].idx;
        p.peer[i].codes = peers[i].codes;
        p.peer[i].absmax = peers[i].absmax;
    }
    p.npeers = npeers;
    p.k = k;
    p.cbytes = (int)code_bytes(k, bits);
    p.n = n;
    p.nchunks = chunks;
    p.out_scale = out_scale;
    p.out = out;
    if (launch_sa(p, chunk, bits, out_dtype == LOCO_BF16, (hipStream_t)stream) != hipSuccess) return LOCO_ERR_HIP;
    return LOCO_OK;
}

// ---- layer operators --------------------------------------------------------------------

namespace loco {

namespace {

bool act_ok(int a) { return a >= LOCO_ACT_NONE && a <= LOCO_ACT_SILU; }
int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// One buffer of a call.  `needed`: a null pointer is an error (of an empty buffer it is not).
struct Buf {
    const void* p;
    int64_t bytes;
    bool written, needed;
};

int check_bufs(std::initializer_list<Buf> bufs) {
    for (const Buf& b : bufs)
        if (b.needed && b.bytes > 0 && !b.p) return LOCO_ERR_INVALID;
    for (const Buf& b : bufs)
        if (b.p && b.bytes > 0 && !aligned16(b.p)) return LOCO_ERR_ALIGN;
    // no buffer that is written may overlap another buffer of the call
    for (const Buf& a : bufs)
        for (const Buf& b : bufs) {
            if (&a == &b || !a.written || !a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) continue;
            if (overlap(range_of(a.p, a.bytes), range_of(b.p, b.bytes))) return LOCO_ERR_INVALID;
        }
    return LOCO_OK;
}

// Rows and columns whose product, in bytes, fits far inside 64 bits.
bool sizes_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && rows <= ((int64_t)1 << 40) && cols <= ((int64_t)1 << 40) &&
           (cols == 0 || rows <= ((int64_t)1 << 52) / cols);
}

int check_ckpt(const loco_checkpoint_t& c) {
    if (c.block < 1) return LOCO_ERR_INVALID;
    return c.block == 32 || c.block == 64 ? LOCO_OK : LOCO_ERR_UNSUPPORTED;
}
CkptDev ckpt_dev(const loco_checkpoint_t* c, int64_t cols) {
    if (!c) return {nullptr, nullptr, 0, 0};
    return {c->codes, c->exps, c->block == 64, nblocks(cols, c->block)};
}
Buf codes_buf(const loco_checkpoint_t* c, int64_t rows, int64_t cols, bool written) {
    return {c ? c->codes : nullptr, c ? rows * cols : 0, written, true};
}
Buf exps_buf(const loco_checkpoint_t* c, int64_t rows, int64_t cols, bool written) {
    return {c ? c->exps : nullptr, c ? rows * nblocks(cols, c->block) : 0, written, true};
}

int hip_status(hipError_t e) { return e == hipSuccess ? LOCO_OK : LOCO_ERR_HIP; }

// Features of a product: counts that the tile kernels' 32-bit offsets hold.
int check_product(int64_t rows, int64_t out_features, int64_t in_features) {
    if (out_features < 0 || in_features < 0) return LOCO_ERR_INVALID;
    if (!sizes_ok(rows, out_features) || !sizes_ok(rows, in_features)) return LOCO_ERR_INVALID;
    constexpr int64_t kMost = (int64_t)1 << 36;  // elements of one matrix: a grid holds the tiles of as many
    const int64_t widest = std::max(out_features, in_features);
    if (widest > kMmMaxFeatures || rows > ((int64_t)1 << 28) || rows * widest > kMost ||
        out_features * in_features > kMost)
        return LOCO_ERR_UNSUPPORTED;
    return LOCO_OK;
}

}  // namespace
}  // namespace loco

LOCO_API int loco_layer_norm(const void* x, loco_dtype_t dtype, const void* weight, const void* bias,
                             loco_dtype_t param_dtype, int64_t rows, int64_t cols, float eps, void* y, float* mean,
                             float* rstd, const loco_checkpoint_t* ckpt, void* stream) {
    if (!sizes_ok(rows, cols) || cols < 1) return LOCO_ERR_INVALID;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return LOCO_ERR_INVALID;
    if (!isfinite(eps) || eps < 0.0f) return LOCO_ERR_INVALID;
    if (ckpt) {
        const int st = check_ckpt(*ckpt);
        if (st != LOCO_OK) return st;
    }
    if (cols > kLnMaxCols) return LOCO_ERR_UNSUPPORTED;
    if (rows == 0) return LOCO_OK;
    const int64_t s = dtype_size(dtype), ps = dtype_size(param_dtype);
    const int st = check_bufs({{x, rows * cols * s, false, true},
                               {weight, cols * ps, false, false},
                               {bias, cols * ps, false, false},
                               {y, rows * cols * s, true, true},
                               {mean, rows * 4, true, true},
                               {rstd, rows * 4, true, true},
                               codes_buf(ckpt, rows, cols, true),
                               exps_buf(ckpt, rows, cols, true)});
    if (st != LOCO_OK) return st;
    LnParams p = {x, weight, bias, y, mean, rstd, ckpt_dev(ckpt, cols), rows, (int)cols, eps,
                  dtype == LOCO_F32, param_dtype == LOCO_F32};
    return hip_status(launch_ln(p, (hipStream_t)stream));
}

LOCO_API int64_t loco_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > kLnMaxCols) return 0;
    return ln_bwd_groups(rows, cols) * 2 * cols * 4;
}

LOCO_API int loco_layer_norm_backward(const void* dy, const void* x, loco_dtype_t dtype, const void* weight,
                                      loco_dtype_t param_dtype, const float* mean, const float* rstd,
                                      const void* residual, int64_t rows, int64_t cols, void* dx, void* dweight,
                                      void* dbias, loco_dtype_t grad_dtype, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
    if (!sizes_ok(rows, cols) || cols < 1) return LOCO_ERR_INVALID;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    if (cols > kLnMaxCols) return LOCO_ERR_UNSUPPORTED;
    const bool sums = dweight || dbias;
    const int64_t need = sums ? loco_layer_norm_backward_workspace(rows, cols) : 0;
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    if (rows == 0 && !sums) return LOCO_OK;
    const int64_t s = dtype_size(dtype), gs = dtype_size(grad_dtype);
    const int st = check_bufs({{dy, rows * cols * s, false, true},
                               {x, rows * cols * s, false, true},
                               {weight, cols * dtype_size(param_dtype), false, false},
                               {mean, rows * 4, false, true},
                               {rstd, rows * 4, false, true},
                               {residual, rows * cols * s, false, false},
                               {dx, rows * cols * s, true, true},
                               {dweight, cols * gs, true, false},
                               {dbias, cols * gs, true, false},
                               {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    LnBwdParams p = {dy, x, weight, mean, rstd, residual, dx, dweight, dbias, sums ? (float*)workspace : nullptr,
                     rows, (int)cols, dtype == LOCO_F32, param_dtype == LOCO_F32, grad_dtype == LOCO_F32};
    return hip_status(launch_ln_bwd(p, (hipStream_t)stream));
}

LOCO_API int loco_checkpoint_write(const void* x, loco_dtype_t dtype, int64_t rows, int64_t cols,
                                   const loco_checkpoint_t* ckpt, void* stream) {
    if (!ckpt || !sizes_ok(rows, cols) || !dtype_ok(dtype)) return LOCO_ERR_INVALID;
    int st = check_ckpt(*ckpt);
    if (st != LOCO_OK) return st;
    if (rows == 0 || cols == 0) return LOCO_OK;
    st = check_bufs({{x, rows * cols * dtype_size(dtype), false, true},
                     codes_buf(ckpt, rows, cols, true),
                     exps_buf(ckpt, rows, cols, true)});
    if (st != LOCO_OK) return st;
    return hip_status(launch_ckpt_write(x, dtype == LOCO_F32, rows, cols, ckpt_dev(ckpt, cols), (hipStream_t)stream));
}

LOCO_API int loco_checkpoint_read(const loco_checkpoint_t* ckpt, int64_t rows, int64_t cols, loco_act_t act, void* out,
                                  loco_dtype_t out_dtype, void* stream) {
    if (!ckpt || !sizes_ok(rows, cols) || !dtype_ok(out_dtype) || !act_ok(act)) return LOCO_ERR_INVALID;
    int st = check_ckpt(*ckpt);
    if (st != LOCO_OK) return st;
    if (rows == 0 || cols == 0) return LOCO_OK;
    st = check_bufs({{out, rows * cols * dtype_size(out_dtype), true, true},
                     codes_buf(ckpt, rows, cols, false),
                     exps_buf(ckpt, rows, cols, false)});
    if (st != LOCO_OK) return st;
    return hip_status(
        launch_ckpt_read(ckpt_dev(ckpt, cols), rows, cols, act, out, cols, out_dtype == LOCO_F32, false,
                         (hipStream_t)stream));
}

namespace {

// The three products of a linear layer, without their epilogues.
MmParams product(const uint16_t* a, const uint16_t* b, int64_t m, int64_t n, int64_t k, bool a_kmajor, bool b_kmajor) {
    MmParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.b = b;
    p.m = m;
    p.n = n;
    p.k = k;
    p.a_kmajor = a_kmajor;
    p.b_kmajor = b_kmajor;
    return p;
}
MmParams forward_product(const uint16_t* x, const uint16_t* w, int64_t rows, int64_t n, int64_t k) {
    return product(x, w, rows, n, k, true, true);
}
MmParams input_grad_product(const uint16_t* dy, const uint16_t* w, int64_t rows, int64_t n, int64_t k) {
    return product(dy, w, rows, k, n, true, false);
}
// The second operand is the checkpoint decoded to bf16 [rows, mm_padded(k)] in the workspace.
MmParams weight_grad_product(const uint16_t* dy, const uint16_t* a, int64_t rows, int64_t n, int64_t k) {
    MmParams p = product(dy, a, n, k, rows, false, false);
    p.b_ld = mm_padded(k);
    return p;
}

// The workspace of the weight gradient: the product's, the bias gradient's partial sums, the
// decoded checkpoint.
struct WeightGradSpace {
    int64_t product, sums, decoded;
    int64_t bytes() const { return product + sums + decoded; }
};
WeightGradSpace weight_grad_space(int64_t rows, int64_t n, int64_t k) {
    if (n == 0) return {0, 0, 0};
    return {round16(mm_workspace(weight_grad_product(nullptr, nullptr, rows, n, k), false)),
            round16(col_sum_groups(rows, n) * n * 4), round16(rows * mm_padded(k) * 2)};
}

}  // namespace

LOCO_API int64_t loco_linear_workspace(int64_t rows, int64_t out_features, int64_t in_features) {
    if (check_product(rows, out_features, in_features) != LOCO_OK) return 0;
    return mm_workspace(forward_product(nullptr, nullptr, rows, out_features, in_features), true);
}

LOCO_API int loco_linear(const uint16_t* x, const uint16_t* weight, const uint16_t* bias, const uint16_t* residual,
                         int64_t rows, int64_t out_features, int64_t in_features, loco_act_t act, void* out,
                         loco_dtype_t out_dtype, const loco_checkpoint_t* ckpt, void* workspace,
                         int64_t workspace_bytes, void* stream) {
    if (!act_ok(act) || !dtype_ok(out_dtype)) return LOCO_ERR_INVALID;
    int st = ckpt ? check_ckpt(*ckpt) : LOCO_OK;
    if (st != LOCO_OK) return st;
    st = check_product(rows, out_features, in_features);
    if (st != LOCO_OK) return st;
    if (rows == 0 || out_features == 0) return LOCO_OK;
    const int64_t n = out_features, k = in_features;
    const int64_t need = mm_workspace(forward_product(x, weight, rows, n, k), ckpt != nullptr);
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    st = check_bufs({{x, rows * k * 2, false, true},
                     {weight, n * k * 2, false, true},
                     {bias, n * 2, false, false},
                     {residual, rows * n * 2, false, false},
                     {out, rows * n * dtype_size(out_dtype), true, true},
                     codes_buf(ckpt, rows, n, true),
                     exps_buf(ckpt, rows, n, true),
                     {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    MmParams p = forward_product(x, weight, rows, n, k);
    p.ep.bias = bias;
    p.ep.ckpt = ckpt_dev(ckpt, n);
    p.ep.act = act;
    p.ep.residual = residual;
    p.ep.out = out;
    p.ep.out_f32 = out_dtype == LOCO_F32;
    p.workspace = workspace;
    return hip_status(launch_mm(p, (hipStream_t)stream));
}

LOCO_API int64_t loco_linear_input_grad_workspace(int64_t rows, int64_t out_features, int64_t in_features) {
    if (check_product(rows, out_features, in_features) != LOCO_OK) return 0;
    return mm_workspace(input_grad_product(nullptr, nullptr, rows, out_features, in_features), false);
}

LOCO_API int loco_linear_input_grad(const uint16_t* dy, const uint16_t* weight, const uint16_t* residual, int64_t rows,
                                    int64_t out_features, int64_t in_features, loco_act_t act,
                                    const loco_checkpoint_t* ckpt, void* dx, loco_dtype_t out_dtype, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (!act_ok(act) || !dtype_ok(out_dtype) || (!ckpt && act != LOCO_ACT_NONE)) return LOCO_ERR_INVALID;
    int st = ckpt ? check_ckpt(*ckpt) : LOCO_OK;
    if (st != LOCO_OK) return st;
    st = check_product(rows, out_features, in_features);
    if (st != LOCO_OK) return st;
    if (rows == 0 || in_features == 0) return LOCO_OK;
    const int64_t n = in_features, k = out_features, need = loco_linear_input_grad_workspace(rows, k, n);
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    st = check_bufs({{dy, rows * k * 2, false, true},
                     {weight, n * k * 2, false, true},
                     {residual, rows * n * 2, false, false},
                     {dx, rows * n * dtype_size(out_dtype), true, true},
                     codes_buf(ckpt, rows, n, false),
                     exps_buf(ckpt, rows, n, false),
                     {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    MmParams p = input_grad_product(dy, weight, rows, k, n);
    if (act != LOCO_ACT_NONE) p.ep.slope = ckpt_dev(ckpt, n);
    p.ep.act = act;
    p.ep.residual = residual;
    p.ep.out = dx;
    p.ep.out_f32 = out_dtype == LOCO_F32;
    p.workspace = workspace;
    return hip_status(launch_mm(p, (hipStream_t)stream));
}

LOCO_API int64_t loco_linear_weight_grad_workspace(int64_t rows, int64_t out_features, int64_t in_features,
                                                   loco_act_t act) {
    if (check_product(rows, out_features, in_features) != LOCO_OK || !act_ok(act)) return 0;
    return weight_grad_space(rows, out_features, in_features).bytes();
}

LOCO_API int loco_linear_weight_grad(const uint16_t* dy, const loco_checkpoint_t* ckpt, int64_t rows,
                                     int64_t out_features, int64_t in_features, loco_act_t act, int accumulate,
                                     void* dweight, void* dbias, loco_dtype_t grad_dtype, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
    if (!ckpt || !act_ok(act) || !dtype_ok(grad_dtype)) return LOCO_ERR_INVALID;
    int st = check_ckpt(*ckpt);
    if (st != LOCO_OK) return st;
    st = check_product(rows, out_features, in_features);
    if (st != LOCO_OK) return st;
    if (out_features == 0) return LOCO_OK;
    const int64_t n = out_features, k = in_features, gs = dtype_size(grad_dtype);
    const WeightGradSpace space = weight_grad_space(rows, n, k);
    const int64_t need = space.bytes();
    if (workspace_bytes < need) return LOCO_ERR_INVALID;
    st = check_bufs({{dy, rows * n * 2, false, true},
                     codes_buf(ckpt, rows, k, false),
                     exps_buf(ckpt, rows, k, false),
                     {dweight, n * k * gs, true, true},
                     {dbias, n * gs, true, false},
                     {workspace, need, true, true}});
    if (st != LOCO_OK) return st;
    const hipStream_t hs = (hipStream_t)stream;
    char* at = (char*)workspace;
    if (k > 0) {
        uint16_t* a = (uint16_t*)(at + space.product + space.sums);
        // The matrix cores take bf16.  A checkpoint's values and their ReLU are bf16 numbers; GELU and
        // SiLU are not.  For bf16 gradients they are rounded to it, as the forward product's operand
        // was: an error of 0.0017 beside the gradient's own rounding of 0.0017.  For fp32 gradients
        // that would be all of the error, so what the rounding leaves (at most 2^-8 of the value,
        // itself rounded by 2^-8 of that) is a second operand, whose product is added to the first's.
        const int parts = grad_dtype == LOCO_F32 && (act == LOCO_ACT_GELU || act == LOCO_ACT_SILU) && rows > 0 ? 2 : 1;
        for (int part = 0; part < parts; ++part) {
            if (rows > 0 &&
                launch_ckpt_read(ckpt_dev(ckpt, k), rows, k, act, a, mm_padded(k), false, part == 1, hs) != hipSuccess)
                return LOCO_ERR_HIP;
            MmParams p = weight_grad_product(dy, a, rows, n, k);
            p.ep.out = dweight;
            p.ep.out_f32 = grad_dtype == LOCO_F32;
            p.ep.accumulate = accumulate != 0 || part == 1;
            p.workspace = at;
            if (launch_mm(p, hs) != hipSuccess) return LOCO_ERR_HIP;
        }
    }
    if (dbias)
        return hip_status(launch_col_sum(dy, rows, n, (float*)(at + space.product), dbias, grad_dtype == LOCO_F32,
                                         accumulate != 0, hs));
    return LOCO_OK;
}
