// Argument checks shared by the C ABI's entry points.
#pragma once

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

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool bits_ok(int bits) { return bits == 2 || bits == 4 || bits == 8; }
inline bool block_ok(int block) { return block == 64 || block == 128 || block == 256 || block == 512; }
inline bool dtype_ok(int d) { return d == LOCO_F32 || d == LOCO_BF16; }
inline int dtype_size(int d) { return d == LOCO_I8 ? 1 : (d == LOCO_BF16 ? 2 : 4); }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
inline bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// True if some written range overlaps any other range (written or read); read-only
// ranges may overlap each other.  Empty ranges never overlap.  Sorted by start, a range
// overlaps an earlier one exactly when it starts before the largest end seen so far.
struct Span {
    Range r;
    bool written;
};
inline bool any_write_overlap(std::vector<Span>& v) {
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

inline int64_t code_bytes(int64_t n, int bits) { return (n * bits + 7) / 8; }
inline int64_t nblocks(int64_t n, int block) { return (n + block - 1) / block; }

// Sizes beyond this are refused: far above any device memory, and safe from overflow in
// the byte arithmetic above.
constexpr int64_t kMaxElems = (int64_t)1 << 52;

inline bool act_ok(int a) { return a >= LOCO_ACT_NONE && a <= LOCO_ACT_SILU; }
inline int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// One buffer of a call.  `needed`: a null pointer is an error (of an empty buffer it is not).  align: what its
// address is a multiple of.
struct Buf {
    const void* p;
    int64_t bytes;
    bool written, needed;
    unsigned align = 16;
};

inline int check_bufs(std::initializer_list<Buf> bufs) {
    for (const Buf& b : bufs)
        if (b.needed && b.bytes > 0 && !b.p) return LOCO_ERR_INVALID;
    for (const Buf& b : bufs)
        if (b.p && b.bytes > 0 && ((uintptr_t)b.p & (b.align - 1))) return LOCO_ERR_ALIGN;
    // no buffer that is written may overlap another buffer of the call
    for (const Buf& a : bufs)
        for (const Buf& b : bufs) {
            if (&a == &b || !a.written || !a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) continue;
            if (overlap(range_of(a.p, a.bytes), range_of(b.p, b.bytes))) return LOCO_ERR_INVALID;
        }
    return LOCO_OK;
}

// Rows and columns whose product, in bytes, fits far inside 64 bits.
inline bool sizes_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && rows <= ((int64_t)1 << 40) && cols <= ((int64_t)1 << 40) &&
           (cols == 0 || rows <= ((int64_t)1 << 52) / cols);
}

inline int check_ckpt(const loco_checkpoint_t& c) {
    if (c.block < 1) return LOCO_ERR_INVALID;
    return c.block == 32 || c.block == 64 ? LOCO_OK : LOCO_ERR_UNSUPPORTED;
}
inline CkptDev ckpt_dev(const loco_checkpoint_t* c, int64_t cols) {
    if (!c) return {nullptr, nullptr, 0, 0};
    return {c->codes, c->exps, c->block == 64, nblocks(cols, c->block)};
}
inline Buf codes_buf(const loco_checkpoint_t* c, int64_t rows, int64_t cols, bool written) {
    return {c ? c->codes : nullptr, c ? rows * cols : 0, written, true};
}
inline Buf exps_buf(const loco_checkpoint_t* c, int64_t rows, int64_t cols, bool written) {
    return {c ? c->exps : nullptr, c ? rows * nblocks(cols, c->block) : 0, written, true};
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? LOCO_OK : LOCO_ERR_HIP; }

}  // namespace loco
