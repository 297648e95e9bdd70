// Matrix products of a linear layer: forward, input gradient and weight gradient, with their
// epilogues, on the bf16 matrix cores.
//
// C[m, n] = sum over k of A B.  The three products differ in which way their operands lie:
// "k-major" operands ([m, k] or [n, k]) hold eight consecutive k of one row in 16 bytes, as
// a matrix instruction takes them; "free-major" operands ([k, m] or [k, n]) hold eight
// consecutive rows' worth of one k and are transposed on their way from LDS to registers
// by ds_read_b64_tr_b16.
//   linear              x [T, K] k-major,      W [N, K] k-major
//   linear_input_grad   dy [T, N] k-major,     W [N, K] free-major
//   linear_weight_grad  dy [T, N] free-major,  checkpoint [T, K] free-major, decoded
//
// A workgroup computes a BM x BN tile in steps of 64 k.  Both operands' tiles go through LDS
// in two buffers: the next step's loads are in flight while this step's tiles are
// multiplied, with one barrier per step.  All sums are fp32 in the accumulators.

#include "loco_layer.hpp"
#include "loco_layer_internal.hpp"

namespace loco {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kStep = 64;  // k per step

// ---- LDS tiles ------------------------------------------------------------------------
//
// A tile of W rows or columns and STEP k is a sequence of 16-byte chunks, written in order
// q = 0, 1, ... by consecutive lanes.  k-major: row r holds STEP/8 chunks; free-major: row k
// holds W/8 chunks.  The chunk at position c of row r is the operand's chunk c ^ swz(r).  LDS
// has 64 banks of 4 bytes, 16 chunks across.  k-major: sixteen lanes read one k of sixteen
// rows, 16 / (STEP/8) rows of which lie in different banks anyway; the swizzle tells the
// others apart.  free-major: a read takes 64 bytes from each of four rows, which the swizzle
// spreads over all banks.
template <bool KMAJOR, int W, int STEP>
struct Tile {
    static constexpr int kChunks = W * STEP / 8;
    static constexpr int kPerRow = KMAJOR ? STEP / 8 : W / 8;
    static __device__ __forceinline__ int swz(int row) {
        return KMAJOR ? row / (16 / kPerRow) & (kPerRow - 1) : (row & 3) * 4;
    }
    static __device__ __forceinline__ int row_of(int q) { return q / kPerRow; }
    static __device__ __forceinline__ int chunk_of(int q) { return (q % kPerRow) ^ swz(row_of(q)); }
};

// Fragment of a 32 x 16 (free x k) operand block: lane l holds free index l % 32 and the
// eight k from 8 * (l / 32).
template <bool KMAJOR, int W, int STEP>
__device__ __forceinline__ bf16x8 read_frag(const u32x4* tile, int free0, int k0, int lane) {
    using T = Tile<KMAJOR, W, STEP>;
    if constexpr (KMAJOR) {
        const int r = free0 + (lane & 31), c = k0 / 8 + (lane >> 5);
        return __builtin_bit_cast(bf16x8, tile[r * T::kPerRow + (c ^ T::swz(r))]);
    } else {
        // Each group of 16 lanes takes 4 rows (k) of 16 columns: lane i of the group reads
        // columns 4 (i % 4) .. of row i / 4 and receives column i of the four rows.
        union {
            s16x4 h[2];
            bf16x8 v;
        } f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + (lane >> 5) * 8 + h * 4 + ((lane & 15) >> 2);
            const int col = free0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
            const int q = k * T::kPerRow + ((col >> 3) ^ T::swz(k));
            const char* p = (const char*)(tile + q) + (col & 4) * 2;
            f.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        }
        return f.v;
    }
}

// ---- staging ------------------------------------------------------------------------

// An operand: [free, k] (k-major) or [k, free], row-major with `ld` elements per row.
struct Operand {
    const uint16_t* p;
    const int8_t* codes;
    const uint8_t* exps;
    int64_t free, k, ld, nblocks;
    int block_shift, act;
};

// The eight elements at (row, col) of a rows x cols matrix; 0 outside.
__device__ __forceinline__ u32x4 load_bf16(const Operand& o, int64_t row, int64_t col, int64_t rows, int64_t cols) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (row < rows && col < cols) {
        const uint16_t* p = o.p + row * o.ld + col;
        if (cols - col >= 8) {
            w = load16(p);
        } else {
            const int n = (int)(cols - col);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        }
    }
    return w;
}

// Raw form of a staged chunk: bf16 elements, or codes with their byte.
template <bool CODES>
struct Raw;
template <>
struct Raw<false> {
    u32x4 w;
    __device__ __forceinline__ void load(const Operand& o, int64_t row, int64_t col, int64_t rows, int64_t cols) {
        w = load_bf16(o, row, col, rows, cols);
    }
    __device__ __forceinline__ u32x4 value(const Operand&) const { return w; }
};
template <>
struct Raw<true> {
    u32x2 w;
    uint32_t e;
    __device__ __forceinline__ void load(const Operand& o, int64_t row, int64_t col, int64_t rows, int64_t cols) {
        w = u32x2{0u, 0u};
        e = 0;
        if (row < rows && col < cols) {
            const int64_t left = cols - col;
            w = load_codes(o.codes + row * o.ld + col, left < 8 ? (int)left : 8);
            e = o.exps[row * o.nblocks + (col >> o.block_shift)];
        }
    }
    // bf16 holds a code's value exactly; an activation's value is rounded to the nearest bf16,
    // as the forward pass's product had it.
    __device__ __forceinline__ u32x4 value(const Operand& o) const {
        float v[8];
        decode_codes(w, e, v);
        act_chunk_any(o.act, v);
        return pack_bf16x8(v);
    }
};

template <bool KMAJOR, int W, int THREADS, bool CODES>
struct Stage {
    using T = Tile<KMAJOR, W, kStep>;
    static constexpr int kPer = T::kChunks / THREADS;
    Raw<CODES> raw[kPer];
    __device__ __forceinline__ void load(const Operand& o, int64_t free0, int64_t k0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int q = j * THREADS + threadIdx.x, r = T::row_of(q), c = T::chunk_of(q) * 8;
            if constexpr (KMAJOR) raw[j].load(o, free0 + r, k0 + c, o.free, o.k);
            else raw[j].load(o, k0 + r, free0 + c, o.k, o.free);
        }
    }
    __device__ __forceinline__ void store(const Operand& o, u32x4* tile) const {
#pragma unroll
        for (int j = 0; j < kPer; ++j) tile[j * THREADS + threadIdx.x] = raw[j].value(o);
    }
};

// ---- epilogue -------------------------------------------------------------------------

// Eight consecutive sums of one row on their way out.  All 64 lanes take part; `valid`
// elements of the chunk exist (none if <= 0).
__device__ __forceinline__ void epilogue(const MmEpilogue& e, int64_t row, int64_t n, int64_t col, int valid,
                                         float (&v)[8]) {
    const int64_t at = row * n + col;
    float t[8];
    if (e.bias) {
        load_chunk(e.bias + col, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    if (e.ckpt.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = i < valid ? v[i] : 0.0f;
        const uint32_t x = ckpt_exp(block_top(t, e.ckpt.block64));
        store_codes(e.ckpt.codes + at, valid, ckpt_codes(t, x));
        const int shift = e.ckpt.block64 ? 6 : 5;
        if ((col & ((1 << shift) - 1)) == 0 && valid > 0)
            e.ckpt.exps[row * e.ckpt.nblocks + (col >> shift)] = (uint8_t)x;
    }
    if (valid <= 0) return;
    if (e.slope.codes) {
        decode_codes(load_codes(e.slope.codes + at, valid),
                     e.slope.exps[row * e.slope.nblocks + (col >> (e.slope.block64 ? 6 : 5))], t);
        slope_chunk_any(e.act, t, v);
    } else {
        act_chunk_any(e.act, v);
    }
    if (e.residual) {
        load_chunk(e.residual + at, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    if (e.accumulate) {
        load_chunk_any(e.out, e.out_f32, at, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    store_chunk_any(e.out, e.out_f32, at, valid, v);
}

// ---- the tile kernel --------------------------------------------------------------------

struct MmArgs {
    Operand a, b;
    int64_t m, n, k;
    int tiles_m, tiles_n;
    int64_t k_split;  // k per split, a multiple of kStep
    float* part;      // null: epilogue
    MmEpilogue ep;
};

// Which tile a workgroup takes.  Workgroups go round-robin over the 8 XCDs; each XCD takes a
// contiguous run of the tile order, which walks columns of 8 tile rows, so that the tiles at
// work on one XCD share operand rows in its L2.
__device__ __forceinline__ void tile_of(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int total = tiles_m * tiles_n;
    const int x = b % kXcds, each = total / kXcds, more = total % kXcds;
    const int id = x * each + min(x, more) + b / kXcds;
    constexpr int GROUP = 8;
    const int width = GROUP * tiles_n;
    const int first = id / width * GROUP, rows = min(tiles_m - first, GROUP);
    tm = first + id % width % rows;
    tn = id % width / rows;
}

// A wave's accumulators to rows: register r of a 32 x 32 block is row 8 (r / 4) + 4 (lane / 32) +
// r % 4, column lane % 32.  32 rows of 64 columns at a time turn through the wave's own
// stretch of LDS, after which eight lanes hold one row's 64 columns: stores, the residual's
// loads and a checkpoint's blocks all take whole chunks.
constexpr int kRowPad = 68;  // floats from row to row: the eight rows of one read start in different banks
template <int MI, int NI>
__device__ __forceinline__ void store_acc(const MmArgs& g, const f32x16 (&acc)[MI][NI], float* mine, int64_t m0,
                                          int64_t n0, int lane) {
    // One copy of the epilogue's code: the loop over the 32 x 64 parts is a real one, and each
    // part's registers are picked by a uniform branch.
#pragma unroll 1
    for (int part = 0; part < MI * NI / 2; ++part) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int h = 0; h < NI / 2; ++h)
                if (part == i * (NI / 2) + h) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            mine[(8 * (r / 4) + 4 * (lane >> 5) + r % 4) * kRowPad + j * 32 + (lane & 31)] =
                                acc[i][2 * h + j][r];
                }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int64_t row0 = m0 + part / (NI / 2) * 32, col0 = n0 + part % (NI / 2) * 64;
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int r = pass * 8 + (lane >> 3), c = (lane & 7) * 8;
            const int64_t row = row0 + r, col = col0 + c;
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = mine[r * kRowPad + c + x];
            const int64_t left = g.n - col;
            const int valid = row >= g.m || left <= 0 ? 0 : left < 8 ? (int)left : 8;
            if (g.part) store_chunk(g.part + ((int64_t)blockIdx.y * g.m + row) * g.n + col, valid, v);
            else epilogue(g.ep, row, g.n, col, valid, v);
        }
    }
}

template <int BM, int BN, int WM, int WN, bool AK, bool BK, bool CODES>
__global__ __launch_bounds__(WM * WN * 64, 2) void mm_kernel(const MmArgs g) {
    constexpr int THREADS = WM * WN * 64;
    constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 32, NI = TN / 32;
    constexpr int ACH = Tile<AK, BM, kStep>::kChunks, BCH = Tile<BK, BN, kStep>::kChunks;
    constexpr int EPI = WM * WN * 32 * kRowPad / 4;  // chunks of the epilogue's staging
    __shared__ u32x4 lds[2 * (ACH + BCH) > EPI ? 2 * (ACH + BCH) : EPI];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int64_t k_lo = (int64_t)blockIdx.y * g.k_split;
    const int64_t k_hi = min(g.k, k_lo + g.k_split);
    const int steps = (int)((k_hi - k_lo + kStep - 1) / kStep);

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};

    Stage<AK, BM, THREADS, false> sa;
    Stage<BK, BN, THREADS, CODES> sb;
    if (steps > 0) {
        sa.load(g.a, m0, k_lo);
        sb.load(g.b, n0, k_lo);
        sa.store(g.a, lds);
        sb.store(g.b, lds + ACH);
    }
    __syncthreads();
    for (int it = 0; it < steps; ++it) {
        const u32x4* ta = lds + (it & 1) * (ACH + BCH);
        const u32x4* tb = ta + ACH;
        const bool more = it + 1 < steps;
        if (more) {
            sa.load(g.a, m0, k_lo + (int64_t)(it + 1) * kStep);
            sb.load(g.b, n0, k_lo + (int64_t)(it + 1) * kStep);
        }
#pragma unroll
        for (int s = 0; s < kStep / 16; ++s) {
            bf16x8 fa[MI], fb[NI];
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i] = read_frag<AK, BM, kStep>(ta, wm * TM + i * 32, s * 16, lane);
#pragma unroll
            for (int j = 0; j < NI; ++j) fb[j] = read_frag<BK, BN, kStep>(tb, wn * TN + j * 32, s * 16, lane);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
        if (more) {
            u32x4* next = lds + ((it + 1) & 1) * (ACH + BCH);
            sa.store(g.a, next);
            sb.store(g.b, next + ACH);
        }
        __syncthreads();
    }

    store_acc<MI, NI>(g, acc, (float*)lds + wave * 32 * kRowPad, m0 + wm * TM, n0 + wn * TN, lane);
}

// ---- the tile kernel, staged past the registers --------------------------------------------
//
// The same tiles with loads that go from memory to LDS directly, 16 bytes a lane.  They need
// rows of whole 16-byte chunks.  A load past the end of the operand writes zeros, which is what
// the last rows, and the last k of a free-major operand, need; the last k of a k-major
// operand, where the next row follows, is sent past the end by its lanes.

struct DmaSrc {
    const char* base;
    int64_t left;  // bytes from base to the operand's end
    int64_t step;  // bytes from one step to the next
};

template <bool KMAJOR, int W, int STEP, int THREADS>
struct Dma {
    using T = Tile<KMAJOR, W, STEP>;
    static constexpr int kPer = T::kChunks / THREADS;
    static constexpr uint32_t kOut = 0x80000000u;  // past any operand: offsets stay below 2^31
    DmaSrc s;
    uint32_t off[kPer];
    int k_chunk;  // k-major: this thread's chunk within a row, the same for each of its loads

    __device__ __forceinline__ void init(const Operand& o, int64_t free0, int64_t k0) {
        static_assert(THREADS % T::kPerRow == 0 && (THREADS / T::kPerRow) % 16 == 0 || !KMAJOR,
                      "a thread's loads share their chunk's place in the row");
        static_assert(THREADS / T::kPerRow % 4 == 0 || KMAJOR, "a thread's loads share their swizzle");
        const int t = threadIdx.x;
        s.base = (const char*)(o.p + (KMAJOR ? free0 * o.ld + k0 : k0 * o.ld + free0));
        s.left = ((KMAJOR ? o.free : o.k) * o.ld) * 2 - (s.base - (const char*)o.p);
        s.step = (KMAJOR ? STEP : STEP * o.ld) * 2;
        k_chunk = T::chunk_of(t);
        const uint32_t per = (uint32_t)(THREADS / T::kPerRow * o.ld * 2);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            off[j] = (uint32_t)(T::row_of(t) * o.ld * 2) + T::chunk_of(t) * 16 + j * per;
    }
    // One of the next step's loads; `k_left` is the k that are left from the step on.  The
    // instruction takes its LDS address from m0 and each lane's 16 bytes follow the last one's.
    // It writes no register, so inline assembly leaves the compiler nothing to track; with the
    // builtin, the compiler would wait for every load ahead of each transposing LDS read, not
    // knowing that they touch different stages.  step_barrier() waits for it.
    __device__ __forceinline__ void issue(uint32_t tile, int j, int k_left) {
        const int64_t bytes = max((int64_t)0, min(s.left, (int64_t)0x7fffffff));
        const uint64_t base = (uint64_t)s.base;
        const u32x4 r = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, (uint32_t)bytes, 0x00020000u};
        const uint32_t to = tile + (uint32_t)(j * THREADS + uniform(threadIdx.x & ~63)) * 16;
        const uint32_t o = KMAJOR && k_left < STEP && k_chunk * 8 >= k_left ? kOut : off[j];
        // the wait states cover scalar registers that a vector instruction has just written
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(to), "v"(o), "s"(r)
                     : "memory", "m0");
    }
    __device__ __forceinline__ void advance() {
        s.base += s.step;
        s.left -= s.step;
    }
};

// Waits until at most `pending` of this wave's loads are on their way and its LDS reads have
// returned, and for the other waves to get there.
template <int PENDING>
__device__ __forceinline__ void step_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((PENDING & 15) | (PENDING >> 4 << 14) | 7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// LDS holds STAGES steps: while one is multiplied, the loads of the next STAGES - 1 are on
// their way.  Within a step the fragments of the next 16 k are read while the matrix cores
// work on the present ones.  The barrier between steps comes before the last 16 k of a step,
// whose fragments are in registers by then: behind it the next step's first fragments are
// read, the loads into the step just read out start, and the matrix cores are busy meanwhile.
// Loads past the last step are started all the same (and write zeros, or k that are not
// multiplied), so that the count of pending loads is the same in every step.
template <int BM, int BN, int WM, int WN, int STEP, int STAGES, bool AK, bool BK>
__global__ __launch_bounds__(WM * WN * 64, WM * WN == 4 && BM == 256 ? 1 : 2) void mm_dma_kernel(const MmArgs g) {
    constexpr int THREADS = WM * WN * 64;
    constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 32, NI = TN / 32;
    using DA = Dma<AK, BM, STEP, THREADS>;
    using DB = Dma<BK, BN, STEP, THREADS>;
    constexpr int ACH = DA::T::kChunks, BCH = DB::T::kChunks, SUB = STEP / 16;
    static_assert(STAGES * (ACH + BCH) * 16 >= WM * WN * 32 * kRowPad * 4, "the epilogue's rows fit the tiles' LDS");
    __shared__ u32x4 lds[STAGES * (ACH + BCH)];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int64_t k_lo = (int64_t)blockIdx.y * g.k_split;
    const int k_all = (int)(min(g.k, k_lo + g.k_split) - k_lo);
    const int steps = (k_all + STEP - 1) / STEP;

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};

    DA da;
    DB db;
    bf16x8 fa[2][MI], fb[2][NI];
    da.init(g.a, m0, k_lo);
    db.init(g.b, n0, k_lo);
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    int k_left = k_all;
    constexpr int LOADS = DA::kPer + DB::kPer;
    // load j of the step that comes next in the order of loading
    auto issue = [&](int stage, int j) {
        const uint32_t t = lds_at + stage * (ACH + BCH) * 16;
        if (j < DA::kPer) da.issue(t, j, k_left);
        else db.issue(t + ACH * 16, j - DA::kPer, k_left);
        if (j == LOADS - 1) {
            da.advance();
            db.advance();
            k_left -= STEP;
        }
    };
    // fragment f of 16 k of a step, in the order in which the products take them
    auto read = [&](int stage, int s, int f) {
        const u32x4* t = lds + stage * (ACH + BCH);
        const int slot = s & 1;
        if (f >= 1 && f <= NI)
            fb[slot][f - 1] = read_frag<BK, BN, STEP>(t + ACH, wn * TN + (f - 1) * 32, s * 16, lane);
        else {
            const int i = f == 0 ? 0 : f - NI;
            fa[slot][i] = read_frag<AK, BM, STEP>(t, wm * TM + i * 32, s * 16, lane);
        }
    };
    constexpr int PENDING = (STAGES - 2) * LOADS;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
        for (int j = 0; j < LOADS; ++j) issue(i, j);
    step_barrier<PENDING>();
#pragma unroll
    for (int f = 0; f < MI + NI; ++f) read(0, 0, f);
#pragma unroll
    for (int j = 0; j < LOADS / 2; ++j) issue(STAGES - 1, j);
    for (int it = 0; it < steps; it += STAGES) {
#pragma unroll
        for (int stage = 0; stage < STAGES; ++stage) {
            if (it + stage >= steps) break;
            constexpr int MF = MI * NI;
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const bool last = s + 1 == SUB;
                if (last) step_barrier<PENDING>();
                // Between two products: the reads of the next 16 k, and behind the barrier and in
                // the next step's first 16 k half of a step's loads each.  The matrix cores are busy
                // for 32 cycles with each product, which hides what issues in between.
#pragma unroll
                for (int x = 0; x < MF; ++x) {
                    acc[x / NI][x % NI] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        fa[s & 1][x / NI], fb[s & 1][x % NI], acc[x / NI][x % NI], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int f = x * (MI + NI) / MF; f < (x + 1) * (MI + NI) / MF; ++f) {
                        if (last) read(stage + 1 == STAGES ? 0 : stage + 1, 0, f);
                        else read(stage, s + 1, f);
                    }
                    if (last || s == 0) {
#pragma unroll
                        for (int j = x * (LOADS / 2) / MF; j < (x + 1) * (LOADS / 2) / MF; ++j)
                            issue(last ? stage : stage == 0 ? STAGES - 1 : stage - 1, last ? j : LOADS / 2 + j);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
    step_barrier<0>();  // the epilogue takes over the LDS that the last loads were written to
    store_acc<MI, NI>(g, acc, (float*)lds + wave * 32 * kRowPad, m0 + wm * TM, n0 + wn * TN, lane);
}

// The splits' partial sums, joined in order, and the epilogue: rows are padded to 64 columns
// so that a checkpoint's blocks stay within eight lanes.
__global__ __launch_bounds__(256) void mm_join_kernel(const MmArgs g, int splits, int64_t per_row, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = t / per_row, col = (t - row * per_row) * 8, left = g.n - col;
    const int valid = row >= g.m || left <= 0 ? 0 : left < 8 ? (int)left : 8;
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int s = 0; s < splits; ++s) {
        load_chunk(g.part + ((int64_t)s * g.m + row) * g.n + col, valid, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    epilogue(g.ep, row, g.n, col, valid, v);
}

#ifndef MM_CFG
#define MM_BM 256
#define MM_BN 256
#define MM_CFG 256, 256, 2, 4, 64, 2
#define MM_THREADS 512
#endif
const void* pick_dma(bool ak, bool bk) {
    if (ak && bk) return (const void*)&mm_dma_kernel<MM_CFG, true, true>;
    if (ak) return (const void*)&mm_dma_kernel<MM_CFG, true, false>;
    return (const void*)&mm_dma_kernel<MM_CFG, false, false>;
}
const void* pick_mm(bool ak, bool bk, bool codes) {
    if (codes) return (const void*)&mm_kernel<128, 128, 2, 2, false, false, true>;
    if (bk) return (const void*)&mm_kernel<128, 128, 2, 2, true, true, false>;
    return (const void*)&mm_kernel<128, 128, 2, 2, true, false, false>;
}

constexpr int kTile = 128;
int64_t tiles_of(int64_t n, int64_t tile = kTile) { return (n + tile - 1) / tile; }

}  // namespace

// Few tiles leave compute units idle: the contraction is split until the workgroups fill
// the chip, with at least 512 k per split.
int mm_splits(int64_t m, int64_t n, int64_t k) {
    const int64_t tiles = tiles_of(m) * tiles_of(n);
    if (tiles <= 0) return 1;
    const int64_t most = k / 512, wanted = 256 / tiles;
    const int64_t s = wanted < most ? wanted : most;
    return s < 2 ? 1 : s > 64 ? 64 : (int)s;
}

hipError_t launch_mm(const MmParams& p, hipStream_t stream) {
    MmArgs g;
    g.a = {p.a, nullptr, nullptr, p.m, p.k, p.a_kmajor ? p.k : p.m, 0, 0, 0};
    g.b = {p.b, p.bq.codes, p.bq.exps, p.n, p.k, p.b_kmajor ? p.k : p.n, p.bq.nblocks, p.bq.block64 ? 6 : 5, p.bq_act};
    g.m = p.m;
    g.n = p.n;
    g.k = p.k;
    const bool dma = !p.b_codes && (p.a_kmajor ? p.k : p.m) % 8 == 0 && (p.b_kmajor ? p.k : p.n) % 8 == 0;
    g.tiles_m = (int)tiles_of(p.m, dma ? MM_BM : kTile);
    g.tiles_n = (int)tiles_of(p.n, dma ? MM_BN : kTile);
    const int64_t steps = (p.k + kStep - 1) / kStep;
    g.k_split = (steps + p.splits - 1) / p.splits * kStep;
    g.part = p.splits > 1 ? p.part : nullptr;
    g.ep = p.ep;
    const void* k = dma ? pick_dma(p.a_kmajor, p.b_kmajor) : pick_mm(p.a_kmajor, p.b_kmajor, p.b_codes != 0);
    void* args[] = {(void*)&g};
    const int64_t tiles = (int64_t)g.tiles_m * g.tiles_n;
    hipError_t err = hipLaunchKernel(k, dim3((unsigned)tiles, (unsigned)p.splits), dim3(dma ? MM_THREADS : 256), args, 0, stream);
    if (err != hipSuccess || p.splits == 1) return err;
    int64_t per_row = (p.n + 63) / 64 * 8, t0 = 0;
    int splits = p.splits;
    const int64_t chunks = p.m * per_row;
    void* jargs[] = {(void*)&g, (void*)&splits, (void*)&per_row, (void*)&t0};
    for (; t0 < chunks; t0 += kMaxGrid * 256) {
        const int64_t left = chunks - t0;
        const int64_t blocks = left < kMaxGrid * 256 ? (left + 255) / 256 : kMaxGrid;
        err = hipLaunchKernel((const void*)&mm_join_kernel, dim3((unsigned)blocks), dim3(256), jargs, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

bool mm_decodes(int64_t m, int64_t n) { return m % 8 == 0 && n % 8 == 0; }

// ---- column sums ------------------------------------------------------------------------

namespace {

// Partial sums of 512 columns per workgroup over every gridDim.y-th group of four rows, one
// row per wave.
__global__ __launch_bounds__(256) void col_sum_kernel(const uint16_t* x, int64_t rows, int64_t n, float* part) {
    __shared__ float join[4][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 512 + lane * 8, left = n - col;
    const int valid = left <= 0 ? 0 : left < 8 ? (int)left : 8;
    float s[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.y * 4 + wave; r < rows; r += (int64_t)gridDim.y * 4) {
        load_chunk(x + r * n + col, valid, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) join[wave][lane * 8 + i] = s[i];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
        const int64_t at = (int64_t)blockIdx.x * 512 + c;
        if (at < n) part[blockIdx.y * n + at] = (join[0][c] + join[1][c]) + (join[2][c] + join[3][c]);
    }
}

__global__ __launch_bounds__(256) void col_join_kernel(const float* part, int64_t groups, int64_t n, void* out, int f32,
                                                       int accumulate) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float v = 0.0f;
#pragma unroll 8
    for (int64_t g = 0; g < groups; ++g) v += part[g * n + c];
    if (f32) ((float*)out)[c] = accumulate ? v + ((float*)out)[c] : v;
    else {
        uint16_t* o = (uint16_t*)out + c;
        *o = bf16_rne(accumulate ? v + __uint_as_float((uint32_t)*o << 16) : v);
    }
}

}  // namespace

int64_t col_sum_groups(int64_t rows, int64_t n) {
    const int64_t blocks = (n + 511) / 512, most = (rows + 15) / 16;
    int64_t g = 512 / blocks;
    g = g < 1 ? 1 : g > 64 ? 64 : g;
    return g < most ? g : most < 1 ? 1 : most;
}

hipError_t launch_col_sum(const uint16_t* x, int64_t rows, int64_t n, float* part, void* out, bool f32, bool accumulate,
                          hipStream_t stream) {
    int64_t groups = col_sum_groups(rows, n);
    void* args[] = {(void*)&x, (void*)&rows, (void*)&n, (void*)&part};
    hipError_t err = hipLaunchKernel((const void*)&col_sum_kernel, dim3((unsigned)((n + 511) / 512), (unsigned)groups),
                                     dim3(256), args, 0, stream);
    if (err != hipSuccess) return err;
    int f = f32, acc = accumulate;
    void* jargs[] = {(void*)&part, (void*)&groups, (void*)&n, (void*)&out, (void*)&f, (void*)&acc};
    return hipLaunchKernel((const void*)&col_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), jargs, 0, stream);
}

}  // namespace loco
