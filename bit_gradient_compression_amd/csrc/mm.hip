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
//   linear_weight_grad  dy [T, N] free-major,  decoded checkpoint [T, K] free-major
//
// A workgroup computes a BM x BN tile in steps of 64 k.  Both operands' tiles go through LDS,
// where the next step's loads land while this step's tiles are multiplied, with one barrier
// per step.  All sums are fp32 in the accumulators.
//
// In the large tile's launches the matrix cores are busy 52 - 59 % of the cycles (counters), at a
// clock of 1.9 - 2.1 of 2.4 GHz.  The rest is not theirs: each step's barrier and waits, the
// epilogue, which no next tile overlaps (registers and LDS hold one 256 x 256 tile per compute
// unit), and the last round of tiles.  The library's product of 8192^3, four full rounds, reaches
// 1592 TFLOP/s where this tile reaches 1349.  Measured, bare products of 8192 rows with 4096 and
// 11008 features: forward 608 us (1215 TFLOP/s), input gradient 604 (1223), weight gradient 578
// (1278, without its decoding and bias gradient).  Bias, GELU and a checkpoint on the way out add 43 - 51 us.
// With few rows the weights' bytes bind: 16 rows of 11008 -> 4096 take 18 us (5 TB/s) and the join 5.

#include "loco_layer.hpp"
#include "loco_layer_internal.hpp"

namespace loco {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kStep = 64;  // k per step

// N pieces of work f(0) ... f(N - 1) spread evenly over SLOTS places in the code; the pieces of
// place x.
template <int SLOTS, int N, typename F>
__device__ __forceinline__ void spread(int x, F f) {
    constexpr int every = SLOTS / N > 1 ? SLOTS / N : 1, at_once = (N + SLOTS - 1) / SLOTS;
    if (x % every == 0) {
#pragma unroll
        for (int c = 0; c < at_once; ++c)
            if (x / every * at_once + c < N) f(x / every * at_once + c);
    }
}

// ---- LDS tiles ------------------------------------------------------------------------
//
// A tile of W rows or columns and STEP k is a sequence of 16-byte chunks, written in order
// q = 0, 1, ... by consecutive lanes.  k-major: row r holds STEP/8 chunks; free-major: row k
// holds W/8 chunks.  The chunk at position c of row r is the operand's chunk c ^ swz(r).  LDS
// has 64 banks of 4 bytes, 16 chunks across.  k-major: sixteen lanes read one k of sixteen
// rows, 16 / (STEP/8) rows of which lie in different banks anyway; the swizzle tells the
// others apart.  free-major: a read takes stretches of four rows, eight rows
// apart for other lanes, which the swizzle spreads over all banks.
template <bool KMAJOR, int W, int STEP>
struct Tile {
    static constexpr int kChunks = W * STEP / 8;
    static constexpr int kPerRow = KMAJOR ? STEP / 8 : W / 8;
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (KMAJOR) return row / (16 / kPerRow) & (kPerRow - 1);
        // free-major: two chunks from each of four rows, and the same eight rows on
        else if constexpr (kPerRow >= 16) return (row & 3) * 4 ^ (row >> 2 & 2);
        else if constexpr (kPerRow == 8) return (row & 2) ^ (row >> 1 & 4);
        else return row >> 2 & 2;
    }
    static_assert(KMAJOR || kPerRow == 4 || kPerRow % 8 == 0, "rows that the swizzle stays inside of");
    static __device__ __forceinline__ int row_of(int q) { return q / kPerRow; }
    static __device__ __forceinline__ int chunk_of(int q) { return (q % kPerRow) ^ swz(row_of(q)); }
};

// The matrix instruction: MS x MS results from MS x KS and KS x MS operands.  Lane l holds
// free index l % MS of an operand and the eight k from 8 * (l / MS).
template <int MS>
struct Mfma;
template <>
struct Mfma<32> {
    static constexpr int KS = 16;
    typedef f32x16 acc_t;
    static __device__ __forceinline__ acc_t mul(bf16x8 a, bf16x8 b, acc_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // row of register r; the column is lane % 32
    static __device__ __forceinline__ int row(int r, int lane) { return 8 * (r / 4) + 4 * (lane >> 5) + r % 4; }
};
template <>
struct Mfma<16> {
    static constexpr int KS = 32;
    typedef f32x4 acc_t;
    static __device__ __forceinline__ acc_t mul(bf16x8 a, bf16x8 b, acc_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ int row(int r, int lane) { return 4 * (lane >> 4) + r; }
};

// An operand's fragment at (free0, k0) of a tile.
template <bool KMAJOR, int W, int STEP, int MS>
__device__ __forceinline__ bf16x8 read_frag(const u32x4* tile, int free0, int k0, int lane) {
    using T = Tile<KMAJOR, W, STEP>;
    if constexpr (KMAJOR) {
        const int r = free0 + (lane & (MS - 1)), c = k0 / 8 + lane / MS;
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
            const int k = k0 + lane / MS * 8 + h * 4 + ((lane & 15) >> 2);
            const int col = free0 + (lane & (MS - 1) & 16) + (lane & 3) * 4;
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
    int64_t free, k, ld;
};

// The eight elements at (row, col) of a rows x cols matrix; 0 outside.
__device__ __forceinline__ u32x4 load_bf16(const Operand& o, int64_t row, int64_t col, int64_t rows, int64_t cols) {
    RawChunk<uint16_t> c;
    const int64_t left = cols - col;
    c.load(o.p + row * o.ld + col, row < rows && left > 0 ? (left < 8 ? (int)left : 8) : 0);
    return c.w;
}

template <bool KMAJOR, int W, int THREADS>
struct Stage {
    using T = Tile<KMAJOR, W, kStep>;
    static constexpr int kPer = T::kChunks / THREADS;
    u32x4 raw[kPer];
    __device__ __forceinline__ void load(const Operand& o, int64_t free0, int64_t k0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int q = j * THREADS + threadIdx.x, r = T::row_of(q), c = T::chunk_of(q) * 8;
            raw[j] = KMAJOR ? load_bf16(o, free0 + r, k0 + c, o.free, o.k) : load_bf16(o, k0 + r, free0 + c, o.k, o.free);
        }
    }
    __device__ __forceinline__ void store(u32x4* tile) const {
#pragma unroll
        for (int j = 0; j < kPer; ++j) tile[j * THREADS + threadIdx.x] = raw[j];
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
    int64_t m_first, n_first;  // the first tile's row and column
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

// ---- from accumulators to rows -----------------------------------------------------------
//
// 32 rows of 64 columns (a part) at a time turn through the wave's own stretch of LDS, after
// which eight lanes hold one row's 64 columns, in four passes of eight rows: stores, the
// residual's loads and a checkpoint's blocks all take whole chunks.
constexpr int kRowPad = 68;  // floats from row to row: the eight rows of one read start in different banks
constexpr int kPasses = 2;  // of eight rows, worked together

// What the epilogue reads of a part, loaded ahead of its use.
struct PartLoads {
    u32x4 residual[kPasses];
    u32x2 codes[kPasses];
    uint32_t exps[kPasses];
    __device__ __forceinline__ void load(const MmEpilogue& e, int64_t n, int64_t row, int64_t col) {
        if (e.residual) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) residual[p] = load16(e.residual + (row + p * 8) * n + col);
        }
        if (e.slope.codes) {
            const int shift = e.slope.block64 ? 6 : 5;
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                __builtin_memcpy(&codes[p], e.slope.codes + (row + p * 8) * n + col, 8);
                exps[p] = e.slope.exps[(row + p * 8) * e.slope.nblocks + (col >> shift)];
            }
        }
    }
};

// The epilogue of rows that lie inside the matrix: epilogue() for whole chunks of several rows,
// without its tests of each chunk's end and with nothing that waits between the passes.
__device__ __forceinline__ void epilogue_part(const MmEpilogue& e, const PartLoads& in, int64_t n, int64_t row,
                                              int64_t col, float (&v)[kPasses][8]) {
    float t[8];
    if (e.bias) {
        unpack_bf16x8(load16(e.bias + col), t);
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] += t[i];
    }
    if (e.ckpt.codes) {
        const int shift = e.ckpt.block64 ? 6 : 5;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const uint32_t x = ckpt_exp(block_top(v[p], e.ckpt.block64));
            store_codes(e.ckpt.codes + (row + p * 8) * n + col, 8, ckpt_codes(v[p], x));
            if ((col & ((1 << shift) - 1)) == 0)
                e.ckpt.exps[(row + p * 8) * e.ckpt.nblocks + (col >> shift)] = (uint8_t)x;
        }
    }
    if (e.slope.codes) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            decode_codes(in.codes[p], in.exps[p], t);
            slope_chunk_any(e.act, t, v[p]);
        }
    } else if (e.act) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) act_chunk_any(e.act, v[p]);
    }
    if (e.residual) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            unpack_bf16x8(in.residual[p], t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] += t[i];
        }
    }
    if (e.accumulate) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            load_chunk_any(e.out, e.out_f32, (row + p * 8) * n + col, 8, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] += t[i];
        }
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) store_chunk_any(e.out, e.out_f32, (row + p * 8) * n + col, 8, v[p]);
}

template <int MS, int MI, int NI>
__device__ __forceinline__ void store_acc(const MmArgs& g, const typename Mfma<MS>::acc_t (&acc)[MI][NI], float* mine,
                                          int64_t m0, int64_t n0, int lane) {
    constexpr int PI = 32 / MS, PJ = 64 / MS;  // blocks of a part
    constexpr int ACROSS = NI / PJ, PARTS = MI / PI * ACROSS;
    const int rl = lane >> 3, cl = (lane & 7) * 8;
    // row and column of a part; uniform, and so is whether it lies inside
    auto row_of = [&](int part) __attribute__((always_inline)) { return m0 + part / ACROSS * 32; };
    auto col_of = [&](int part) __attribute__((always_inline)) { return n0 + part % ACROSS * 64; };
    auto inside = [&](int part) __attribute__((always_inline)) { return row_of(part) + 32 <= g.m && col_of(part) + 64 <= g.n; };
    // One copy of the epilogue's code: the loop over the parts is a real one, and each part's
    // registers are picked by a uniform branch.
#pragma unroll 1
    for (int part = 0; part < PARTS; ++part) {
        const int64_t row0 = row_of(part) + rl, col = col_of(part) + cl;
        PartLoads in;
        const bool whole = inside(part), ep = whole && !g.part;
        if (ep) in.load(g.ep, g.n, row0, col);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int x = 0; x < PARTS; ++x)
            if (part == x) {
#pragma unroll
                for (int i = 0; i < PI; ++i)
#pragma unroll
                    for (int j = 0; j < PJ; ++j)
#pragma unroll
                        for (int r = 0; r < MS * MS / 64; ++r)
                            mine[(i * MS + Mfma<MS>::row(r, lane)) * kRowPad + j * MS + (lane & (MS - 1))] =
                                acc[x / ACROSS * PI + i][x % ACROSS * PJ + j][r];
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (whole) {
#pragma unroll
            for (int q = 0; q < 4 / kPasses; ++q) {
                float v[kPasses][8];
                const int64_t row = row0 + q * kPasses * 8;
#pragma unroll
                for (int p = 0; p < kPasses; ++p)
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[p][x] = mine[((q * kPasses + p) * 8 + rl) * kRowPad + cl + x];
                if (g.part) {
                    float* out = g.part + ((int64_t)blockIdx.y * g.m + row) * g.n + col;
#pragma unroll
                    for (int p = 0; p < kPasses; ++p) store_chunk(out + p * 8 * g.n, 8, v[p]);
                } else {
                    epilogue_part(g.ep, in, g.n, row, col, v);
                    if (q + 1 < 4 / kPasses) in.load(g.ep, g.n, row + kPasses * 8, col);
                }
            }
            continue;
        }
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {
            const int64_t row = row0 + p * 8, left = g.n - col;
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = mine[(p * 8 + rl) * kRowPad + cl + x];
            const int valid = row >= g.m || left <= 0 ? 0 : left < 8 ? (int)left : 8;
            if (g.part) store_chunk(g.part + ((int64_t)blockIdx.y * g.m + row) * g.n + col, valid, v);
            else epilogue(g.ep, row, g.n, col, valid, v);
        }
    }
}

template <int BM, int BN, int WM, int WN, bool AK, bool BK>
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
    const int64_t m0 = g.m_first + (int64_t)tm * BM, n0 = g.n_first + (int64_t)tn * BN;
    const int64_t k_lo = (int64_t)blockIdx.y * g.k_split;
    const int64_t k_hi = min(g.k, k_lo + g.k_split);
    const int steps = (int)((k_hi - k_lo + kStep - 1) / kStep);

    f32x16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x16{};

    Stage<AK, BM, THREADS> sa;
    Stage<BK, BN, THREADS> sb;
    if (steps > 0) {
        sa.load(g.a, m0, k_lo);
        sb.load(g.b, n0, k_lo);
        sa.store(lds);
        sb.store(lds + ACH);
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
            for (int i = 0; i < MI; ++i) fa[i] = read_frag<AK, BM, kStep, 32>(ta, wm * TM + i * 32, s * 16, lane);
#pragma unroll
            for (int j = 0; j < NI; ++j) fb[j] = read_frag<BK, BN, kStep, 32>(tb, wn * TN + j * 32, s * 16, lane);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
        if (more) {
            u32x4* next = lds + ((it + 1) & 1) * (ACH + BCH);
            sa.store(next);
            sb.store(next + ACH);
        }
        __syncthreads();
    }

    store_acc<32, MI, NI>(g, acc, (float*)lds + wave * 32 * kRowPad, m0 + wm * TM, n0 + wn * TN, lane);
}

// ---- the tile kernel, staged past the registers --------------------------------------------
//
// The same tiles with loads that go from memory to LDS directly, 16 bytes a lane.  They need
// rows of whole 16-byte chunks.  A load past the end of the operand writes zeros, which is what
// the last rows, and the last k of a free-major operand, need; the last k of a k-major
// operand, where the next row follows, is sent past the end by its lanes.

struct DmaSrc {
    const char* base;
    int64_t left;  // bytes from base to the operand's end (free-major: to the split's)
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

    __device__ __forceinline__ void init(const Operand& o, int64_t free0, int64_t k0, int64_t k_hi) {
        static_assert(THREADS % T::kPerRow == 0 && (THREADS / T::kPerRow) % 16 == 0 || !KMAJOR,
                      "a thread's loads share their chunk's place in the row");
        const int t = threadIdx.x;
        s.base = (const char*)(o.p + (KMAJOR ? free0 * o.ld + k0 : k0 * o.ld + free0));
        s.left = ((KMAJOR ? o.free : min(o.k, k_hi)) * o.ld) * 2 - (s.base - (const char*)o.p);
        s.step = (KMAJOR ? STEP : STEP * o.ld) * 2;
        k_chunk = T::chunk_of(t);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int q = t + j * THREADS;
            off[j] = (uint32_t)(T::row_of(q) * o.ld * 2) + T::chunk_of(q) * 16;
        }
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
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: what is declared is that it changes
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(to), "v"(o), "s"(r)
                     : "memory", "m0");
#pragma clang diagnostic pop
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
// read, the loads into the step just read out start, and the matrix cores are busy meanwhile
// (the barrier sits where a quarter of those products is left).
// Loads past the last step are started all the same, so that the count of pending loads is the
// same in every step.  They write zeros.
template <int BM, int BN, int WM, int WN, int STEP, int STAGES, int MS, bool AK, bool BK>
__global__ __launch_bounds__(WM * WN * 64, WM * WN == 4 && BM == 256 ? 1 : 2) void mm_dma_kernel(const MmArgs g) {
    constexpr int THREADS = WM * WN * 64;
    constexpr int TM = BM / WM, TN = BN / WN, MI = TM / MS, NI = TN / MS;
    using M = Mfma<MS>;
    using DA = Dma<AK, BM, STEP, THREADS>;
    using DB = Dma<BK, BN, STEP, THREADS>;
    constexpr int ACH = DA::T::kChunks, BCH = DB::T::kChunks, SUB = STEP / M::KS;
    static_assert(STAGES * (ACH + BCH) * 16 >= WM * WN * 32 * kRowPad * 4, "the epilogue's rows fit the tiles' LDS");
    __shared__ u32x4 lds[STAGES * (ACH + BCH)];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int64_t m0 = g.m_first + (int64_t)tm * BM, n0 = g.n_first + (int64_t)tn * BN;
    const int64_t k_lo = (int64_t)blockIdx.y * g.k_split;
    const int k_all = (int)(min(g.k, k_lo + g.k_split) - k_lo);
    const int steps = (k_all + STEP - 1) / STEP;

    typename M::acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = typename M::acc_t{};

    DA da;
    DB db;
    bf16x8 fa[2][MI], fb[2][NI];
    da.init(g.a, m0, k_lo, k_lo + g.k_split);
    db.init(g.b, n0, k_lo, k_lo + g.k_split);
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    int k_left = k_all;
    constexpr int LOADS = DA::kPer + DB::kPer, EARLY = LOADS / 2;
    // load j of the step that comes next in the order of loading
    auto issue = [&](int stage, int j) __attribute__((always_inline)) {
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
    auto read = [&](int stage, int s, int f) __attribute__((always_inline)) {
        const u32x4* t = lds + stage * (ACH + BCH);
        const int slot = s & 1;
        if (f >= 1 && f <= NI)
            fb[slot][f - 1] = read_frag<BK, BN, STEP, MS>(t + ACH, wn * TN + (f - 1) * MS, s * M::KS, lane);
        else {
            const int i = f == 0 ? 0 : f - NI;
            fa[slot][i] = read_frag<AK, BM, STEP, MS>(t, wm * TM + i * MS, s * M::KS, lane);
        }
    };
    constexpr int PENDING = (STAGES - 2) * LOADS;
    constexpr int MF = MI * NI, BARX = MF * 3 / 4;
    // An odd number of steps ends with one of zeros: without a way out between the stages the
    // compiler finds registers that save 2 % (with both operands free-major it finds too few).
    constexpr bool EVEN = BM == 256 && BN == 256 && AK;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
        for (int j = 0; j < LOADS; ++j) issue(i, j);
    step_barrier<PENDING>();
#pragma unroll
    for (int f = 0; f < MI + NI; ++f) read(0, 0, f);
#pragma unroll
    for (int j = 0; j < EARLY; ++j) issue(STAGES - 1, j);
    for (int it = 0; it < steps; it += STAGES) {
#pragma unroll
        for (int stage = 0; stage < STAGES; ++stage) {
            if (!EVEN && it + stage >= steps) break;
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const bool last = s + 1 == SUB;
                // Between two products: the reads of the next fragments, and behind the barrier and
                // in the next step's first products half of a step's loads each.
#pragma unroll
                for (int x = 0; x < MF; ++x) {
                    if (last && x == BARX) step_barrier<PENDING>();
                    acc[x / NI][x % NI] = M::mul(fa[s & 1][x / NI], fb[s & 1][x % NI], acc[x / NI][x % NI]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (last) {
                        if (x >= BARX) {
                            spread<MF - BARX, MI + NI>(x - BARX, [&](int f) __attribute__((always_inline)) {
                                read(stage + 1 == STAGES ? 0 : stage + 1, 0, f);
                            });
                            spread<MF - BARX, EARLY>(
                                x - BARX, [&](int j) __attribute__((always_inline)) { issue(stage, j); });
                        }
                    } else {
                        spread<MF, MI + NI>(x, [&](int f) __attribute__((always_inline)) { read(stage, s + 1, f); });
                        if (s == 0)
                            spread<MF, LOADS - EARLY>(x, [&](int j) __attribute__((always_inline)) {
                                issue(stage == 0 ? STAGES - 1 : stage - 1, EARLY + j);
                            });
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
    step_barrier<0>();  // the epilogue takes over the LDS that the last loads were written to
    store_acc<MS, MI, NI>(g, acc, (float*)lds + wave * 32 * kRowPad, m0 + wm * TM, n0 + wn * TN, lane);
}

// The splits' partial sums, joined in order, and the epilogue: rows are padded to 64 columns
// so that a checkpoint's blocks stay within eight lanes.
__global__ __launch_bounds__(256) void mm_join_kernel(const MmArgs g, int splits, int64_t per_row, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = t / per_row, col = (t - row * per_row) * 8, left = g.n - col;
    const int valid = row >= g.m || left <= 0 ? 0 : left < 8 ? (int)left : 8;
    const float* part = g.part + row * g.n + col;
    float v[8], u[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    // eight splits' loads at a time, added in order
    for (int s0 = 0; s0 < splits; s0 += 8) {
#pragma unroll
        for (int s = 0; s < 8; ++s) load_chunk(part + min(s0 + s, splits - 1) * (g.m * g.n), valid, u[s]);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = s0 + s < splits ? v[i] + u[s][i] : v[i];
    }
    epilogue(g.ep, row, g.n, col, valid, v);
}

// ---- few rows ---------------------------------------------------------------------------
//
// Up to 16 rows of k-major operands, the single tokens of serving: latencies and launches bind.
// A workgroup takes 16 columns and all of k, so that nothing is joined in a second launch: its
// waves take blocks of 64 k in turn, each row of a block one line of 128 bytes, straight into
// registers, kFewAhead blocks ahead of the products, and their sums meet in LDS in a fixed
// order.  Rows past the operands' ends read the last row, and what comes of them is not stored.
// Rows of any alignment are read as they are.  Eight and sixteen waves were slower (16 x 4096 ->
// 4096: 13.3 and 16.7 us against 12.0), and so were 32 and 64 columns (17 and 27).
constexpr int kFewAhead = 4, kFewWaves = 4;

// Eight elements from col on of a row of k, zeros past its end; none of the loads waits for
// another.
__device__ __forceinline__ u32x4 row_end(const uint16_t* row, int64_t col, int64_t k) {
    u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t e = row[min(col + i, k - 1)];
        w[i >> 1] |= (col + i < k ? e : 0u) << (16 * (i & 1));
    }
    return w;
}

__global__ __launch_bounds__(kFewWaves * 64) void mm_few_kernel(const MmArgs g) {
    using M = Mfma<16>;
    constexpr int SUB = kStep / M::KS;
    __shared__ float sums[kFewWaves][16][17];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int r = lane & 15, c = (lane >> 4) * 8;
    const uint16_t* pa = g.a.p + min((int64_t)r, g.m - 1) * g.a.ld;
    const uint16_t* pb = g.b.p + min(n0 + r, g.n - 1) * g.b.ld;

    M::acc_t acc = {};
    u32x4 fa[kFewAhead][SUB], fb[kFewAhead][SUB];
    const int blocks = (int)(g.k / kStep), mine = blocks > wave ? (blocks - wave + kFewWaves - 1) / kFewWaves : 0;
    auto load = [&](int slot, int x) __attribute__((always_inline)) {
        const int64_t k0 = ((int64_t)min(x, mine - 1) * kFewWaves + wave) * kStep + c;
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            fa[slot][s] = load16(pa + k0 + s * M::KS);
            fb[slot][s] = load16(pb + k0 + s * M::KS);
        }
    };
    auto mul = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
            acc = M::mul(__builtin_bit_cast(bf16x8, fa[slot][s]), __builtin_bit_cast(bf16x8, fb[slot][s]), acc);
    };
    if (mine > 0) {
#pragma unroll
        for (int d = 0; d < kFewAhead; ++d) load(d, d);
        int x = 0;
        for (; x + kFewAhead <= mine; x += kFewAhead) {
#pragma unroll
            for (int d = 0; d < kFewAhead; ++d) {
                mul(d);
                load(d, x + d + kFewAhead);
            }
        }
#pragma unroll
        for (int d = 0; d < kFewAhead; ++d)
            if (x + d < mine) mul(d);
    }
    if (wave == blocks % kFewWaves && (int64_t)blocks * kStep < g.k) {  // the last, short block
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            const int64_t k0 = (int64_t)blocks * kStep + s * M::KS + c;
            fa[0][s] = row_end(pa, k0, g.k);
            fb[0][s] = row_end(pb, k0, g.k);
        }
        mul(0);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) sums[wave][M::row(x, lane)][r] = acc[x];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int row = threadIdx.x >> 1, at = (threadIdx.x & 1) * 8;
        const int64_t left = g.n - n0 - at;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) v[i] += sums[w][row][at + i];
        }
        epilogue(g.ep, row, g.n, n0 + at, row >= g.m || left <= 0 ? 0 : left < 8 ? (int)left : 8, v);
    }
}

constexpr int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// The layouts that occur: both operands k-major, the second free-major, both free-major.
enum : int { kKK = 0, kKF = 1, kFF = 2 };
int layout_of(bool ak, bool bk) { return ak ? (bk ? kKK : kKF) : kFF; }

// The tile shapes.  `slots` workgroups are at work at once; `step_us` is the time of one step of
// 64 k with one workgroup on a compute unit and with all slots taken, `tile_us` that of a
// tile's start and epilogue.
struct Shape {
    int bm, bn, threads, slots;
    double step_us[2], tile_us;
    const void* kernel[3];
};
template <int BM, int BN, int WM, int WN, int STAGES>
Shape shape(int slots, double alone_us, double full_us, double tile_us) {
    return {BM, BN, WM * WN * 64, slots, {alone_us, full_us}, tile_us,
            {(const void*)&mm_dma_kernel<BM, BN, WM, WN, kStep, STAGES, 16, true, true>,
             (const void*)&mm_dma_kernel<BM, BN, WM, WN, kStep, STAGES, 16, true, false>,
             (const void*)&mm_dma_kernel<BM, BN, WM, WN, kStep, STAGES, 16, false, false>}};
}
constexpr int kShapes = 5;
const Shape& shape_at(int i) {
    static const Shape shapes[kShapes] = {
        shape<256, 256, 2, 4, 2>(256, 1.38, 1.38, 12.0),
        shape<128, 128, 2, 2, 2>(512, 0.78, 1.02, 5.5),
        shape<64, 128, 1, 2, 3>(512, 0.55, 0.65, 5.0),
        shape<128, 64, 2, 1, 3>(512, 0.55, 0.65, 5.0),
        shape<32, 256, 1, 4, 4>(256, 0.48, 0.48, 2.5),
    };
    return shapes[i];
}

// Rows of whole 16-byte chunks can go past the registers.  A copy of an operand in such rows
// costs its bytes twice; that is cheap beside a large product, whose steps are faster by half.
bool chunked(const Operand& o) { return o.ld % 8 == 0; }
int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
double copy_us(const Operand& o) { return 3.0 + (double)(o.free * o.k) * 4.0 / 4.5e6; }

// Rounds of `tiles` workgroups of `steps` each.
double round_us(const Shape& s, int64_t tiles, int64_t steps) {
    return tiles_of(tiles, s.slots) * (steps * s.step_us[tiles > 256] + s.tile_us);
}
constexpr double kTailUs = 8.0;  // a second launch, and the first one's last tiles end alone

struct Plan {
    int shape;  // -1: the tile staged through registers
    int splits;
    int tail_shape;
    int64_t tail_m, tail_n;  // rows or columns from here on go in a second launch (m and n: none)
};

// The shape and the splits of the contraction that finish first: rounds of workgroups, each the
// steps of its split, and for splits the time to write the partial sums and to join them.
// Splits are what fills the chip where there are few tiles and many k.
Plan plan(const Operand& a, const Operand& b) {
    const int64_t m = a.free, n = b.free, steps = tiles_of(a.k, kStep);
    const bool fast = chunked(a) && chunked(b);
    const double copies = (chunked(a) ? 0.0 : copy_us(a)) + (chunked(b) ? 0.0 : copy_us(b));
    Plan best = {0, 1, 0, m, n};
    double best_us = 0.0;
    for (int i = fast ? 0 : -1; i < kShapes; ++i) {
        // the tile staged through the registers reaches half the rate of the others
        const Shape s = i >= 0 ? shape_at(i) : Shape{128, 128, 256, 512, {0.9, 1.3}, 8.0, {}};
        const int64_t tiles = tiles_of(m, s.bm) * tiles_of(n, s.bn);
        for (int64_t splits = 1; splits <= 64; splits = splits < 8 ? splits + 1 : splits * 5 / 4) {
            const int64_t per = tiles_of(steps, splits);
            if (splits > 1 && (per < 4 || tiles_of(steps, per) < splits)) continue;
            double us = round_us(s, tiles * splits, per) + (i >= 0 ? copies : 0.0);
            if (splits > 1) us += 4.0 + splits * (double)(m * n) * 8.0 / 6e6;
            if (best_us == 0.0 || us < best_us) {
                best = {i, (int)splits, 0, m, n};
                best_us = us;
            }
        }
    }
    // Where the last round would leave most of the chip idle, the columns or rows that fill whole
    // rounds go first and a second launch takes the rest in the tiles that suit them (8192 x 4096
    // -> 11008, 5.4 rounds of the large tile: 620 us in one launch, 608 in two; 3136 x 5347 over
    // 3636, 1.1 rounds: 179 and 136).
    for (int i = 0; i < kShapes; ++i) {
        const Shape& s = shape_at(i);
        const int64_t tm = tiles_of(m, s.bm), tn = tiles_of(n, s.bn), whole = tm * tn / s.slots * s.slots;
        for (int rows = 0; rows < 2; ++rows) {
            const int64_t across = rows ? tn : tm, first = whole / across, at = first * (rows ? s.bm : s.bn);
            if (first < 1 || at >= (rows ? m : n)) continue;
            const int64_t tail_rows = rows ? m - at : m, tail_cols = rows ? n : n - at;
            const double us = copies + kTailUs + round_us(s, first * across, steps);
            for (int j = 0; j < kShapes; ++j) {
                const Shape& t = shape_at(j);
                const double all = us + round_us(t, tiles_of(tail_rows, t.bm) * tiles_of(tail_cols, t.bn), steps);
                if (all < best_us) {
                    best = {i, 1, j, rows ? at : m, rows ? n : at};
                    best_us = all;
                }
            }
        }
    }
    return best;
}

const void* pick_mm(int layout) {
    if (layout == kKK) return (const void*)&mm_kernel<128, 128, 2, 2, true, true>;
    if (layout == kKF) return (const void*)&mm_kernel<128, 128, 2, 2, true, false>;
    return (const void*)&mm_kernel<128, 128, 2, 2, false, false>;
}

// An operand's copy in rows of `ld` elements, zeros past its columns: a k-major operand's zeros
// take part in the products.
__global__ __launch_bounds__(256) void pad_kernel(const uint16_t* in, int64_t rows, int64_t cols, uint16_t* out,
                                                  int64_t ld, int64_t t0) {
    const int64_t t = t0 + (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = ld / 8;
    const int64_t row = rows * per_row < (int64_t)1 << 31 ? (uint32_t)t / (uint32_t)per_row : t / per_row;
    if (row >= rows) return;
    const int64_t col = (t - row * per_row) * 8, left = cols - col;
    RawChunk<uint16_t> c;
    c.load(in + row * cols + col, left < 8 ? (int)left : 8);
    store16(out + row * ld + col, c.w);
}

hipError_t pad(Operand& o, bool kmajor, uint16_t* to, hipStream_t stream) {
    int64_t rows = kmajor ? o.free : o.k, cols = kmajor ? o.k : o.free, ld = padded(cols), t0 = 0;
    const uint16_t* from = o.p;
    void* args[] = {(void*)&from, (void*)&rows, (void*)&cols, (void*)&to, (void*)&ld, (void*)&t0};
    const int64_t chunks = rows * (ld / 8);
    for (; t0 < chunks; t0 += kMaxGrid * 256) {
        const int64_t left = chunks - t0;
        const int64_t blocks = left < kMaxGrid * 256 ? tiles_of(left, 256) : kMaxGrid;
        const hipError_t err = hipLaunchKernel((const void*)&pad_kernel, dim3((unsigned)blocks), dim3(256), args, 0, stream);
        if (err != hipSuccess) return err;
    }
    o.p = to;
    o.ld = ld;
    if (kmajor) o.k = ld;
    return hipSuccess;
}

Operand operand_a(const MmParams& p) { return {p.a, p.m, p.k, p.a_kmajor ? p.k : p.m}; }
Operand operand_b(const MmParams& p) { return {p.b, p.n, p.k, p.b_ld ? p.b_ld : p.b_kmajor ? p.k : p.n}; }

// Where a few rows' products take fewer microseconds in one launch of 16 columns a workgroup than
// in tiles with k split: 4 x 1000 -> 4000 6.4 against 11.0, 16 x 4096 -> 4096 12.0 against 14.8,
// 16 x 1003 -> 1001, whose rows would be copied, 9.7 against 16.3.  Past 4096 columns, with more
// than a workgroup on a compute unit, the rows of A are read too often (16 x 4096 -> 11008 29.9
// against 23.0); past 4096 k a workgroup's waves take too long (16 x 14336 -> 1000 29.0 against
// 21.6).  A checkpoint's blocks would span workgroups.
bool few_rows(const MmParams& p, bool with_ckpt) {
    return p.a_kmajor && p.b_kmajor && p.m <= 16 && p.n <= 4096 && p.k <= 4096 && !with_ckpt;
}

hipError_t launch_few(const MmParams& p, hipStream_t stream) {
    MmArgs g = {};
    g.a = operand_a(p);
    g.b = operand_b(p);
    g.m = p.m;
    g.n = p.n;
    g.k = p.k;
    g.ep = p.ep;
    void* args[] = {(void*)&g};
    return hipLaunchKernel((const void*)&mm_few_kernel, dim3((unsigned)tiles_of(p.n, 16)), dim3(kFewWaves * 64), args, 0,
                           stream);
}

// The workspace of a product: partial sums, then the operands' copies.
struct Spaces {
    int64_t part, a, b;
};
Spaces spaces(const MmParams& p, const Plan& pl) {
    auto round16 = [](int64_t n) { return (n + 15) / 16 * 16; };
    const Operand a = operand_a(p), b = operand_b(p);
    Spaces s = {pl.splits > 1 ? round16(pl.splits * p.m * p.n * 4) : 0, 0, 0};
    if (pl.shape >= 0 && !chunked(a)) s.a = (p.a_kmajor ? p.m : p.k) * padded(p.a_kmajor ? p.k : p.m) * 2;
    if (pl.shape >= 0 && !chunked(b)) s.b = (p.b_kmajor ? p.n : p.k) * padded(p.b_kmajor ? p.k : p.n) * 2;
    return s;
}

}  // namespace

int64_t mm_padded(int64_t n) { return padded(n); }

int64_t mm_workspace(const MmParams& p, bool with_ckpt) {
    if (p.m <= 0 || p.n <= 0 || few_rows(p, with_ckpt)) return 0;
    const Spaces s = spaces(p, plan(operand_a(p), operand_b(p)));
    return s.part + s.a + s.b;
}

hipError_t launch_mm(const MmParams& p, hipStream_t stream) {
    if (few_rows(p, p.ep.ckpt.codes)) return launch_few(p, stream);
    MmArgs g;
    g.a = operand_a(p);
    g.b = operand_b(p);
    const Plan pl = plan(g.a, g.b);
    const Spaces space = spaces(p, pl);
    char* at = (char*)p.workspace;
    hipError_t err = hipSuccess;
    if (space.a) err = pad(g.a, p.a_kmajor, (uint16_t*)(at + space.part), stream);
    if (err == hipSuccess && space.b) err = pad(g.b, p.b_kmajor, (uint16_t*)(at + space.part + space.a), stream);
    if (err != hipSuccess) return err;
    g.m = p.m;
    g.n = p.n;
    g.k = g.a.k;  // with the zeros of a copy
    const int layout = layout_of(p.a_kmajor, p.b_kmajor);
    g.k_split = tiles_of(tiles_of(p.k, kStep), pl.splits) * kStep;
    g.part = pl.splits > 1 ? (float*)at : nullptr;
    g.ep = p.ep;
    void* args[] = {(void*)&g};
    auto tiles = [&](int shape, int64_t m0, int64_t m1, int64_t n0, int64_t n1) {
        const Shape* s = shape >= 0 ? &shape_at(shape) : nullptr;
        g.tiles_m = (int)tiles_of(m1 - m0, s ? s->bm : 128);
        g.tiles_n = (int)tiles_of(n1 - n0, s ? s->bn : 128);
        g.m_first = m0;
        g.n_first = n0;
        return hipLaunchKernel(s ? s->kernel[layout] : pick_mm(layout),
                               dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n), (unsigned)pl.splits),
                               dim3(s ? s->threads : 256), args, 0, stream);
    };
    err = tiles(pl.shape, 0, pl.tail_m, 0, pl.tail_n);
    if (err == hipSuccess && pl.tail_n < p.n) err = tiles(pl.tail_shape, 0, p.m, pl.tail_n, p.n);
    if (err == hipSuccess && pl.tail_m < p.m) err = tiles(pl.tail_shape, pl.tail_m, p.m, 0, p.n);
    if (err != hipSuccess || pl.splits == 1) return err;
    int64_t per_row = tiles_of(p.n, 64) * 8, t0 = 0;
    int splits = pl.splits;
    const int64_t chunks = p.m * per_row;
    void* jargs[] = {(void*)&g, (void*)&splits, (void*)&per_row, (void*)&t0};
    for (; t0 < chunks; t0 += kMaxGrid * 256) {
        const int64_t left = chunks - t0;
        const int64_t blocks = left < kMaxGrid * 256 ? tiles_of(left, 256) : kMaxGrid;
        err = hipLaunchKernel((const void*)&mm_join_kernel, dim3((unsigned)blocks), dim3(256), jargs, 0, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// ---- column sums ------------------------------------------------------------------------

namespace {

// A column's sum on its way out.
struct ColOut {
    void* p;
    int f32, accumulate;
    __device__ __forceinline__ void put(int64_t c, float v) const {
        if (f32) {
            float* o = (float*)p + c;
            *o = accumulate ? v + *o : v;
        } else {
            uint16_t* o = (uint16_t*)p + c;
            *o = bf16_rne(accumulate ? v + __uint_as_float((uint32_t)*o << 16) : v);
        }
    }
};

// Bound by HBM: 8192 x 11008 takes 30 us (6.1 TB/s) and 5 to join, in eight workgroups per
// compute unit.  Sums of 8 << lanes_log2 columns per workgroup over every gridDim.y-th group of rows, a row to
// 1 << lanes_log2 lanes (all 64 of a wave from 512 columns on): partial sums, or with one group
// the result.
__global__ __launch_bounds__(256) void col_sum_kernel(const uint16_t* x, int64_t rows, int64_t n, int lanes_log2,
                                                      float* part, ColOut out) {
    __shared__ float join[256 * 8];
    const int lane = threadIdx.x & ((1 << lanes_log2) - 1), team = threadIdx.x >> lanes_log2, teams = 256 >> lanes_log2;
    const int cols = 8 << lanes_log2;
    const int64_t col0 = (int64_t)blockIdx.x * cols, left = n - col0 - lane * 8;
    const int valid = left <= 0 ? 0 : left < 8 ? (int)left : 8;
    float s[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.y * teams + team; r < rows; r += (int64_t)gridDim.y * teams) {
        load_chunk(x + r * n + col0 + lane * 8, valid, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) join[team * cols + lane * 8 + i] = s[i];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += 256) {
        float v = 0.0f;
        for (int t = 0; t < teams; ++t) v += join[t * cols + c];
        if (col0 + c < n) {
            if (gridDim.y == 1) out.put(col0 + c, v);
            else part[blockIdx.y * n + col0 + c] = v;
        }
    }
}

// The groups' partial sums: 32 columns per workgroup, 32 threads down the groups.
__global__ __launch_bounds__(1024) void col_join_kernel(const float* part, int64_t groups, int64_t n, ColOut out) {
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, g0 = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cl;
    float v = 0.0f;
    if (c < n)
        for (int64_t g = g0; g < groups; g += 32) v += part[g * n + c];
    s[g0][cl] = v;
    __syncthreads();
    if (threadIdx.x < 32 && c < n) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s[i][cl];
        out.put(c, v);
    }
}

}  // namespace

namespace {
int col_lanes_log2(int64_t n) {
    int l = 0;
    while (l < 6 && (8 << l) < n) ++l;
    return l;
}
}  // namespace

int64_t col_sum_groups(int64_t rows, int64_t n) {
    const int l = col_lanes_log2(n);
    const int64_t blocks = tiles_of(n, 8 << l), teams = 256 >> l;
    const int64_t most = tiles_of(rows, teams * 8);  // a team takes eight rows or more
    const int64_t wanted = 2048 / blocks;  // eight workgroups on a compute unit
    const int64_t g = wanted < 1 ? 1 : wanted > 256 ? 256 : wanted;
    return g < most ? g : most < 1 ? 1 : most;
}

hipError_t launch_col_sum(const uint16_t* x, int64_t rows, int64_t n, float* part, void* out, bool f32, bool accumulate,
                          hipStream_t stream) {
    int64_t groups = col_sum_groups(rows, n);
    int lanes = col_lanes_log2(n);
    ColOut to = {out, f32, accumulate};
    void* args[] = {(void*)&x, (void*)&rows, (void*)&n, (void*)&lanes, (void*)&part, (void*)&to};
    hipError_t err = hipLaunchKernel((const void*)&col_sum_kernel,
                                     dim3((unsigned)tiles_of(n, 8 << lanes), (unsigned)groups), dim3(256), args, 0, stream);
    if (err != hipSuccess || groups == 1) return err;
    void* jargs[] = {(void*)&part, (void*)&groups, (void*)&n, (void*)&to};
    return hipLaunchKernel((const void*)&col_join_kernel, dim3((unsigned)((n + 31) / 32)), dim3(1024), jargs, 0, stream);
}

}  // namespace loco
