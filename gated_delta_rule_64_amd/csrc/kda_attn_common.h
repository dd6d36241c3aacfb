// Device-side parts shared by the attention kernels (prefill, its gradients,
// draft trees): the 32 x 32 matrix-core products for both element types, the
// ragged tile search and the bounded row loads.
//
// Matrix-core layouts used throughout (lane l, half h = l / 32, c = l % 32):
//   v_mfma_f32_32x32x16_bf16  A: row c, contraction 8 h .. 8 h + 7
//                             B: column c, contraction 8 h .. 8 h + 7
//   v_mfma_f32_32x32x2_f32    A: row c, contraction h;  B: column c, contraction h
//   result (both)             column c, register r holds row 8 (r / 4) + 4 h + r % 4
// A contraction index may be permuted as long as A and B agree, which is used
// twice.  First, an operand row is read in 16-byte pieces, piece 2 s + h by
// the lanes of half h: 8 bf16 (one product) or 4 floats (four products), the
// same bytes for A and B.  Second, a result becomes the B operand of the next
// product without leaving its registers: the rows that a lane holds are its
// contraction indices, and the A operand is read in that order.
#pragma once

#include "kda_common.h"

namespace kda {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The maximum that softmax weights are taken against moves only when a row
// outgrows it by 2^kRise: until then they stay below 2^kRise, which fp32 sums
// and bf16 weights hold as well as 1.  Most tiles then leave the sums as they
// are (16 multiplications per 32 channels and lane).
constexpr float kRise = 6.f;

// A weight is e^((s - m) scale), formed as 2^(s c - m c) with one fused
// multiply-add (c = scale log2(e)) while |m c| stays below 2^kFar: m c is off by
// half a step, at most 2^-12 there, less than the fp32 scores themselves.  Past
// it the maximum is taken off first (at |m c| of 2^33 the half step alone would
// make every weight of a row 0 or infinite).
constexpr float kFar = 4096.f;

constexpr int kBufferDword3 = 0x00020000;  // raw buffer: byte offsets, reads past the end give 0

// One 16-byte operand piece of A times one of B, added to a 32 x 32 result.
template <typename T>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mma<bf16>(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mma<float>(u32x4 a, u32x4 b, f32x16 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

// Sizes that depend on the element type: elements in 16 bytes, and the pieces
// into which the 32 rows of a result fall when it becomes an operand.
template <typename T>
struct Elem {
    static constexpr int kSize = sizeof(T);
    static constexpr int kPer16 = 16 / sizeof(T);
    static constexpr int kPieces = 16 / kPer16;  // bf16: 2 (16 rows each), fp32: 4 (8 rows each)
    static constexpr int kMfmas = sizeof(T) == 2 ? 1 : 4;  // products of one operand piece
    static constexpr int kTrReads = sizeof(T) == 2 ? 2 : 4;  // LDS reads of a transposed operand
};

// Piece p of a 32 x 32 result as a B operand: registers p * kPer16 ..
template <typename T>
__device__ __forceinline__ u32x4 as_operand(const f32x16& x, int p);
template <>
__device__ __forceinline__ u32x4 as_operand<bf16>(const f32x16& x, int p) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(x[8 * p + 2 * i], x[8 * p + 2 * i + 1]);
    return r;
}
template <>
__device__ __forceinline__ u32x4 as_operand<float>(const f32x16& x, int p) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(x[4 * p + i]);
    return r;
}

// The A operand that goes with as_operand(x, p) is the transpose of a row-major
// LDS tile: 32 columns as operand rows, contraction over the tile's rows in the
// order in which the lane's half holds them.  For bf16 two transposing LDS
// reads of four rows each: in a group of 16 lanes, lane i names row
// r0 + (i >> 2) at column col + 4 (i & 3) and receives column col + i of rows
// r0 .. r0 + 3 (TileRead::columns).
typedef short tr16_v4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 lds_read_tr(const char* p) {
    const tr16_v4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tr16_v4*)(p));
    return __builtin_bit_cast(uint2, v);
}
__device__ __forceinline__ uint2 buffer_load8(__amdgpu_buffer_rsrc_t r, int offset) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, offset, 0, 0));
}

// Asks the scheduler to keep kAhead LDS operands in front of the products that
// use them, in a block of kOperands operands of kReads reads and kMfmas
// products each (left to itself it issues a read, waits for it and multiplies).
template <int kOperands, int kAhead, int kMfmas, int kReads = 1>
__device__ __forceinline__ void lookahead() {
    constexpr int kMfma = 0x8, kDsRead = 0x100;
    constexpr int kFirst = kAhead < kOperands ? kAhead : kOperands;
    __builtin_amdgcn_sched_group_barrier(kDsRead, kFirst * kReads, 0);
#pragma unroll
    for (int i = 0; i < kOperands - kFirst; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, kMfmas, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, kReads, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, kFirst * kMfmas, 0);
}

// Larger of the two halves' values (lanes l and l + 32)
__device__ __forceinline__ float xor32_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, int offset) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}

// A value that the compiler knows nothing about.  A mask inside a wave-uniform
// branch compares with such a value and so stays in its branch: turned into
// selects, what one tile in many needs would cost every tile its compares.
template <typename X>
__device__ __forceinline__ X opaque(X x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Waits for loads that a loop uses in every pass.  Left to their first use
// inside the loop, the wait there (a count of loads in flight) would also wait
// for the tile that the pass has just put in flight, in every pass.
template <int N>
__device__ __forceinline__ void arrive(u32x4 (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

// A wave-uniform value in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Rows [first, first + rows) of a row-major matrix as a bounded buffer: reads
// past the last row give 0, so rows behind a sequence's end (the next
// sequence's, or memory that is not the tensor's) are never read.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, int64_t first, int64_t row_bytes, int rows) {
    const char* p = static_cast<const char*>(base) + first * row_bytes;
    const int64_t bytes = rows > 0 ? rows * row_bytes : 0;
    // (the same in every lane, and said so: a descriptor that the compiler
    // takes for different ones makes a loop over the lanes of every load)
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<char*>(uniform64(reinterpret_cast<int64_t>(p))), 0,
                                             uniform(static_cast<int>(bytes)), kBufferDword3);
}

// One tile of a packed batch: rows [start + first, start + len) of the tensor
// from its first row on, `first` a multiple of the tile height.
struct Tile {
    int64_t start;  // the sequence's first token
    int len;        // its tokens
    int level;      // tiles of the same sequence before this one
    int tiles;      // tiles of the sequence
    bool there;
};

// Sequence n's tokens, whatever cu holds: inside [0, T).
__device__ __forceinline__ void seq_bounds(const int32_t* cu, int n, int64_t T, int64_t& start, int& len) {
    if (cu == nullptr) {
        start = 0;
        len = static_cast<int>(T);
        return;
    }
    int64_t a = cu[n], b = cu[n + 1];
    a = a < 0 ? 0 : a > T ? T : a;
    b = b < a ? a : b > T ? T : b;
    start = a;
    len = static_cast<int>(b - a);
}

// Sum over the wave without the LDS path (as wave_sum, for whole numbers)
__device__ __forceinline__ int wave_sum_int(int x) {
    x += __builtin_amdgcn_mov_dpp(x, 0x121, 0xF, 0xF, false);
    x += __builtin_amdgcn_mov_dpp(x, 0x122, 0xF, 0xF, false);
    x += __builtin_amdgcn_mov_dpp(x, 0x124, 0xF, 0xF, false);
    x += __builtin_amdgcn_mov_dpp(x, 0x128, 0xF, 0xF, false);
    const auto a = __builtin_amdgcn_permlane16_swap(static_cast<unsigned>(x), static_cast<unsigned>(x), false, false);
    x = static_cast<int>(a[0] + a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(static_cast<unsigned>(x), static_cast<unsigned>(x), false, false);
    return uniform(static_cast<int>(b[0] + b[1]));
}

// The rank-th tile of the batch.  The tiles of a sequence follow each other, so
// that the workgroups that read the same keys (or queries) run at about the
// same time and find them in the L2; the longest sequences come first, and
// within one the levels fall (in causal attention a tile's work grows with its
// level), so that the short tiles fill the end.  Sequences are ordered so in
// groups of 64, a lane each: a lane counts the tiles of those before its own
// and the one whose range holds the rank answers.  All 64 lanes call it.
template <int kRows>
__device__ __forceinline__ Tile find_tile(const int32_t* cu, int N, int64_t T, int64_t rank) {
    Tile t;
    t.there = false;
    t.start = 0;
    t.len = t.level = t.tiles = 0;
    const int lane = threadIdx.x & 63;
    if (N == 1) {
        seq_bounds(cu, 0, T, t.start, t.len);
        t.len = uniform(t.len);
        t.start = uniform64(t.start);
        t.tiles = (t.len + kRows - 1) / kRows;
        t.there = rank < t.tiles;
        t.level = t.there ? t.tiles - 1 - static_cast<int>(rank) : 0;
        return t;
    }
    int left = static_cast<int>(rank);  // below 2^31 / kRows + N
    for (int n0 = 0; n0 < N; n0 += 64) {
        int64_t start = 0;
        int len = 0;
        if (n0 + lane < N) seq_bounds(cu, n0 + lane, T, start, len);
        const int mine = (len + kRows - 1) / kRows, all = wave_sum_int(mine);
        if (left >= all) {
            left -= all;
            continue;
        }
        int before = 0;
        for (int m = 0; m < min(64, N - n0); ++m) {
            const int other = __builtin_amdgcn_readlane(mine, m);
            before += other > mine || (other == mine && m < lane) ? other : 0;
        }
        const int owner = uniform(__ffsll(static_cast<long long>(__ballot(left >= before && left < before + mine))) - 1);
        t.start = __builtin_amdgcn_readlane(static_cast<int>(start), owner);  // below 2^31
        t.len = __builtin_amdgcn_readlane(len, owner);
        t.tiles = __builtin_amdgcn_readlane(mine, owner);
        t.level = t.tiles - 1 - (left - __builtin_amdgcn_readlane(before, owner));
        t.there = true;
        return t;
    }
    return t;
}

// Whether a key is before a row's window and not among the first tokens (key,
// least and sink from the same place on): one comparison, as 16 of two each
// would hold more masks than there are scalar registers.
__device__ __forceinline__ bool outside(int key, int least, int sink) { return ((key - least) & (sink - 1 - key)) < 0; }

// Whether a windowed workgroup takes 32 rows of four heads of a group, not 128 of one.
inline bool heads_share(int H, int Hkv) { return H / Hkv % 4 == 0; }

// The key tiles of kKeys that a tile of 128 query rows from q_first on attends,
// in order: all up to its own last row, or with a window (kWin) those that hold
// one of the sequence's first `sinks` tokens and those from the first row's
// window on.  A tile is named by its first key, a multiple of kKeys.
template <bool kWin, int kKeys>
struct KeyWalk {
    int len;
    int window, sinks;      // below 2^30 each, as are len and q_first
    int sink_end, win;      // the tiles before sink_end and from win on are walked
    __device__ __forceinline__ KeyWalk(int q_first, int len_, int window_, int sinks_) : len(len_) {
        if constexpr (kWin) {
            window = window_;
            sinks = sinks_;
            sink_end = (sinks + kKeys - 1) / kKeys * kKeys;
            win = max(0, q_first - window + 1) / kKeys * kKeys;
        } else {
            window = sinks = sink_end = win = 0;
        }
    }
    __device__ __forceinline__ int next(int j0) const {
        const int j = j0 + kKeys;
        if constexpr (kWin) return j >= sink_end ? max(j, win) : j;
        return j;
    }
    // Tiles that are walked before j0 (one that is walked itself, or the end)
    __device__ __forceinline__ int before(int j0) const {
        if constexpr (kWin) return j0 <= sink_end ? min(j0, sink_end) / kKeys : (j0 - max(win, sink_end) + sink_end) / kKeys;
        return j0 / kKeys;
    }
    // The n-th of them
    __device__ __forceinline__ int nth(int n) const {
        if constexpr (kWin) return n * kKeys < sink_end ? n * kKeys : n * kKeys + max(win - sink_end, 0);
        return n * kKeys;
    }
    // Rows of a tile that some row may attend; what is behind them reads as 0,
    // so that a value that is not finite there meets no weight of 0.
    __device__ __forceinline__ int rows(int j0) const {
        if constexpr (kWin) return min(kKeys, (j0 < win ? sinks : len) - j0);
        return min(kKeys, len - j0);
    }
    // The first token of row i's window (may be negative)
    __device__ __forceinline__ int least(int i) const { return i - window + 1; }
    // Whether the rows from q0 on have all left the tile behind them, and
    // whether the window of one of the 32 from q0 on begins behind its first key
    __device__ __forceinline__ bool passed(int j0, int q0) const {
        if constexpr (kWin) return j0 + kKeys <= least(q0) && j0 >= sinks;
        return false;
    }
    __device__ __forceinline__ bool edge(int j0, int q0) const { return kWin && j0 < least(q0 + 31) && j0 + kKeys > sinks; }
};

// A tile in LDS without padding: rows of kPieces 16-byte pieces, piece p of row
// r stored in place p ^ turn(r).  LDS has 64 banks of 4 bytes, 16 pieces side
// by side, and the turn is such that neither way of reading meets itself in a
// bank: the same piece of 16 rows (operand rows), or 64 bytes of each of four
// neighbouring rows (transposed).  It depends on r % 16 alone.
template <int kPieces>
__device__ __forceinline__ int turn(int r) {
    if constexpr (kPieces % 16 == 0) return (r & 3) << 2 | (r >> 2 & 3);      // a row fills the banks
    else if constexpr (kPieces % 8 == 0) return (r >> 1 & 1) << 2 | (r >> 2 & 3);  // rows start 8 pieces apart
    else if constexpr (kPieces == 4) return r >> 2 & 3;
    else return r >> 3 & 1;
}

// Reads of such a tile (columns of T, kCols a row) by one lane.  The lane's
// offsets are computed once; tiles, rows 32 apart and neighbouring tiles in
// LDS are constant offsets from them.
template <typename T, int kCols>
struct TileRead {
    static constexpr int kRow = kCols * static_cast<int>(sizeof(T));
    static constexpr int kPieces = kRow / 16;
    static constexpr int kOps = kPieces / 2;          // operand pieces of a row, per half
    static constexpr int kTiles = (kCols + 31) / 32;  // 32-column tiles, transposed
    // bf16: the offsets themselves; fp32, whose products leave the vector
    // units idle and whose rows would take twice the registers: what they are
    // made of
    static constexpr bool kStored = sizeof(T) == 2;
    int row[kStored ? kOps : 2];
    int col[kStored ? kTiles : 1][2];
    // operand rows: this lane's row is c
    __device__ __forceinline__ void init_rows(int c, int half) {
        if constexpr (kStored) {
#pragma unroll
            for (int p = 0; p < kOps; ++p) row[p] = c * kRow + ((2 * p + half) ^ turn<kPieces>(c)) * 16;
        } else {
            row[0] = c * kRow;
            row[1] = (half ^ turn<kPieces>(c)) * 16;
        }
    }
    __device__ __forceinline__ u32x4 rows(const char* tile, int p) const {
        if constexpr (kStored) return *reinterpret_cast<const u32x4*>(tile + row[p]);
        else return *reinterpret_cast<const u32x4*>(tile + row[0] + (row[1] ^ 32 * p));
    }
    // transposed: see lds_read_tr for which lane names which element.  A
    // 32-column tile of a narrower matrix reads into the row behind it, and
    // up to 64 bytes behind the last; those results are not used.
    __device__ __forceinline__ void init_columns(int lane) {
        const int half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            const int i = lane & 15, g = lane >> 4 & 1;
            const int r = 4 * half + (i >> 2);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const int piece = 4 * t + 2 * g + ((i & 3) >> 1);
                col[t][0] = r * kRow + (piece ^ turn<kPieces>(r)) * 16 + (i & 1) * 8;
                col[t][1] = (r + 8) * kRow + (piece ^ turn<kPieces>(r + 8)) * 16 + (i & 1) * 8;
            }
        } else {
            col[0][0] = (lane & 31) * 4;
            col[0][1] = 4 * half;
        }
    }
    __device__ __forceinline__ u32x4 columns(const char* tile, int t, int p) const {
        if constexpr (sizeof(T) == 2) {
            const uint2 a = lds_read_tr(tile + 16 * p * kRow + col[t][0]), b = lds_read_tr(tile + 16 * p * kRow + col[t][1]);
            return u32x4{a.x, a.y, b.x, b.y};
        } else {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 8 * p + col[0][1] + i;
                r[i] = *reinterpret_cast<const uint32_t*>(tile + at * kRow + ((128 * t + col[0][0]) ^ turn<kPieces>(at) * 16));
            }
            return r;
        }
    }
};
constexpr int tr_slack(int cols) { return cols < 32 ? 64 : 0; }

// Copy of kRows rows into such a tile in two steps: load() puts this thread's
// pieces in flight, store() writes them to LDS.
template <typename T, int kRows, int kCols, int kThreads>
struct TileCopy {
    static constexpr int kRow = kCols * static_cast<int>(sizeof(T));
    static constexpr int kRowPieces = kRow / 16;
    static constexpr int kPieces = kRows * kRowPieces;
    static constexpr int kEach = (kPieces + kThreads - 1) / kThreads;
    static constexpr int kBytes = kRows * kRow;
    u32x4 r[kEach];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t src, int row_bytes, int tid) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = tid + i * kThreads;
            if (kPieces % kThreads == 0 || p < kPieces)
                r[i] = buffer_load16(src, (p / kRowPieces) * row_bytes + (p % kRowPieces) * 16);
        }
    }
    __device__ __forceinline__ void store(char* dst, int tid) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = tid + i * kThreads, row = p / kRowPieces;
            if (kPieces % kThreads == 0 || p < kPieces)
                *reinterpret_cast<u32x4*>(dst + row * kRow + (p % kRowPieces ^ turn<kRowPieces>(row)) * 16) = r[i];
        }
    }
};

__device__ __forceinline__ void wave_lds_fence() {
    // LDS operations of one wave complete in order; this keeps the compiler
    // from moving them past each other (lanes read what other lanes wrote)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Hands out a transposed result (lane column c: row c; register 4 i + e of tile
// t: channel 32 t + 8 i + 4 half + e) as 16-byte pieces of whole rows:
// put(row, channel, values), neighbouring lanes with neighbouring pieces, so
// that stores (and the loads that go with them) take whole rows; straight from
// the registers a store instruction touches 32 rows, 16 bytes of each.
// lds: 32 * D floats of this wave's own.
template <typename T, int D, int kTiles, typename Put>
__device__ __forceinline__ void by_rows(char* lds, const f32x16 (&acc)[kTiles], int lane, Put put) {
    constexpr int kPieces = D / 4, kPer = 16 / static_cast<int>(sizeof(T));
    const int c = lane & 31, half = lane >> 5;
    wave_lds_fence();
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = 8 * t + 2 * i + half;
            if (4 * p < D)
                *reinterpret_cast<f32x4*>(lds + c * D * 4 + (p ^ turn<kPieces>(c)) * 16) =
                    f32x4{acc[t][4 * i], acc[t][4 * i + 1], acc[t][4 * i + 2], acc[t][4 * i + 3]};
        }
    wave_lds_fence();
#pragma unroll
    for (int n = 0; n < 32 * D / (64 * kPer); ++n) {
        const int at = lane + 64 * n, row = at / (D / kPer), ch = at % (D / kPer) * kPer;
        float y[kPer];
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(lds + row * D * 4 + ((ch / 4 + q) ^ turn<kPieces>(row)) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[4 * q + e] = x[e];
        }
        put(row, ch, y);
    }
}
__device__ __forceinline__ void store_piece(bf16* p, const float (&x)[8]) { st8(p, x); }
__device__ __forceinline__ void store_piece(float* p, const float (&x)[4]) { st4(p, x); }
__device__ __forceinline__ void unpack_piece(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack_piece(u32x4 v, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
}

// Workgroup barrier that orders LDS accesses only: loads from memory stay in
// flight across it.
__device__ __forceinline__ void tile_barrier() { lds_barrier(); }

}  // namespace attn
}  // namespace kda
