// Attention of a tree of drafted tokens over a paged cache; with one token per
// sequence, plain decode.
//
// Row (t, g) of sequence b and key head f is query token t of head f G + g.
// It attends the sequence's committed tokens (in the cache's pages) and those
// drafted tokens whose bits its mask word has; the softmax is that of
// kda_attn_prefill.hip (S^T = K Q^T, running maximum and sum, O^T += V^T P^T).
//
// The cache is read once and sets the time, so every wave walks its own tiles
// of 32 keys (no barrier in the loop), the next tile's rows in flight in
// registers while one is worked on.  A sequence's tiles are split over the
// workgroup's waves and, where there are few sequences and heads, over
// workgroups: the parts (unnormalised sums, maximum, sum of weights, all fp32)
// are joined in LDS and, across workgroups, by a second kernel.
//
// bf16, 32 heads of 128 over 8: a decode step of 256 sequences of 1,024 to 4,096
// tokens reads 2.66 GB, what it cannot do without, in 461 us (5.8 TB/s of the
// 6.3 that a streaming read reaches); trees of 16 over 32 ragged sequences take
// 136 us with their join, 1.07 times the traffic; a chain of 4 over 262,144
// tokens 191 us (5.6 TB/s).
//
// With a window only the tiles that hold a first token or one of some row's
// window are walked; those where a window begins are masked per row, and values
// there that are not finite are taken out and given to the rows that attend them.
// The decode step under a window of 1,024: 1.08 GB in 192 us (5.6 TB/s); the trees
// under one of 2,000: 61 us for 244 MB (4.0 TB/s; a workgroup's start and the join
// of its waves are a fourth of its time).
#include <cfloat>

#include "kda_attn_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kKeys = 32;  // keys of a tile
constexpr int kMaxSplits = 256;

struct TreeK {
    int B, T, H, Hkv;
    float scale;
    const void *q, *k_new, *v_new, *z;
    const int64_t* mask;
    const void *k_cache, *v_cache;
    int pages, page_shift;
    const int32_t* table;
    int slots, max_pages;
    const int32_t *lens, *slot_indices;
    void* out;
    float* lse;
    float* part;   // [splits][B, Hkv, T G][dv]
    float* stats;  // [splits][B, Hkv, T G][2]: maximum (raw scores), sum of weights
    int splits, blocks;  // workgroups per (sequence, key head): parts of the keys, blocks of rows
    int units;           // all but the blocks: sequences, key heads and parts
    int window, sinks;
};

template <typename T, int DK, int DV>
struct TreeSizes {
    static constexpr int kTile = kKeys * (DK + DV) * static_cast<int>(sizeof(T)) + tr_slack(DV);
    static constexpr int kWaves = 4 * kTile <= 160 * 1024 ? 4 : 2;
    static constexpr int kVTiles = (DV + 31) / 32;
    static constexpr int kPart = kVTiles * 16 * 64 * 4;        // one wave's sums
    static constexpr int kJoin = kWaves / 2 * (kPart + 2 * 64 * 4);
    static constexpr int kLds = kWaves * kTile > kJoin ? kWaves * kTile : kJoin;
};

// The slot of sequence b and its committed tokens; false: a padding row.
__device__ __forceinline__ bool slot_of(const TreeK& a, int b, int& slot, int& ctx) {
    slot = a.slot_indices != nullptr ? a.slot_indices[b] : b;
    if (slot < 0 || slot >= a.slots) return false;
    const int64_t most = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int n = a.lens[slot];
    ctx = n < 0 ? 0 : static_cast<int>(n > most ? most : n);
    return true;
}

// What a row's sums are multiplied by, and its lse.  l is 0 where nothing is
// attended (m is -infinity), and where every attended score is -infinity (m is
// kLowest): that row is NaN, as is one whose l is NaN.
constexpr float kLowest = -FLT_MAX;
struct Norm {
    float inv, lse;
};
__device__ __forceinline__ bool attends(float m, float l) { return l != 0.f || m != -INFINITY; }
__device__ __forceinline__ Norm normalise(float m, float l, float sc) {
    if (l > 0.f) return Norm{1.f / l, (m * sc + __builtin_amdgcn_logf(l)) * kLn2};
    return attends(m, l) ? Norm{NAN, NAN} : Norm{0.f, -INFINITY};
}

// Final rows: y = o / l, gated, and the log of the sum.
template <typename T>
__device__ __forceinline__ void store4(T* out, const T* z, float (&y)[4]) {
    if (z != nullptr) {
        float g[4];
        ld4(z, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= sigmoid_fast(g[e]);
    }
    st4(out, y);
}

// Replaces the values of a 16-byte piece that are not finite by 0; other than 0
// if there are any.  An exponent of all ones is found by its carry.
template <typename T>
__device__ __forceinline__ uint32_t take_odd(u32x4& x) {
    constexpr uint32_t kExponent = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u, kOne = sizeof(T) == 2 ? 0x00800080u : 0x00800000u;
    constexpr uint32_t kCarry = sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t odd = ((x[i] & kExponent) + kOne) & kCarry;
        x[i] &= ~(sizeof(T) == 2 ? (odd >> 15) * 0xffffu : static_cast<uint32_t>(static_cast<int32_t>(odd) >> 31));
        any |= odd;
    }
    return any;
}

// kWin: of a row's tokens in order, the cached ones and then the drafts of its
// mask word, the last `window` and the first `sinks` are attended.
template <typename T, int DK, int DV, bool kWin>
__global__ __launch_bounds__((64 * TreeSizes<T, DK, DV>::kWaves), (sizeof(T) == 2 && DK <= 128 ? 2 : 1)) void attn_tree_kernel(TreeK a) {
    using Sz = TreeSizes<T, DK, DV>;
    constexpr int kE = sizeof(T);
    constexpr int kQPieces = DK / (2 * Elem<T>::kPer16);
    constexpr int kVTiles = Sz::kVTiles, kWaves = Sz::kWaves;
    constexpr int kP = Elem<T>::kPieces;
    constexpr int kKRow = DK * kE, kVRow = DV * kE;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 31, half = lane >> 5;
    char* sK = smem + wave * Sz::kTile;
    char* sV = sK + kKeys * kKRow;
    TileRead<T, DK> rk;
    TileRead<T, DV> rv;
    rk.init_rows(c, half);
    rv.init_columns(lane);

    const int G = a.H / a.Hkv, rows = a.T * G;
    // The row blocks of the same keys eight workgroups apart: on the same XCD
    // (workgroups go to the eight in turn) and at about the same time, so that
    // the keys come from its L2 for all but one of them.
    const int group = blockIdx.x / (8 * a.blocks), within = blockIdx.x % (8 * a.blocks);
    const int block = within / 8;
    int id = group * 8 + within % 8;
    if (id >= a.units) return;
    const int split = id % a.splits;
    id /= a.splits;
    const int kvh = id % a.Hkv, b = id / a.Hkv;
    int slot, ctx = 0;
    const bool real = slot_of(a, b, slot, ctx);
    slot = uniform(slot);
    ctx = uniform(ctx);

    // this lane's row (column of the transposed scores)
    const int row = block * 32 + c;
    const bool mine = row < rows;
    const int token = (mine ? row : 0) / G;
    const int64_t q_at = (static_cast<int64_t>(b) * a.T + token) * a.H + kvh * G + (mine ? row : 0) % G;  // the row in [B, T, H]
    f32x16 acc[kVTiles];
    float m = -INFINITY, l = 0.f;
    uint32_t any = 0;  // other than 0: the row attends some token of this wave's
#pragma unroll
    for (int i = 0; i < kVTiles; ++i) acc[i] = f32x16{};

    // The cache's tiles that some row reads: with a window those of the first
    // tokens, sink_tiles of them, and those from `skip` tiles further on.
    int ctx_tiles = (ctx + kKeys - 1) / kKeys, sink_tiles = ctx_tiles, skip = 0, low = 0, sinks = 0;
    if constexpr (kWin) {
        low = max(0, ctx - a.window);  // (a row of an empty mask word sees back to here)
        sinks = min(a.sinks, ctx);
        sink_tiles = (sinks + kKeys - 1) / kKeys;
        skip = max(0, low / kKeys - sink_tiles);
        ctx_tiles -= skip;
    }
    const int tiles = ctx_tiles + (a.T + kKeys - 1) / kKeys;
    const int each = (tiles + a.splits - 1) / a.splits;
    const int t_end = real ? min(tiles, (split + 1) * each) : 0;
    int tile = split * each + wave;

    if (tile < t_end) {
        // the row's query stays in registers, but for the longest fp32 one,
        // which is read again from the caches for every tile
        constexpr bool kKeep = kE == 2 || DK <= 128;
        u32x4 qf[kKeep ? kQPieces : 1];
        const char* q_row = static_cast<const char*>(a.q) + q_at * kKRow + half * 16;
        if constexpr (kKeep) {
#pragma unroll
            for (int p = 0; p < kQPieces; ++p) qf[p] = *reinterpret_cast<const u32x4*>(q_row + p * 32);
        }
        uint64_t seen = a.mask != nullptr ? static_cast<uint64_t>(a.mask[static_cast<int64_t>(b) * a.T + token])
                                          : ~0ull >> (63 - token);
        int least = 0;  // the first cached token of the row's window
        if constexpr (kWin) {
            seen &= ~0ull >> (64 - a.T);
            const int drafts = __popcll(seen);
            least = ctx + drafts - a.window;
            // a window of fewer tokens than the row's drafts: the first of them
            // go, but for those among the sequence's first tokens
            if (drafts > a.window) {
                const int stay = max(0, a.sinks - ctx);
                uint64_t rest = seen;
                for (int n = 0; n < drafts - a.window; ++n) {
                    if (n >= stay) seen &= ~(rest & -rest);
                    rest &= rest - 1;
                }
            }
        }
        const float sc = a.scale * kLog2e;

        // Half a tile: 16 rows of keys and of values, 16-byte pieces
        constexpr int kKPieces = kKRow, kVPieces = kVRow;  // 16 rows of kRow / 16 pieces
        constexpr int kKEach = (kKPieces + 63) / 64, kVEach = (kVPieces + 63) / 64;
        // fp32 tiles, twice as large, do not fit beside the sums: their halves
        // pass through the same registers when they are stored
        constexpr bool kAhead = kE == 2;
        u32x4 kr[kAhead ? 2 : 1][kKEach], vr[kAhead ? 2 : 1][kVEach];
        // The table entries of a tile's halves, read as scalars: a vector load
        // would have to be waited for behind the rows in flight.
        typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
        const scalar_ints entries = (scalar_ints)(a.table + static_cast<int64_t>(slot) * a.max_pages);
        struct Halves {
            int page[2], rows[2];  // rows that hold a token
        };
        const int in_page = (1 << a.page_shift) - 1;
        auto real = [&](int n) __attribute__((always_inline)) { return kWin && n >= sink_tiles ? n + skip : n; };
        auto look_up = [&](int n) __attribute__((always_inline)) {
            Halves e;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int first = real(n) * kKeys, t0 = first + 16 * x;
                // (a tile before every window: what is behind the first tokens reads as 0)
                e.rows[x] = min(16, max(0, (kWin && first + kKeys <= low ? sinks : ctx) - t0));
                // (clamped: a column behind the context is not looked at)
                e.page[x] = entries[min(t0, ctx - 1) >> a.page_shift];
            }
            return e;
        };
        auto fetch_half = [&](int n, Halves& e, int x) __attribute__((always_inline)) {
            const bool there = e.page[x] >= 0 && e.page[x] < a.pages;  // else its tokens are not attended
            e.rows[x] = there ? e.rows[x] : 0;
            const int64_t head = static_cast<int64_t>(there ? e.page[x] : 0) * a.Hkv + kvh;
            const int64_t first = (head << a.page_shift) + ((real(n) * kKeys + 16 * x) & in_page);
            const auto ks = rows_of(a.k_cache, first, kKRow, e.rows[x]);
            const auto vs = rows_of(a.v_cache, first, kVRow, e.rows[x]);
            const int to = kAhead ? x : 0;
#pragma unroll
            for (int i = 0; i < kKEach; ++i)
                if (kKPieces >= 64 || lane < kKPieces) kr[to][i] = buffer_load16(ks, (lane + 64 * i) * 16);
#pragma unroll
            for (int i = 0; i < kVEach; ++i)
                if (kVPieces >= 64 || lane < kVPieces) vr[to][i] = buffer_load16(vs, (lane + 64 * i) * 16);
        };
        auto put_half = [&](int x) __attribute__((always_inline)) {
            const int from = kAhead ? x : 0;
#pragma unroll
            for (int i = 0; i < kKEach; ++i) {
                const int p = lane + 64 * i, r = 16 * x + p / (kKRow / 16);
                if (kKPieces >= 64 || lane < kKPieces)
                    *reinterpret_cast<u32x4*>(sK + r * kKRow + (p % (kKRow / 16) ^ turn<kKRow / 16>(r)) * 16) = kr[from][i];
            }
#pragma unroll
            for (int i = 0; i < kVEach; ++i) {
                const int p = lane + 64 * i, r = 16 * x + p / (kVRow / 16);
                if (kVPieces >= 64 || lane < kVPieces)
                    *reinterpret_cast<u32x4*>(sV + r * kVRow + (p % (kVRow / 16) ^ turn<kVRow / 16>(r)) * 16) = vr[from][i];
            }
        };
        // the tile in LDS; hide(scores) masks its scores
        auto work = [&](auto hide) __attribute__((always_inline)) {
            wave_lds_fence();
            f32x16 s{};
#pragma unroll
            for (int p = 0; p < kQPieces; ++p) {
                u32x4 x;
                if constexpr (kKeep) x = qf[p];
                else x = *reinterpret_cast<const u32x4*>(q_row + p * 32);
                s = mma<T>(rk.rows(sK, p), x, s);
            }
            hide(s);
            float top = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
            top = xor32_max(top);
            if (__any((top - m) * sc > kRise)) {
                const float next = fmaxf(m, top);
                const float alpha = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - next) * sc);
                m = next;
                l *= alpha;
#pragma unroll
                for (int i = 0; i < kVTiles; ++i) acc[i] *= alpha;
            }
            float ms = m == -INFINITY ? 0.f : m * sc;
            if (__any(fabsf(ms) > kFar)) {
                const float off = opaque(m == -INFINITY ? 0.f : m);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] -= off;
                ms = 0.f;
            }
            float sum = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -ms));
                sum += s[r];
            }
            l += sum;
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const u32x4 x = as_operand<T>(s, p);
#pragma unroll
                for (int i = 0; i < kVTiles; ++i) acc[i] = mma<T>(rv.columns(sV, i, p), x, acc[i]);
            }
        };
        // register r of a score: key 8 (r / 4) + 4 half + r % 4 of the tile

        // adds the values of a row of V that are not finite, where this lane's row attends it
        // (four channels at a time: all at once would not fit beside the rows in flight)
        auto add_odd = [&](const T* from, bool attended) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    if (32 * i + 8 * r4 >= DV) continue;
                    float v[4];
                    ld4(from + 32 * i + 8 * r4 + 4 * half, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (attended && !(fabsf(v[e]) < INFINITY)) acc[i][4 * r4 + e] += v[e];
                    __builtin_amdgcn_sched_barrier(0);
                }
        };

        // the committed tokens: a tile's rows are in flight while the one
        // before is worked on, its table entries one tile earlier still
        const int c_end = min(t_end, ctx_tiles);
        if (tile < c_end) {
            Halves now = look_up(tile), next = now;
            if constexpr (kAhead) {
                fetch_half(tile, now, 0);
                fetch_half(tile, now, 1);
            }
            if (tile + kWaves < c_end) next = look_up(tile + kWaves);
            if constexpr (kKeep) arrive(qf);
            for (; tile < c_end; tile += kWaves) {
                wave_lds_fence();
                // where a window begins: the tile holds keys that some rows attend and others do not
                const int t0 = real(tile) * kKeys;
                const bool edge = kWin && t0 + kKeys > low && t0 - a.T < ctx - a.window && t0 + kKeys > sinks;
                uint32_t odd = 0;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if constexpr (!kAhead) fetch_half(tile, now, x);
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < kVEach; ++i)
                            if (kVPieces >= 64 || lane < kVPieces) odd |= take_odd<T>(vr[kAhead ? x : 0][i]);
                    }
                    put_half(x);
                }
                const int n0 = now.rows[0], n1 = now.rows[1];
                const int page0 = now.page[0], page1 = now.page[1];
                if constexpr (kWin)
                    any |= (n0 > 0 && (t0 < sinks || t0 + n0 > least)) || (n1 > 0 && (t0 + 16 < sinks || t0 + 16 + n1 > least));
                else
                    any |= n0 | n1;
                if (tile + kWaves < c_end) {
                    now = next;
                    if constexpr (kAhead) {
                        fetch_half(tile + kWaves, now, 0);
                        fetch_half(tile + kWaves, now, 1);
                    }
                    if (tile + 2 * kWaves < c_end) next = look_up(tile + 2 * kWaves);
                }
                work([&](f32x16& s) __attribute__((always_inline)) {
                    if (edge) {
                        const int from = opaque(least - t0 - 4 * half), sink = opaque(sinks - t0 - 4 * half);
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (outside(8 * (r / 4) + r % 4, from, sink)) s[r] = -INFINITY;
                    }
                    if (n0 + n1 == kKeys) return;
                    const int lo = opaque(n0 - 4 * half), hi = opaque(n1 - 4 * half);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (8 * (r / 4) + r % 4 - (r >= 8 ? 16 : 0) >= (r >= 8 ? hi : lo)) s[r] = -INFINITY;
                });
                if constexpr (kWin) {
                    // (rare) values that are not finite reach the rows that attend them
                    if (__any(odd != 0)) {
                        for (int key = 0; key < kKeys; ++key) {
                            if ((key & 15) >= (key < 16 ? n0 : n1)) continue;
                            const int64_t head = static_cast<int64_t>(key < 16 ? page0 : page1) * a.Hkv + kvh;
                            const T* from = static_cast<const T*>(a.v_cache) + ((head << a.page_shift) + ((t0 + key) & in_page)) * DV;
                            add_odd(from, t0 + key < sinks || t0 + key >= least);
                        }
                    }
                }
            }
        }
        // the drafts: dense rows, a tile or two
        for (; tile < t_end; tile += kWaves) {
            const int t0 = (tile - ctx_tiles) * kKeys;
            const int k_step = kKRow * a.Hkv, v_step = kVRow * a.Hkv;
            const char* kb = static_cast<const char*>(a.k_new) + (static_cast<int64_t>(b) * a.T + t0) * k_step + kvh * kKRow;
            const char* vb = static_cast<const char*>(a.v_new) + (static_cast<int64_t>(b) * a.T + t0) * v_step + kvh * kVRow;
            wave_lds_fence();
            uint32_t odd = 0;
            constexpr int kAtOnce = kAhead ? 2 : 1;
#pragma unroll kAtOnce
            for (int x = 0; x < 2; ++x) {
                const int to = kAhead ? x : 0;
#pragma unroll
                for (int i = 0; i < kKEach; ++i) {
                    const int p = lane + 64 * i, r = 16 * x + p / (kKRow / 16);
                    kr[to][i] = t0 + r < a.T ? *reinterpret_cast<const u32x4*>(kb + static_cast<int64_t>(r) * k_step + p % (kKRow / 16) * 16) : u32x4{};
                }
#pragma unroll
                for (int i = 0; i < kVEach; ++i) {
                    const int p = lane + 64 * i, r = 16 * x + p / (kVRow / 16);
                    vr[to][i] = t0 + r < a.T ? *reinterpret_cast<const u32x4*>(vb + static_cast<int64_t>(r) * v_step + p % (kVRow / 16) * 16) : u32x4{};
                }
                // A value that is not finite must not meet a weight of 0 in a
                // product: rows that do not attend its draft would get NaN.
#pragma unroll
                for (int i = 0; i < kVEach; ++i) odd |= take_odd<T>(vr[to][i]);
                put_half(x);
            }
            const uint32_t bits = static_cast<uint32_t>(seen >> t0);
            any |= bits & ~0u >> max(0, kKeys - (a.T - t0));
            work([&](f32x16& s) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int key = 8 * (r / 4) + 4 * half + r % 4;
                    if (t0 + key >= a.T || (bits >> key & 1) == 0) s[r] = -INFINITY;
                }
            });
            // (rare) such values reach the rows that attend them, as they are
            if (__any(odd != 0)) {
                const T* from = reinterpret_cast<const T*>(vb);
                for (int key = 0; key < kKeys && t0 + key < a.T; ++key, from += a.Hkv * DV) add_odd(from, (bits >> key & 1) != 0);
            }
        }
    }
    l = xor32_add(l);
    if (any != 0 && m == -INFINITY) m = kLowest;

    // join the waves, the upper half of them into the lower, until one is left
    __syncthreads();
    const float sc = a.scale * kLog2e;
    for (int left = kWaves / 2; left >= 1; left /= 2) {
        char* at = smem + (wave % left) * (Sz::kPart + 2 * 64 * 4);
        float* stats = reinterpret_cast<float*>(at + Sz::kPart);
        if (wave >= left && wave < 2 * left) {
#pragma unroll
            for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4)
                    *reinterpret_cast<f32x4*>(at + ((i * 4 + r4) * 64 + lane) * 16) =
                        f32x4{acc[i][4 * r4], acc[i][4 * r4 + 1], acc[i][4 * r4 + 2], acc[i][4 * r4 + 3]};
            stats[lane] = m;
            stats[64 + lane] = l;
        }
        __syncthreads();
        if (wave < left) {
            const float mo = stats[lane], lo = stats[64 + lane];
            const float top = fmaxf(m, mo);
            const float fa = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - top) * sc);
            const float fb = mo == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((mo - top) * sc);
            m = top;
            l = l * fa + lo * fb;
#pragma unroll
            for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const f32x4 o = *reinterpret_cast<const f32x4*>(at + ((i * 4 + r4) * 64 + lane) * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][4 * r4 + e] = acc[i][4 * r4 + e] * fa + o[e] * fb;
                }
        }
        __syncthreads();
    }
    if (wave != 0 || !mine) return;

    if (a.splits > 1) {
        if (!real) return;  // the joining kernel writes padding rows
        const int64_t at = ((static_cast<int64_t>(split) * a.B + b) * a.Hkv + kvh) * rows + row;
        if (half == 0) {
            a.stats[2 * at] = m;
            a.stats[2 * at + 1] = l;
        }
        if (attends(m, l)) {
#pragma unroll
            for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const int ch = 32 * i + 8 * r4 + 4 * half;
                    if (ch < DV)
                        *reinterpret_cast<f32x4*>(a.part + at * DV + ch) =
                            f32x4{acc[i][4 * r4], acc[i][4 * r4 + 1], acc[i][4 * r4 + 2], acc[i][4 * r4 + 3]};
                }
        }
        return;
    }
    const Norm norm = normalise(m, l, sc);
    if (a.lse != nullptr && half == 0) a.lse[q_at] = norm.lse;
    T* out = static_cast<T*>(a.out) + q_at * DV;
    const T* z = a.z != nullptr && real ? static_cast<const T*>(a.z) + q_at * DV : nullptr;
#pragma unroll
    for (int i = 0; i < kVTiles; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int ch = 32 * i + 8 * r4 + 4 * half;
            if (ch >= DV) continue;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = acc[i][4 * r4 + e] * norm.inv;
            store4<T>(out + ch, z != nullptr ? z + ch : nullptr, y);
        }
}

// Joins the parts, kWaves waves to a row: thread s of the row weighs part s,
// then the row's half waves take the parts in turn, four channels a lane, and
// their sums are added in LDS.  Many rows of few parts take a wave each (16,384
// rows of 2 parts: 15 us, with four waves each 29 us; 4,096 of 16: 8 against
// 12); few rows of many parts four (512 rows of 32 parts: 7 us, with one wave
// each 8.3; 128 of 64: 7.3 against 11.5).
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 16;
static_assert(kMaxSplits <= kJoinThreads && kFewParts <= 64, "a thread per part");

template <typename T, int DV, int kWaves>
__global__ __launch_bounds__(kJoinThreads) void attn_tree_join_kernel(TreeK a) {
    constexpr int kRows = 4 / kWaves, kThreads = 64 * kWaves, kTurns = 2 * kWaves;
    __shared__ float weight[kJoinThreads], tops[4], sums[4];
    __shared__ f32x4 added[8][32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, ch = (lane & 31) * 4;
    const int mine = wave / kWaves, tid = threadIdx.x % kThreads, turn = tid >> 5, first = mine * kWaves;
    // a wave's row: below 2^30, so that its divisions are scalar and short
    const int r0 = uniform(static_cast<int>(blockIdx.x) * kRows + mine), total = a.B * a.T * a.H;
    const int64_t r = r0 < total ? r0 : total - 1;
    const int G = a.H / a.Hkv, rows = a.T * G;
    const int token = static_cast<int>(r) / a.H, h = static_cast<int>(r) - token * a.H, b = token / a.T, t = token - b * a.T;
    const int64_t at = (static_cast<int64_t>(b) * a.Hkv + h / G) * rows + t * G + h % G;
    const int64_t step = static_cast<int64_t>(a.B) * a.Hkv * rows;
    int slot, ctx;
    const bool real = slot_of(a, b, slot, ctx);
    const float sc = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    if (real && tid < a.splits) {
        m = a.stats[2 * (at + tid * step)];
        l = a.stats[2 * (at + tid * step) + 1];
    }
    float top = m;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[first + w]);
    // No part was written where nothing is attended: its weight is below 0.
    // Every other part is added, also with a weight of 0, so that a value that
    // is not finite reaches the row as it does in one piece.
    const bool there = attends(m, l);
    const float f = there ? __builtin_amdgcn_exp2f((m - top) * sc) : 0.f;
    weight[threadIdx.x] = there ? f : -1.f;
    l = wave_sum(l * f);
    if (lane == 0) sums[wave] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) l += sums[first + w];
    f32x4 y{};
    if (ch < DV) {
        constexpr int kEach = 4;  // parts in flight
        for (int s0 = turn; s0 < a.splits; s0 += kTurns * kEach) {
            f32x4 o[kEach];
            float w[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int s = s0 + kTurns * i;
                w[i] = s < a.splits ? weight[mine * kThreads + s] : -1.f;
                o[i] = !(w[i] < 0.f) ? *reinterpret_cast<const f32x4*>(a.part + (at + s * step) * DV + ch) : f32x4{};
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += o[i][e] * w[i];
        }
    }
    added[mine * kTurns + turn][lane & 31] = y;
    __syncthreads();
    if (turn != 0 || r0 >= total) return;
#pragma unroll
    for (int p = 1; p < kTurns; ++p) {
        const f32x4 o = added[mine * kTurns + p][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += o[e];
    }
    const Norm norm = normalise(top, l, sc);
    float out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = y[e] * norm.inv;
    if (a.lse != nullptr && lane == 0) a.lse[r] = norm.lse;
    if (ch < DV)
        store4<T>(static_cast<T*>(a.out) + r * DV + ch,
                  a.z != nullptr && real ? static_cast<const T*>(a.z) + r * DV + ch : nullptr, out);
}

// Row blocks and parts of a call.
struct TreePlan {
    int blocks, splits;
};
constexpr int kWantUnits = 1024, kWantUnitsOfOne = 512;  // workgroups below which a call is split

// The tokens of a cache that a windowed row can read, of a context of at most
// max_ctx: what the parts of a call go by.
int64_t window_reach(int64_t max_ctx, int window, int sinks) {
    const int64_t reach = static_cast<int64_t>(window) + sinks + 64;  // a tile at the window's start and at the sinks' end
    return window > 0 && reach < max_ctx ? reach : max_ctx;
}

// even: the sequences read equally much.
TreePlan tree_plan(int B, int T, int H, int Hkv, int64_t max_ctx, bool even) {
    const int64_t rows = static_cast<int64_t>(T) * (H / Hkv);
    TreePlan p;
    p.blocks = static_cast<int>((rows + 31) / 32);
    const int64_t units = static_cast<int64_t>(B) * Hkv * p.blocks;
    const int64_t tiles = (max_ctx + kKeys - 1) / kKeys + (T + kKeys - 1) / kKeys;
    // Of bf16 at up to 128 channels two workgroups fit a CU.  The parts of one
    // sequence are equally long: one round of them (262,144 tokens: 193 us and
    // 8 us to join them, against 198 and 9 us in two rounds).  Sequences differ,
    // and two rounds let the short ones fill up behind the long (64 of up to
    // 8,000 tokens: 219 us against 239 us in one).  The other forms fit a CU
    // once and take the same numbers, in twice the rounds: 32 sequences of up
    // to 8,000 tokens 366 us in fp32 at 192 channels and 119 in bf16, with half
    // as many parts 433 and 124; one of 100,000 tokens 289 and 100, with half
    // as many 284 and 96.
    // A window shorter than the contexts evens them out: one round (32 trees of
    // 16 under a window of 2,000, 75 us in two rounds with their join, 61 in one
    // without; fp32 270 against 243 us; a window of 7,000 of at most 8,000 tokens
    // 134 against 130).
    const int64_t want = B == 1 || even ? kWantUnitsOfOne : kWantUnits;
    int64_t s = (want + units - 1) / units;
    if (s > tiles / 8) s = tiles / 8;  // two tiles a wave at least
    p.splits = static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    return p;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename T, int DK, int DV, bool kWin>
hipError_t launch_tree(const TreeArgs& a, hipStream_t s) {
    const int64_t max_ctx = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int64_t reach = window_reach(max_ctx, a.window, a.sinks);
    const TreePlan p = tree_plan(a.B, a.T, a.H, a.Hkv, reach, reach < max_ctx);
    const size_t parts = static_cast<size_t>(p.splits) * a.B * a.T * a.H;
    float* part = static_cast<float*>(a.ws);
    float* stats = reinterpret_cast<float*>(static_cast<char*>(a.ws) + up256(parts * DV * 4));
    const TreeK k{a.B, a.T, a.H, a.Hkv, a.scale, a.q, a.k_new, a.v_new, a.z, a.mask, a.k_cache, a.v_cache,
                  a.pages, a.page_shift, a.table, a.slots, a.max_pages, a.lens, a.slot_indices, a.out, a.lse,
                  part, stats, p.splits, p.blocks, a.B * a.Hkv * p.splits, a.window, a.sinks};
    using Sz = TreeSizes<T, DK, DV>;
    static_assert(Sz::kLds <= 160 * 1024, "one workgroup's LDS");
    auto fn = attn_tree_kernel<T, DK, DV, kWin>;
    if (Sz::kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, Sz::kLds);
        if (e != hipSuccess) return e;
    }
    {
        LaunchTimer timer(kWin ? "attn_window_tree" : "attn_tree", s);
        const int64_t groups = static_cast<int64_t>((k.units + 7) / 8) * 8 * k.blocks;
        fn<<<dim3(static_cast<unsigned>(groups)), dim3(64 * Sz::kWaves), Sz::kLds, s>>>(k);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    LaunchTimer timer("attn_tree_join", s);
    const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.H;
    if (p.splits <= kFewParts)
        attn_tree_join_kernel<T, DV, 1><<<dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(kJoinThreads), 0, s>>>(k);
    else
        attn_tree_join_kernel<T, DV, 4><<<dim3(static_cast<unsigned>(rows)), dim3(kJoinThreads), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

namespace {
size_t parts_bytes(const TreePlan& p, int B, int T, int H, int dv) {
    if (p.splits == 1) return 0;
    const size_t parts = static_cast<size_t>(p.splits) * B * T * H;
    return up256(parts * dv * 4) + up256(parts * 8);
}
}  // namespace

size_t attn_tree_workspace_bytes(int B, int T, int H, int Hkv, int dv, int64_t max_ctx, int window, int sinks) {
    if (B == 0 || T == 0) return 0;
    const int64_t reach = window_reach(max_ctx, window, sinks);
    return parts_bytes(tree_plan(B, T, H, Hkv, reach, reach < max_ctx), B, T, H, dv);
}

// More sequences or tokens have fewer parts of more rows, so what a call needs
// does not rise with its sizes: all that are split are tried.  Nor with its
// contexts under a window: those no longer than it are cut into more parts.
size_t attn_tree_max_workspace_bytes(int B, int T, int H, int Hkv, int dv, int64_t max_ctx, int window, int sinks) {
    const int64_t reach = window_reach(max_ctx, window, sinks);
    size_t most = 0;
    for (int t = 1; t <= T; ++t) {
        const int64_t units = static_cast<int64_t>(Hkv) * ((static_cast<int64_t>(t) * (H / Hkv) + 31) / 32);  // of a sequence
        for (int b = 1; b <= B && b * units < kWantUnits; ++b) {
            const size_t need = parts_bytes(tree_plan(b, t, H, Hkv, reach, false), b, t, H, dv);
            most = need > most ? need : most;
        }
    }
    return most;
}

hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t s) {
    if (a.B == 0 || a.T == 0) return hipSuccess;
    return attn_dispatch(a.x, a.dk, a.dv, [&](auto t, auto dk, auto dv) {
        using X = typename decltype(t)::type;
        constexpr int kDk = decltype(dk)::value, kDv = decltype(dv)::value;
        return a.window > 0 ? launch_tree<X, kDk, kDv, true>(a, s) : launch_tree<X, kDk, kDv, false>(a, s);
    });
}

}  // namespace kda
