// The attention weights that a sequence's last tokens give to its cached
// tokens, summed per cached token.
//
//   w_j += sum over queries i and heads h of e^(s_ijh - lse_ih),
//   s_ijh = scale q_ih . k_j(h / G), over the keys j that query i attends
//
// lse is what the attention call gave, so the weights need no statistics of
// their own: one pass over the keys, no values.
//
// Two kernels: one for few queries a sequence (a decode step, accepted drafts),
// one for many (the last tokens of prompts, whole prompts).  Either is right for
// any number; the host chooses by the average, as only the device knows a
// sequence's own.
//
// bf16, 32 heads of 128 over 8: a decode step's 256 queries over 1,024 to 4,096
// tokens each read 1.33 GB in 244 us (5.5 TB/s); all of a prompt of 8,000 tokens
// 306 to 325 us by the card (810 to 860 TFLOP/s of the 1,390 that a large product
// reaches; floor 189), the last 64 tokens of 8 prompts 50 us (floor 14).
#include "kda_attn_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32;  // rows of a product: queries of a head, or queries and heads of a group

struct WeighK {
    CacheArgs c;
    WeighArgs a;
    int groups;      // workgroups of a sequence
    float* part;     // [N, groups][keys of a tile]
};

// Sequence n's queries and its slot's tokens; false: nothing to do.
struct Weighed {
    int64_t first;  // its first query's index
    int count, slot, ctx;
    int p_first;    // the first query's place; below 0: it has no token
};
__device__ __forceinline__ bool weighed(const WeighK& k, int n, Weighed& w) {
    seq_bounds(k.a.cu, n, k.a.tokens, w.first, w.count);
    w.count = uniform(w.count);
    w.first = uniform64(w.first);
    const int slot = k.a.slot_indices != nullptr ? k.a.slot_indices[n] : n;
    w.slot = uniform(slot);
    if (w.count == 0 || slot < 0 || slot >= k.c.slots || k.a.src_rows == 0) return false;
    const int64_t most = static_cast<int64_t>(k.c.max_pages) << k.c.page_shift;
    const int len = k.c.lens[slot];
    w.ctx = uniform(len < 0 ? 0 : static_cast<int>(len > most ? most : len));
    w.p_first = w.ctx - w.count;
    return w.ctx > 0;
}

// The tiles of `keys` keys that some query attends, in order (the n-th begins at
// key first(n)): those of the first tokens and those from the first query's
// window on.
struct Tiles {
    int keys, sinks, sink_tiles, skip, count;
    __device__ __forceinline__ Tiles(const WeighArgs& a, const Weighed& w, int keys_) : keys(keys_) {
        const int low = a.window > 0 ? max(0, w.p_first - a.window + 1) : 0;
        sinks = a.window > 0 ? min(a.sinks, w.ctx) : 0;
        sink_tiles = (sinks + keys - 1) / keys;
        skip = max(0, low / keys - sink_tiles);
        count = (w.ctx + keys - 1) / keys - skip;
    }
    __device__ __forceinline__ int first(int n) const { return (n >= sink_tiles ? n + skip : n) * keys; }
};

// The row of place `pos` in head 0 of the pool, and whether it holds a token.
__device__ __forceinline__ int64_t row_of(const WeighK& k, const Weighed& w, int pos, bool& there) {
    const CacheArgs& c = k.c;
    const int page = pos < w.ctx ? c.table[static_cast<int64_t>(w.slot) * c.max_pages + (pos >> c.page_shift)] : -1;
    there = page >= 0 && page < c.pages;
    return ((static_cast<int64_t>(there ? page : 0) * c.Hkv) << c.page_shift) + (there ? pos & ((1 << c.page_shift) - 1) : 0);
}

__device__ __forceinline__ float* weight_of(const WeighK& k, const Weighed& w, int pos) {
    return k.a.weights + ((static_cast<int64_t>(w.slot) * k.c.max_pages) << k.c.page_shift) + pos;
}

// What a key gathers: weights, or sums of one head's, that are NaN or infinite come
// from that head's key not being finite.  A row that attends such a key has an lse
// that is not finite (and weighs nothing) or no weight there, unless its lse is of
// a window that the key is not in.  Where many queries are, whose broken rows read
// as 0, it is taken for a step of one head, so that the others' stay.
__device__ __forceinline__ float gathered(float x) { return x < INFINITY ? x : 0.f; }

template <typename T, int DK>
struct FewSizes {
    static constexpr int kKeys = 32;  // of a tile
    static constexpr int kTile = kKeys * DK * static_cast<int>(sizeof(T));
    static constexpr int kRow = DK * static_cast<int>(sizeof(T));
    static constexpr int kQueries = 16384 / kRow > kRows ? 16384 / kRow : kRows;  // rows of queries that LDS holds
    static constexpr int kSums = kWaves * kTile, kQ = kSums + kWaves * kKeys * 4, kLse = kQ + kQueries * kRow;
    static constexpr int kLds = kLse + kQueries * 4;
};

// Few queries: bound by reading the keys.  Scores transposed (S^T = K Q^T, 32
// keys by the group's rows), a lane's row and its lse the same for every tile,
// its 16 sums added over the lanes once per tile.  A wave takes its own tiles,
// all heads of one after another (or shares a tile's heads with the others of
// its workgroup, where there are few tiles).  Keys are read by whole rows, the
// next head's in flight while one is worked on, and laid out in LDS for the
// product.  So are the queries, of as many heads as fit, once for all tiles (read
// from the caches for every tile and head they took more of the L1 than the
// keys: a decode step of 256 sequences 259 us).
template <typename T, int DK>
__global__ __launch_bounds__(kThreads, (DK * sizeof(T) <= 256 ? 3 : 1)) void cache_weigh_few_kernel(WeighK k) {
    extern __shared__ __align__(16) char smem[];
    using Sz = FewSizes<T, DK>;
    constexpr int kKeys = Sz::kKeys;
    constexpr int kPieces = DK / (2 * Elem<T>::kPer16);
    constexpr int kRow = DK * static_cast<int>(sizeof(T)), kRowPieces = kRow / 16;
    constexpr int kHalf = 16 * kRowPieces, kEach = (kHalf + 63) / 64;  // 16-byte pieces of 16 rows, of a lane
    const CacheArgs& c = k.c;
    const WeighArgs& a = k.a;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    char* sK = smem + wave * Sz::kTile;
    float(*sums)[kKeys] = reinterpret_cast<float(*)[kKeys]>(smem + Sz::kSums);
    char* sQ = smem + Sz::kQ;
    float* sLse = reinterpret_cast<float*>(smem + Sz::kLse);
    const int n = blockIdx.x / k.groups, group = blockIdx.x % k.groups;
    Weighed w;
    if (!weighed(k, n, w)) return;
    const int G = a.H / c.Hkv;
    const Tiles tiles(a, w, kKeys);
    const float sc = a.scale * kLog2e;
    // Where there are few tiles, waves share one and take equal runs of its heads.
    const int64_t all = static_cast<int64_t>(tiles.count) * a.N;
    const int share = all >= 4096 || c.Hkv < 2 ? 1 : all >= 2048 || c.Hkv < 4 ? 2 : 4;
    const int member = wave % share, team = wave / share, teams = kWaves / share;
    // every wave of a workgroup takes as many turns (they meet where they share)
    const int stride = k.groups * teams;
    const int turns = (tiles.count - group * teams + stride - 1) / stride;
    if (turns <= 0) return;

    // 32 rows at a time: all of them in the calls that this kernel is for
    const int64_t rows = static_cast<int64_t>(w.count) * G;
    for (int64_t r0 = 0; r0 < rows; r0 += kRows) {
        // this lane's row: a query and a head of the group
        const int64_t r = min(r0 + col, rows - 1);
        const int64_t t = w.first + r / G, src = a.rows != nullptr ? a.rows[t] : t;
        const int p_here = max(w.p_first + static_cast<int>(r / G), -1);
        const bool on = r0 + col < rows && p_here >= 0 && src >= 0 && src < a.src_rows;

        // A tile's halves of 16 rows, each in one page
        typedef const __attribute__((address_space(4))) int32_t* scalar_ints;
        const scalar_ints entries = (scalar_ints)(c.table + static_cast<int64_t>(w.slot) * c.max_pages);
        struct Place {
            int page[2], rows[2];  // rows that hold a token
        };
        auto look = [&](int tile) __attribute__((always_inline)) {
            Place x;
            const int first = tile < tiles.count ? tiles.first(tile) : w.ctx;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = first + 16 * h;
                const int page = entries[min(p, w.ctx - 1) >> c.page_shift];
                const bool there = page >= 0 && page < c.pages;
                x.rows[h] = there ? min(16, max(0, w.ctx - p)) : 0;
                x.page[h] = there ? page : 0;
            }
            return x;
        };
        u32x4 kr[2][kEach];
        const int here_rows = static_cast<int>(min<int64_t>(kRows, rows - r0)), my_row = min(col, here_rows - 1);
        TileRead<T, DK> rq;
        rq.init_rows(my_row, half);
        const int mask = (1 << c.page_shift) - 1;
        auto load_k = [&](const Place& x, int tile, int f) __attribute__((always_inline)) {
            const int first = tile < tiles.count ? tiles.first(tile) : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t row = ((static_cast<int64_t>(x.page[h]) * c.Hkv + min(f, c.Hkv - 1)) << c.page_shift) + ((first + 16 * h) & mask);
                const auto from = rows_of(c.k_cache, row, kRow, x.rows[h]);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (kHalf >= 64 || lane < kHalf) kr[h][i] = buffer_load16(from, (lane + 64 * i) * 16);
            }
        };
        TileRead<T, DK> rk;
        rk.init_rows(col, half);
        auto put = [&]() __attribute__((always_inline)) {
            wave_lds_fence();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int p = lane + 64 * i, row = 16 * h + p / kRowPieces;
                    if (kHalf >= 64 || lane < kHalf)
                        *reinterpret_cast<u32x4*>(sK + row * kRow + (p % kRowPieces ^ turn<kRowPieces>(row)) * 16) = kr[h][i];
                }
            wave_lds_fence();
        };
        f32x16 acc{};
        auto work = [&](int f, int first) __attribute__((always_inline)) {  // f: the head's place among those in LDS
            f32x16 s{};
            const char* at = sQ + f * here_rows * kRow;
            const float lse = sLse[f * here_rows + my_row];
#pragma unroll
            for (int p = 0; p < kPieces; ++p) s = mma<T>(rk.rows(sK, p), rq.rows(at, p), s);
            const bool good = on && fabsf(lse) < INFINITY;  // a row that attends nothing, or a broken one, weighs nothing
            const float lse2 = good ? lse * kLog2e : INFINITY;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = gathered(__builtin_amdgcn_exp2f(fmaf(s[i], sc, -lse2)));
            if (first + kKeys - 1 > w.p_first || (a.window > 0 && first < w.ctx - a.window && first + kKeys > tiles.sinks)) {
                const int most = opaque(p_here - first - 4 * half);
                const int least = opaque(a.window > 0 ? p_here - a.window + 1 - first - 4 * half : INT32_MIN / 2);
                const int sink = opaque(tiles.sinks - first - 4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = 8 * (i / 4) + i % 4;
                    if (key > most || outside(key, least, sink)) s[i] = 0.f;
                }
            }
            acc += s;
        };
        // the place that this lane writes when a tile is done, and what stands there
        auto mine = [&](const Place& x) { return member == 0 && half == 0 && (col & 15) < (col < 16 ? x.rows[0] : x.rows[1]); };
        auto finish = [&](int first, const Place& x, float had) __attribute__((always_inline)) {
            // over the lanes of a half; key 8 (i / 4) + 4 half + i % 4
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = row_ror_add<1>(acc[i]);
                v = row_ror_add<2>(v);
                v = row_ror_add<4>(v);
                v = xor16_add(row_ror_add<8>(v));
                if (col == 0) sums[wave][8 * (i / 4) + 4 * half + i % 4] = v;
            }
            acc = f32x16{};
            if (share > 1) __syncthreads();
            else wave_lds_fence();
            if (mine(x)) {
                float v = 0.f;
                for (int m = 0; m < share; ++m) v += sums[wave + m][col];
                *weight_of(k, w, first + col) = had + v;
            }
            if (share > 1) __syncthreads();
            else wave_lds_fence();
        };
        const int at_once = Sz::kQueries / here_rows;  // heads whose queries LDS holds
        for (int g0 = 0; g0 < c.Hkv; g0 += at_once) {
            const int heads = min(at_once, c.Hkv - g0);
            __syncthreads();  // (the queries before these are done with)
            for (int x = threadIdx.x; x < here_rows * heads * kRowPieces; x += kThreads) {
                const int piece = x % kRowPieces, to = x / kRowPieces, row = to % here_rows, f = g0 + to / here_rows;
                const int64_t ri = r0 + row, ti = w.first + ri / G, si = a.rows != nullptr ? a.rows[ti] : ti;
                const int64_t from = (si >= 0 && si < a.src_rows ? si : 0) * a.H + f * G + ri % G;
                *reinterpret_cast<u32x4*>(sQ + to * kRow + (piece ^ turn<kRowPieces>(row)) * 16) =
                    *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + from * kRow + piece * 16);
                if (piece == 0) sLse[to] = a.lse[from];
            }
            __syncthreads();
            const int f0 = g0 + heads * member / share, f1 = g0 + heads * (member + 1) / share;
            int tile = group * teams + team;
            Place here = look(tile), next = look(tile + stride);
            load_k(here, tile, f0);
            for (int turn = 0; turn < turns; ++turn) {
                const int first = tile < tiles.count ? tiles.first(tile) : 0;
                const float had = mine(here) ? *weight_of(k, w, first + col) : 0.f;
                for (int f = f0; f < f1; ++f) {
                    put();
                    if (f + 1 < f1) load_k(here, tile, f + 1);
                    else load_k(next, tile + stride, f0);
                    work(f - g0, first);
                }
                finish(first, here, had);
                tile += stride;
                here = next;
                if (turn + 2 < turns) next = look(tile + stride);
            }
        }
    }
}

constexpr int kMostParts = 64;

// How a sequence's tiles go to its workgroups: a tile each in turn, or, where
// there are fewer tiles, several to a tile, that take equal parts of its work.
struct Shares {
    int parts;
    __device__ __forceinline__ Shares(const WeighK& k, int tiles)
        : parts(tiles >= k.groups ? 1 : min(k.groups / max(tiles, 1), kMostParts)) {}
};

template <typename T, int DK>
struct ManySizes {
    static constexpr int kSub = sizeof(T) == 2 ? 2 : 1;  // blocks of 32 keys of a wave, in its registers
    static constexpr int kKeys = kWaves * 32 * kSub;
    static constexpr int kTile = kRows * DK * static_cast<int>(sizeof(T));
    static constexpr int kBuf = kTile + kRows * 4;  // rows of queries and their lse
};

// Many queries: bound by the products and exponentials (8,000 tokens: matrix cores
// 34 % of the cycles, vector units 46 %, waits 24 %; a wave's step of 64 keys by 32
// queries has 16 products of 32 cycles and 32 exponentials of 8, each with a
// multiply-add and an addition of 4).  One workgroup per
// (sequence, tile of keys, part): a wave's keys stay in its registers, the
// queries of a head pass through LDS, once for four waves, two steps in flight
// (a step is shorter than a load takes).  S = Q K^T, so that a lane holds one
// key's scores and one sum.  The tile's work is the sequence of its steps, head
// by head.
// kPicked: the queries' rows are named by a list (64 of each of 8 prompts: 59 us).
template <typename T, int DK, bool kPicked>
__global__ __launch_bounds__(kThreads, (DK * sizeof(T) <= 256 ? 2 : 1)) void cache_weigh_many_kernel(WeighK k) {
    __shared__ __align__(16) char smem[2 * ManySizes<T, DK>::kBuf];
    using Sz = ManySizes<T, DK>;
    constexpr int kSub = Sz::kSub, kKeys = Sz::kKeys;
    constexpr int kPieces = DK / (2 * Elem<T>::kPer16);
    constexpr int kRow = DK * static_cast<int>(sizeof(T)), kRowPieces = kRow / 16;
    constexpr int kPiecesOfStep = kRows * kRowPieces, kEach = (kPiecesOfStep + kThreads - 1) / kThreads;
    constexpr bool kFull = kPiecesOfStep % kThreads == 0;
    const CacheArgs& c = k.c;
    const WeighArgs& a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int n = blockIdx.x / k.groups, group = blockIdx.x % k.groups;
    Weighed w;
    if (!weighed(k, n, w)) return;
    const int G = a.H / c.Hkv;
    const Tiles tiles(a, w, kKeys);
    const int parts = Shares(k, tiles.count).parts, part = group % parts;
    // this thread's pieces of a step: where they come from and go to
    const int q_row = a.H * kRow;
    int row_in[kEach], piece_in[kEach], put_at[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = tid + i * kThreads;
        row_in[i] = p / kRowPieces;
        piece_in[i] = p % kRowPieces;
        put_at[i] = row_in[i] * kRow + (piece_in[i] ^ turn<kRowPieces>(row_in[i])) * 16;
    }
    for (int tile = group / parts; tile < tiles.count; tile += k.groups / parts) {
        const int k_first = tiles.first(tile), k0 = k_first + wave * 32 * kSub;
        // the queries that attend some key of the tile
        const int i_low = max(0, k_first - w.p_first);
        int i_end = w.count;
        if (a.window > 0 && k_first >= tiles.sinks) i_end = static_cast<int>(min<int64_t>(i_end, static_cast<int64_t>(k_first) + kKeys - 1 + a.window - w.p_first));
        const int steps = max(0, (i_end - i_low + kRows - 1) / kRows);
        const int64_t all = static_cast<int64_t>(steps) * a.H;
        int64_t s_now = all * part / parts;
        const int64_t s_end = all * (part + 1) / parts;

        int64_t at[kSub];
        bool there[kSub];
        u32x4 key[kSub][kPieces];
        float acc[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            at[u] = row_of(k, w, k0 + 32 * u + col, there[u]);
            acc[u] = 0.f;
        }
        const float sc = a.scale * kLog2e;
        TileRead<T, DK> rq;
        rq.init_rows(col, half);

        // the step to fetch, and the one worked on
        int f_head = uniform(s_now < s_end ? static_cast<int>(s_now / steps) : 0);
        int f_i = uniform(i_low + (s_now < s_end ? static_cast<int>(s_now % steps) * kRows : 0));
        int head = f_head, i0 = f_i, kvh = -1;
        struct Step {
            u32x4 q[kEach];
            float of[kEach], lse;  // the lse of the pieces' rows, and of row `col`
            bool there;            // row `col` is one
            uint32_t named;        // of the pieces' rows, a bit each
        };
        // (behind the last step it reads nothing, but in no branch: a wait for the
        // step before would be one for this one too)
        int64_t s_fetch = s_now;
        auto fetch = [&](Step& x) __attribute__((always_inline)) {
            const int here = s_fetch < s_end ? min(kRows, i_end - f_i) : 0;
            ++s_fetch;
            if constexpr (!kPicked) {  // what is behind the last row reads as 0
                const auto q = rows_of(static_cast<const T*>(a.q) + f_head * DK, w.first + f_i, q_row, here);
                const auto l = rows_of(a.lse + f_head, w.first + f_i, a.H * 4, here);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (kFull || tid + i * kThreads < kPiecesOfStep) {
                        x.q[i] = buffer_load16(q, row_in[i] * q_row + piece_in[i] * 16);
                        x.of[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(l, row_in[i] * a.H * 4, 0, 0));
                    }
                x.lse = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(l, col * a.H * 4, 0, 0));
                x.there = col < here;
                x.named = ~0u;
            } else {
                // query i's row in q and lse; the tensor's first one for none, which is not to be looked at
                auto row_at = [&](int i, bool& named) {
                    const int64_t r = i < here ? a.rows[w.first + f_i + i] : -1;
                    named = r >= 0 && r < a.src_rows;
                    return (named ? r : 0) * a.H + min(f_head, a.H - 1);
                };
                x.named = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (kFull || tid + i * kThreads < kPiecesOfStep) {
                        bool named;
                        const int64_t r = row_at(row_in[i], named);
                        x.named |= static_cast<uint32_t>(named) << i;
                        x.q[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + r * kRow + piece_in[i] * 16);
                        x.of[i] = a.lse[r];
                    }
                const int64_t r = col < here ? a.rows[w.first + f_i + col] : -1;
                x.there = r >= 0 && r < a.src_rows;
                x.lse = a.lse[(x.there ? r : 0) * a.H + min(f_head, a.H - 1)];
            }
            f_i += kRows;
            if (f_i >= i_low + steps * kRows) {
                f_i = i_low;
                ++f_head;
            }
        };
        // A row that is not there, attends nothing or is broken: e^(0 - infinity).
        auto put = [&](char* buf, const Step& x) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (kFull || tid + i * kThreads < kPiecesOfStep)
                    *reinterpret_cast<u32x4*>(buf + put_at[i]) = (x.named >> i & 1) != 0 && fabsf(x.of[i]) < INFINITY ? x.q[i] : u32x4{};
            if (tid < kRows) reinterpret_cast<float*>(buf + Sz::kTile)[col] = x.there && fabsf(x.lse) < INFINITY ? x.lse * kLog2e : INFINITY;
        };
        auto work = [&](const char* sQ) __attribute__((always_inline)) {
            const f32x4* lse2 = reinterpret_cast<const f32x4*>(sQ + Sz::kTile);
            const int f = head / G, p0 = w.p_first + i0;  // the first row's place
            i0 += kRows;
            if (i0 >= i_low + steps * kRows) {
                i0 = i_low;
                ++head;
            }
            if (f != kvh) {
                kvh = uniform(f);
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const char* from = static_cast<const char*>(c.k_cache) + (at[u] + (static_cast<int64_t>(kvh) << c.page_shift)) * kRow + half * 16;
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) key[u][p] = *reinterpret_cast<const u32x4*>(from + p * 32);
                }
                // waited for here: at their use, every step would wait for the queries in flight
#pragma unroll
                for (int u = 0; u < kSub; ++u) arrive(key[u]);
            }
            if (p0 + kRows <= k0) return;  // queries before this wave's keys
            // one half's products, then the other's, then all exponentials without a branch between:
            // the first half's run beside the other half's products (8,000 tokens 331 to 315 us)
            f32x16 s[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) s[u] = f32x16{};
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int p = 0; p < kPieces; ++p) s[u] = mma<T>(rq.rows(sQ, p), key[u][p], s[u]);
            f32x4 l4[4];
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) l4[r4] = lse2[2 * r4 + half];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], sc, -l4[r / 4][r % 4]));
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const int key0 = k0 + 32 * u;
                // register r: the query at place p0 + 8 (r / 4) + 4 half + r % 4; key key0 + col
                if (p0 < key0 + 31 || (a.window > 0 && p0 + kRows > key0 + a.window && key0 + 32 > tiles.sinks)) {
                    const int least = opaque(key0 + col - p0 - 4 * half);
                    const int most = opaque(a.window > 0 && key0 + col >= tiles.sinks ? key0 + col + a.window - p0 - 4 * half : INT32_MAX);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (8 * (r / 4) + r % 4 < least || 8 * (r / 4) + r % 4 >= most) s[u][r] = 0.f;
                }
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += s[u][r];
                acc[u] += gathered(sum);
            }
        };
        Step x, y;
        fetch(x);
        fetch(y);
        put(smem, x);
        for (; s_now < s_end; s_now += 2) {
            tile_barrier();
            fetch(x);
            work(smem);
            if (s_now + 1 >= s_end) break;
            put(smem + Sz::kBuf, y);
            tile_barrier();
            fetch(y);
            work(smem + Sz::kBuf);
            put(smem, x);
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            const float x = xor32_add(acc[u]);
            if (half != 0) continue;
            if (parts > 1)
                k.part[(static_cast<int64_t>(n) * k.groups + group) * kKeys + wave * 32 * kSub + 32 * u + col] = x;
            else if (there[u])
                *weight_of(k, w, k0 + 32 * u + col) += x;
        }
        tile_barrier();  // the next tile's first queries go where this one's were
    }
}

// Adds the parts in their order, a key per thread.
template <int kKeys>
__global__ __launch_bounds__(kKeys) void cache_weigh_sum_kernel(WeighK k) {
    const int n = blockIdx.x / k.groups, tile = blockIdx.x % k.groups;
    Weighed w;
    if (!weighed(k, n, w)) return;
    const Tiles tiles(k.a, w, kKeys);
    const int parts = Shares(k, tiles.count).parts;
    if (parts == 1 || tile >= tiles.count) return;
    const int pos = tiles.first(tile) + threadIdx.x;
    bool there;
    row_of(k, w, pos, there);
    const float* from = k.part + (static_cast<int64_t>(n) * k.groups + tile * parts) * kKeys + threadIdx.x;
    float sum = 0.f;
    constexpr int kEach = 8;  // in flight (one after the other, up to 64 of them, 11 us)
    for (int p0 = 0; p0 < parts; p0 += kEach) {
        float x[kEach];
#pragma unroll
        for (int p = 0; p < kEach; ++p) x[p] = p0 + p < parts ? from[(p0 + p) * kKeys] : 0.f;
#pragma unroll
        for (int p = 0; p < kEach; ++p) sum += x[p];
    }
    if (!there) return;
    *weight_of(k, w, pos) += sum;
}

// Workgroups of a call.  The host knows how many tiles a table row can hold, not
// how many there are: workgroups without work cost, where few fit a CU, most of a
// short call (43 fp32 sequences of up to 20 tokens, 32 heads of 128: 215 us with
// 4,096 of them, 35 with one per tile of the table).
// Few queries: three workgroups a CU up to 50 KB of LDS (a decode step of 256
// sequences 263 us by events, with 2,048 workgroups 270); else one or two (the
// step in fp32 692 us, with 4,096 workgroups 775).
// Many queries: a prompt of 8,000 tokens 392 us by events, with 512 workgroups 607
// (the tiles differ), with 2,048 the last 64 tokens of 8 prompts 61 us for 56.
// Parts of a tile: 8,000 tokens of 4 heads 59 us, with a part per head 222.
constexpr int kFewWant = 4096, kFewWantWide = 1024, kManyWant = 1024;

// of a sequence that has work for `most` at most
int per_sequence(int64_t want, int64_t N, int64_t most) {
    const int64_t p = (want + N - 1) / N;
    return static_cast<int>(p < most ? p : most < 1 ? 1 : most);
}

// Few queries: their rows of one key head are 32 on the average at most.  A batch
// that holds both kinds is right either way and slow: 300 decode steps over 2,000
// tokens beside 2,000 queries of a prompt (32 heads of 128 over 8) take 10.4 ms, as
// the prompt's keys are read again for every 32 of its rows by the few workgroups
// of a sequence; 255 steps with it, 2.9 ms, 32 rows of product for one query of
// each step.  The two kinds in a call each: 0.28 and 0.23 ms.
bool few_queries(int64_t tokens, int64_t N, int G) { return tokens * G <= kRows * N; }

template <typename T, int DK>
hipError_t launch_weigh(const CacheArgs& c, const WeighArgs& a, hipStream_t s) {
    const int64_t max_ctx = static_cast<int64_t>(c.max_pages) << c.page_shift;
    auto tiles_of = [&](int keys) { return (max_ctx + keys - 1) / keys; };
    WeighK k{};
    k.c = c;
    k.a = a;
    if (a.window >= max_ctx) k.a.window = 0;  // it holds every token
    if (few_queries(a.tokens, a.N, a.H / c.Hkv)) {
        constexpr int lds = FewSizes<T, DK>::kLds;
        k.groups = per_sequence(3 * lds > 160 * 1024 ? kFewWantWide : kFewWant, a.N, tiles_of(FewSizes<T, DK>::kKeys));
        auto fn = cache_weigh_few_kernel<T, DK>;
        if (lds > 64 * 1024) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        LaunchTimer timer("cache_weigh_few", s);
        fn<<<dim3(static_cast<unsigned>(static_cast<int64_t>(a.N) * k.groups)), dim3(kThreads), lds, s>>>(k);
        return hipGetLastError();
    }
    constexpr int kKeys = ManySizes<T, DK>::kKeys;
    k.groups = per_sequence(kManyWant, a.N, kMostParts * tiles_of(kKeys));
    k.part = static_cast<float*>(a.ws);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.N) * k.groups));
    {
        LaunchTimer timer("cache_weigh_many", s);
        if (a.rows != nullptr) cache_weigh_many_kernel<T, DK, true><<<grid, dim3(kThreads), 0, s>>>(k);
        else cache_weigh_many_kernel<T, DK, false><<<grid, dim3(kThreads), 0, s>>>(k);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || k.groups == 1) return e;
    LaunchTimer timer("cache_weigh_sum", s);
    cache_weigh_sum_kernel<kKeys><<<grid, dim3(kKeys), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

size_t cache_weigh_workspace_bytes(int64_t tokens, int N, int H, int Hkv) {
    if (few_queries(tokens, N, H / Hkv)) return 0;
    return static_cast<size_t>(N) * per_sequence(kManyWant, N, kManyWant) * 256 * 4;  // a tile has 256 keys at most
}

hipError_t launch_cache_weigh(const CacheArgs& c, const WeighArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return attn_dispatch(c.x, c.dk, c.dk == 192 ? 128 : c.dk, [&](auto t, auto dk, auto) {
        return launch_weigh<typename decltype(t)::type, decltype(dk)::value>(c, a, s);
    });
}

}  // namespace kda
