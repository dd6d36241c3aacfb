// Gradients of the causal attention of kda_attn_prefill.hip.
//
// With do = dy * sigmoid(z), delta_i = sum_c dy_ic y_ic (= do_i . o_i) and
// P_ij = e^(s_ij - lse_i):
//   dv_j = sum_i P_ij do_i              dS_ij = scale P_ij (do_i . v_j - delta_i)
//   dq_i = sum_j dS_ij k_j              dk_j  = sum_i dS_ij q_i
//   dz   = dy * y * (1 - sigmoid(z))    (y sigmoid'(z) / sigmoid(z); no division)
// i over the queries of every head that shares the key head.
//
// Three kernels: delta, dz and the gated do per row; then dk and dv per tile of
// keys, looping over the queries, and dq per tile of queries, looping over the
// keys; then the sum of dk's and dv's parts, where there are several.  The
// scores are formed in both, seven products for five, and in exchange every sum
// is one workgroup's, in a fixed order: no atomics.
//
// 4,096 tokens of 32 heads of 128 over 8, bf16: 490 to 512 us in all, 670 to 700
// TFLOP/s on five products (940 to 980 on the seven), matrix cores 51 % of the
// cycles, waits 30 %.  Six ragged fp32 sequences of up to 500 tokens, 8 heads of
// 64 over 2: 70 us, bound by the length of a workgroup's chain of fp32 products.
//
// With a window a key tile has the queries up to its last key's window, and
// queries of 32 rows of four heads share a workgroup where the group allows it.
// What later queries give to the first tokens is summed apart (far queries,
// below), else the first tile would be as long as the sequence: 8,192 tokens
// under a window of 1,024, 849 us with it in one piece, 517 to 531 now (floor 233;
// 610 to 625 TFLOP/s on five products, matrix cores 44 %, vector units 30 %, waits 38 %).
// The six fp32 sequences under a window of 100: 60 us (47 of them the gradients,
// matrix cores 26 %; chains of 3 to 5 steps of 4 us each and their starts).
#include "kda_attn_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kRows = 128;  // rows of a workgroup, 32 a wave
constexpr int kMostParts = 8;

struct BwdK {
    int64_t T;
    int H, Hkv, N;
    const int32_t* cu;
    const void *q, *k, *v, *z, *out, *dy;
    const float* lse;
    void *dq, *dk, *dv, *dz;
    float2* stats;    // [T, H]: lse log2(e), delta
    void* dog;        // [T, H, dv]: dy * sigmoid(z), or dy itself without a gate
    float scale;
    int parts, q_parts;
    float* part;      // [parts][T, Hkv][dk + dv]
    float* q_part;    // [q_parts][T, H][dk]
    int window, sinks;
    // With a window: the first tokens' far queries, worked on apart (far_parts 0: not).
    int far_tiles, far_parts;
    int64_t far_buckets;
    float* far;       // [1 + far_parts][far_buckets, sinks, Hkv][dk + dv]
};

// The kernel's arguments (its only parameter but for numbers), read again: the
// compiler loads all of them at the start and would keep those that only the
// results need in scalar registers that the loop has no room for.
__device__ __forceinline__ BwdK again() {
    typedef const __attribute__((address_space(4))) BwdK* Args;
    uint64_t at = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(at));
    const Args from = reinterpret_cast<Args>(at);
    BwdK a;
    __builtin_memcpy(&a, from, sizeof(a));
    return a;
}

// The first tokens of a sequence are attended by every token of it, the others
// by window + 127 of their tile at most: a tile of first tokens would be many
// times as long as the rest.  So it takes as many queries as the others do, and
// those behind, from far_from() on, go to workgroups of their own, in parts.
// Only sequences of reach() tokens or more have such queries: a bucket for each
// sequence, or, where that is fewer, one for each reach() tokens, in which at most
// one of them begins, the one that holds the bucket's last token.
__device__ __forceinline__ int reach(const BwdK& a) { return a.window + kRows; }
template <int kQ>
__device__ __forceinline__ int far_from(const BwdK& a, int k_first, int len) {
    return k_first + (min(len - k_first, kRows - 1 + a.window) + kQ - 1) / kQ * kQ;
}
__device__ __forceinline__ bool far_by_sequence(const BwdK& a) { return a.N <= a.far_buckets; }
__device__ __forceinline__ bool far_sequence(const BwdK& a, int64_t bucket, int64_t& start, int& len) {
    if (far_by_sequence(a)) {
        seq_bounds(a.cu, static_cast<int>(bucket), a.T, start, len);
        return len >= reach(a);
    }
    const int64_t token = (bucket + 1) * reach(a) - 1;
    seq_bounds(a.cu, a.cu == nullptr ? 0 : find_seq(a.cu, a.N, token), a.T, start, len);
    return start >= bucket * reach(a) && start <= token && token < start + len && len >= reach(a);
}
// The bucket of the sequence that begins at `start`.
__device__ __forceinline__ int64_t far_bucket(const BwdK& a, int64_t start) {
    if (!far_by_sequence(a)) return start / reach(a);
    return a.cu == nullptr ? 0 : find_seq(a.cu, a.N, start);
}
// A row's place in the far sums.
__device__ __forceinline__ float* far_row(const BwdK& a, int slot, int64_t bucket, int key, int kvh, int width) {
    return a.far + (((slot * a.far_buckets + bucket) * a.sinks + key) * a.Hkv + kvh) * width;
}

// One row (token, head) per 16 lanes, so that a load takes whole lines of
// neighbouring rows.  Bound by memory: 131,072 rows of 128, 68 MB, in 15 us
// (4.5 TB/s).
template <typename T, int DV>
__global__ __launch_bounds__(kThreads) void attn_bwd_rows_kernel(BwdK a) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    const int64_t tokens = a.cu == nullptr ? a.T : min(static_cast<int64_t>(max(a.cu[a.N], 0)), a.T);
    const bool there = row < tokens * a.H;  // rows behind the last sequence are left as they are
    constexpr int kV = 4;
    float sum = 0.f;
    if (there) {
        const int64_t at = row * DV;
#pragma unroll
        for (int ch = kV * c; ch < DV; ch += 16 * kV) {
            float dy[kV], y[kV];
            ld4(static_cast<const T*>(a.dy) + at + ch, dy);
            ld4(static_cast<const T*>(a.out) + at + ch, y);
            if (a.z == nullptr) {
#pragma unroll
                for (int e = 0; e < kV; ++e) sum += dy[e] * y[e];
                continue;
            }
            // delta from the gated gradient as it is stored, do . o with
            // o = y / sigmoid(z): do . v - delta then cancels as it must in
            // rows of few keys (dy . y, of the unrounded gradient, leaves the
            // rounding of do there).  A gate that is all but closed has y = 0.
            float z[kV], g[kV];
            ld4(static_cast<const T*>(a.z) + at + ch, z);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float sg = sigmoid_fast(z[e]);
                g[e] = round_to<T>(dy[e] * sg);
                sum += sg > 1e-30f ? g[e] * (y[e] / sg) : 0.f;
                z[e] = dy[e] * y[e] * sigmoid_fast(-z[e]);  // 1 - sigmoid(z) without cancellation
            }
            st4(static_cast<T*>(a.dog) + at + ch, g);
            st4(static_cast<T*>(a.dz) + at + ch, z);
        }
    }
    sum = row_ror_add<1>(sum);
    sum = row_ror_add<2>(sum);
    sum = row_ror_add<4>(sum);
    sum = row_ror_add<8>(sum);
    if (there && c == 0) a.stats[row] = make_float2(a.lse[row] * kLog2e, sum);
}

// Writes a transposed 32-column result (register 4 i + e: channel 8 i + 4 half
// + e of tile `tile`) of this lane's row.
template <typename T, int D, int kTiles>
__device__ __forceinline__ void store_rows(T* row, const f32x16 (&acc)[kTiles], float f, int half) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int ch = 32 * i + 8 * r4 + 4 * half;
            if (ch >= D) continue;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = acc[i][4 * r4 + e] * f;
            st4(row + ch, y);
        }
}

template <typename T, int DK, int DV>
struct DqSizes {
    // 64 keys a tile where two workgroups' registers allow it (fp32 at 64
    // channels: 256 and 2 spilled, with 32 keys 218)
    static constexpr int kKeys = sizeof(T) == 4 && DK >= 64 ? 32 : 64;
    static constexpr int kBuf = kKeys * (DK + DV) * static_cast<int>(sizeof(T));
    static constexpr int kLds = 2 * kBuf + tr_slack(DV);
};

// Query gradients: one workgroup per (tile of 128 queries, head, part of the
// keys), or of 32 queries of four heads that share their keys (as the prefill); a wave's queries, output gradients and sums stay in its registers, the
// keys and values pass through LDS once for four waves.
template <typename T, int DK, int DV, bool kWin, int kTileRows>
__device__ __forceinline__ void query_gradients(const BwdK& a, unsigned block, char* smem) {
    using Sz = DqSizes<T, DK, DV>;
    constexpr int kKeys = Sz::kKeys, kSub = kKeys / 32;
    constexpr int kQPieces = DK / (2 * Elem<T>::kPer16), kVPieces = DV / (2 * Elem<T>::kPer16);
    constexpr int kKTiles = (DK + 31) / 32;
    constexpr int kP = Elem<T>::kPieces;
    constexpr int kV = kKeys * DK * static_cast<int>(sizeof(T));  // the values, behind the keys

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int G = a.H / a.Hkv;
    constexpr int kHeads = kRows / kTileRows;
    const int slots = a.H / kHeads * a.q_parts;
    const int64_t rank = block / slots;
    const int slot = block % slots / a.q_parts, part = block % a.q_parts;
    const int kvh = slot % a.Hkv, h = kvh * G + slot / a.Hkv * kHeads + (kHeads > 1 ? wave : 0);
    const Tile t = find_tile<kTileRows>(a.cu, a.N, a.T, rank);
    if (!t.there) return;
    const int q0 = t.level * kTileRows + (kHeads > 1 ? 0 : wave * 32);
    const int rows = min(32, t.len - q0);

    const int q_row = a.H * DK * static_cast<int>(sizeof(T)), o_row = a.H * DV * static_cast<int>(sizeof(T));
    const int k_row = a.Hkv * DK * static_cast<int>(sizeof(T)), v_row = a.Hkv * DV * static_cast<int>(sizeof(T));
    u32x4 qf[kQPieces], of[kVPieces];
    {
        const auto qs = rows_of(static_cast<const T*>(a.q) + h * DK, t.start + q0, q_row, rows);
        const auto os = rows_of(static_cast<const T*>(a.dog) + h * DV, t.start + q0, o_row, rows);
#pragma unroll
        for (int s = 0; s < kQPieces; ++s) qf[s] = buffer_load16(qs, c * q_row + (2 * s + half) * 16);
#pragma unroll
        for (int s = 0; s < kVPieces; ++s) of[s] = buffer_load16(os, c * o_row + (2 * s + half) * 16);
    }
    const int64_t at = (t.start + q0 + c) * a.H + h;
    const float2 stat = c < rows ? a.stats[at] : make_float2(0.f, 0.f);
    const float lse2 = stat.x, delta = stat.y;
    const float sc = a.scale * kLog2e;

    f32x16 acc[kKTiles];
#pragma unroll
    for (int i = 0; i < kKTiles; ++i) acc[i] = f32x16{};
    TileCopy<T, kKeys, DK, kThreads> ck;
    TileCopy<T, kKeys, DV, kThreads> cv;
    TileRead<T, DK> rk;
    TileRead<T, DV> rv;
    rk.init_rows(c, half);
    rk.init_columns(lane);
    rv.init_rows(c, half);
    const KeyWalk<kWin, kKeys> walk(t.level * kTileRows, t.len, a.window, a.sinks);
    // tiles that some row attends
    const int64_t steps = walk.before((min(t.level * kTileRows + kTileRows, t.len) + kKeys - 1) / kKeys * kKeys);
    const int start = walk.nth(static_cast<int>(steps * part / a.q_parts));
    const int last = walk.nth(static_cast<int>(steps * (part + 1) / a.q_parts));
    const T* kbase = static_cast<const T*>(a.k) + kvh * DK;
    const T* vbase = static_cast<const T*>(a.v) + kvh * DV;
    auto fetch = [&](int j0) {
        const int there = walk.rows(j0);
        ck.load(rows_of(kbase, t.start + j0, k_row, there), k_row, tid);
        cv.load(rows_of(vbase, t.start + j0, v_row, there), v_row, tid);
    };
    auto put = [&](char* buf) {
        ck.store(buf, tid);
        cv.store(buf + kV, tid);
    };
    auto work = [&](const char* sK, int j0) __attribute__((always_inline)) {
        const char* sV = sK + kV;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            const int k0 = j0 + 32 * u;
            if (k0 > q0 + 31) break;
            if constexpr (kWin) {
                if (k0 + 32 <= walk.least(q0) && k0 >= walk.sinks) continue;
            }
            f32x16 s{}, dp{};
#pragma unroll
            for (int p = 0; p < kQPieces; ++p) {
                s = mma<T>(rk.rows(sK + 32 * u * rk.kRow, p), qf[p], s);
                if (p < kVPieces) dp = mma<T>(rv.rows(sV + 32 * u * rv.kRow, p), of[p < kVPieces ? p : 0], dp);
            }
            lookahead<kQPieces + kVPieces, sizeof(T) == 2 ? 3 : 1, Elem<T>::kMfmas>();
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -lse2)) * (dp[r] - delta);
            if (k0 + 31 > q0) {  // the diagonal: keys behind the row's own are not attended
                const int most = opaque(q0 + c - k0 - 4 * half);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r / 4) + r % 4 > most) s[r] = 0.f;
            }
            if constexpr (kWin) {
                if (k0 < walk.least(q0 + 31) && k0 + 32 > walk.sinks) {  // keys before the row's window, but for the first ones
                    const int least = opaque(walk.least(q0 + c) - k0 - 4 * half), sink = opaque(walk.sinks - k0 - 4 * half);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (outside(8 * (r / 4) + r % 4, least, sink)) s[r] = 0.f;
                }
            }
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const u32x4 b = as_operand<T>(s, p);
#pragma unroll
                for (int i = 0; i < kKTiles; ++i)
                    acc[i] = mma<T>(rk.columns(sK + 32 * u * rk.kRow, i, p), b, acc[i]);
            }
            if constexpr (sizeof(T) == 2) lookahead<kKTiles * kP, 3, 1, 2>();
        }
    };
    if (start < last) {
        fetch(start);
        arrive(qf);
        arrive(of);
        put(smem);
    }
    for (int j0 = start; j0 < last;) {
        const int j1 = walk.next(j0), j2 = walk.next(j1);
        tile_barrier();
        if (j1 < last) fetch(j1);
        work(smem, j0);
        if (j1 >= last) break;
        put(smem + Sz::kBuf);
        tile_barrier();
        if (j2 < last) fetch(j2);
        work(smem + Sz::kBuf, j1);
        if (j2 < last) put(smem);
        j0 = j2;
    }
    if (c >= rows) return;
    const BwdK b = kWin ? again() : a;
    if (b.q_parts > 1)
        store_rows<float, DK>(b.q_part + (static_cast<int64_t>(part) * b.T * b.H + at) * DK, acc, b.scale, half);
    else
        store_rows<T, DK>(static_cast<T*>(b.dq) + at * DK, acc, b.scale, half);
}

template <typename T, int DK, int DV>
struct DkvSizes {
    static constexpr int kQ = 32;  // queries of a step
    static constexpr int kStats = kQ * 2 * 4;  // lse and delta of the step's queries, in pairs
    static constexpr int kBuf = kQ * (DK + DV) * static_cast<int>(sizeof(T)) + kStats;
    // Where a lane's sums, keys and values together exceed half its registers,
    // the values are read from LDS for every step: two workgroups then share a
    // CU, and one's products cover the other's exponentials and LDS reads.  In
    // fp32 they would else come from the caches: ragged sequences of up to 1,000
    // tokens take 301 us so at 64 channels (304 from the caches) and 676 at 128
    // (697); at 16 channels the caches are faster (47 against 51 us).
    static constexpr bool kValuesInLds = DK == 128 || (sizeof(T) == 4 && DK == 64);
    static constexpr int kValues = kValuesInLds ? kRows * DV * static_cast<int>(sizeof(T)) : 0;
    static constexpr int kLds = 2 * kBuf + tr_slack(DV) + kValues;
};

// Key and value gradients: one workgroup per (tile of 128 keys, key head, part).  The tile's work is
// the sequence of its steps of 32 queries, head by head of the group; the
// parts cut it into equal pieces where there are few tiles, and their sums
// (fp32) are added by attn_bwd_sum_kernel.
template <typename T, int DK, int DV, bool kWin, bool kFar>
__device__ __forceinline__ void key_gradients(const BwdK& a, unsigned block, char* smem) {
    using Sz = DkvSizes<T, DK, DV>;
    constexpr int kQ = Sz::kQ;
    constexpr int kKPieces = DK / (2 * Elem<T>::kPer16), kVPieces = DV / (2 * Elem<T>::kPer16);
    constexpr int kKTiles = (DK + 31) / 32, kVTiles = (DV + 31) / 32;
    constexpr int kP = Elem<T>::kPieces;
    constexpr int kO = kQ * DK * static_cast<int>(sizeof(T));       // the output gradients, behind the queries
    constexpr int kS = kO + kQ * DV * static_cast<int>(sizeof(T));  // the statistics, behind both

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int G = a.H / a.Hkv;
    int kvh, part, parts, k_first;
    int64_t bucket = 0;
    Tile t;
    if constexpr (kFar) {
        parts = a.far_parts;
        part = block % parts;
        kvh = block / parts % a.Hkv;
        k_first = static_cast<int>(block / (parts * a.Hkv) % a.far_tiles) * kRows;
        bucket = block / (parts * a.Hkv) / a.far_tiles;
        if (!far_sequence(a, bucket, t.start, t.len)) return;
        t.len = uniform(t.len);
        t.start = uniform64(t.start);
        if (far_from<kQ>(a, k_first, t.len) >= t.len) return;
    } else {
        const int64_t rank = block / (a.Hkv * a.parts);
        const int slot = block % (a.Hkv * a.parts);
        parts = a.parts;
        kvh = slot % a.Hkv;
        part = slot / a.Hkv;
        t = find_tile<kRows>(a.cu, a.N, a.T, rank);
        if (!t.there) return;
        // the first keys of a sequence have the most queries: levels from the end
        k_first = (t.tiles - 1 - t.level) * kRows;
    }
    const int k0 = k_first + wave * 32;
    const int rows = min(32, t.len - k0);

    const int q_row = a.H * DK * static_cast<int>(sizeof(T)), o_row = a.H * DV * static_cast<int>(sizeof(T));
    const int k_row = a.Hkv * DK * static_cast<int>(sizeof(T)), v_row = a.Hkv * DV * static_cast<int>(sizeof(T));
    // bf16: this wave's keys, and its values where they fit, stay in registers.
    // fp32: they would not fit beside the sums, and each step, whose products
    // take four times as many cycles per byte, reads them again, the keys from
    // the caches.
    constexpr bool kKeep = sizeof(T) == 2;
    const auto ks = rows_of(static_cast<const T*>(a.k) + kvh * DK, t.start + k0, k_row, rows);
    const auto vs = rows_of(static_cast<const T*>(a.v) + kvh * DV, t.start + k0, v_row, rows);
    const int k_at = c * k_row + half * 16, v_at = c * v_row + half * 16;
    constexpr bool kVLds = Sz::kValuesInLds, kVKeep = kKeep && !kVLds;
    char* sV = smem + 2 * Sz::kBuf + tr_slack(DV);
    u32x4 kf[kKeep ? kKPieces : 1], vf[kVKeep ? kVPieces : 1];
    if constexpr (kKeep) {
#pragma unroll
        for (int s = 0; s < kKPieces; ++s) kf[s] = buffer_load16(ks, k_at + s * 32);
    }
    if constexpr (kVKeep) {
#pragma unroll
        for (int s = 0; s < kVPieces; ++s) vf[s] = buffer_load16(vs, v_at + s * 32);
    }
    if constexpr (kVLds) {
        TileCopy<T, kRows, DV, kThreads> cv;
        cv.load(rows_of(static_cast<const T*>(a.v) + kvh * DV, t.start + k_first, v_row, min(kRows, t.len - k_first)), v_row, tid);
        cv.store(sV, tid);
    }
    const float sc = a.scale * kLog2e;
    f32x16 gk[kKTiles], gv[kVTiles];
#pragma unroll
    for (int i = 0; i < kKTiles; ++i) gk[i] = f32x16{};
#pragma unroll
    for (int i = 0; i < kVTiles; ++i) gv[i] = f32x16{};

    TileCopy<T, kQ, DK, kThreads> cq;
    TileCopy<T, kQ, DV, kThreads> co;
    TileRead<T, DK> rq;
    TileRead<T, DV> ro;
    rq.init_rows(c, half);
    rq.init_columns(lane);
    ro.init_rows(c, half);
    ro.init_columns(lane);
    uint2 stat{};
    // the queries that attend some key of the tile, and this workgroup's share of them: [i_first, end)
    int i_first = k_first, end = t.len;
    if constexpr (kFar) i_first = far_from<kQ>(a, k_first, t.len);
    else if constexpr (kWin) {
        if (k_first >= a.sinks || a.far_parts > 0) end = min(t.len, k_first + kRows - 1 + a.window);
    }
    const int steps = (end - i_first + kQ - 1) / kQ;  // per head
    const int64_t all = static_cast<int64_t>(steps) * G;
    int n = static_cast<int>(all * part / parts);
    const int n_end = static_cast<int>(all * (part + 1) / parts);
    // With a window and a tile in one piece: each head's steps begin where the
    // other tiles' do, modulo their number, so that the tiles that need the same
    // queries read them at about the same time (8,192 tokens under a window of
    // 1,024: 0.57 GB read from memory for 1.48, 530 to 521 us).
    int i_start = i_first;
    if constexpr (kWin && !kFar)
        if (parts == 1) i_start = uniform(i_first + (steps - k_first / kQ % steps) % steps * kQ);
    int f_head = uniform(kvh * G + n / steps), f_i0 = uniform(i_start + n % steps * kQ);  // the next step to fetch
    auto fetch = [&]() __attribute__((always_inline)) {
        const int here = min(kQ, t.len - f_i0);
        cq.load(rows_of(static_cast<const T*>(a.q) + f_head * DK, t.start + f_i0, q_row, here), q_row, tid);
        co.load(rows_of(static_cast<const T*>(a.dog) + f_head * DV, t.start + f_i0, o_row, here), o_row, tid);
        // rows behind the sequence's end are 0 in all three and add nothing
        if (wave == 0)
            stat = buffer_load8(rows_of(a.stats + f_head, t.start + f_i0, a.H * 8, here), c * a.H * 8);
        f_i0 += kQ;
        if constexpr (kWin && !kFar) {
            if (f_i0 >= end) f_i0 = i_first;
            if (f_i0 == i_start) ++f_head;
        } else if (f_i0 >= end) {
            f_i0 = i_first;
            ++f_head;
        }
    };
    auto put = [&](char* buf) __attribute__((always_inline)) {
        cq.store(buf, tid);
        co.store(buf + kO, tid);
        if (wave == 0) reinterpret_cast<uint2*>(buf + kS)[c] = stat;
    };
    int i0 = f_i0 - kQ;  // the step worked on
    auto work = [&](const char* sQ) __attribute__((always_inline)) {
        i0 = i0 + kQ < end ? i0 + kQ : i_first;
        if (i0 + kQ - 1 < k0) return;  // queries before this wave's keys
        if constexpr (kWin) {
            if (i0 - a.window > k0 + 30 && k0 >= a.sinks) return;  // and those that have left them behind
        }
        const char* sO = sQ + kO;
        const f32x4* sStats = reinterpret_cast<const f32x4*>(sQ + kS);
        f32x16 s{}, dp{};
#pragma unroll
        for (int p = 0; p < kKPieces; ++p) {
            s = mma<T>(rq.rows(sQ, p), kKeep ? kf[kKeep ? p : 0] : buffer_load16(ks, k_at + p * 32), s);
            if (p < kVPieces) {
                u32x4 v;
                if constexpr (kVLds) v = ro.rows(sV + wave * 32 * ro.kRow, p);
                else if constexpr (kVKeep) v = vf[p < kVPieces ? p : 0];
                else v = buffer_load16(vs, v_at + p * 32);
                dp = mma<T>(ro.rows(sO, p), v, dp);
            }
        }
        if constexpr (kVKeep) lookahead<kKPieces + kVPieces, 4, Elem<T>::kMfmas>();
        else if constexpr (kVLds) lookahead<kKPieces, 1, 2, 3>();
        // register r: query i0 + 8 (r / 4) + 4 half + r % 4; key k0 + c
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const f32x4 lo = sStats[4 * r4 + 2 * half], hi = sStats[4 * r4 + 2 * half + 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * r4 + e;
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -(e < 2 ? lo : hi)[e % 2 * 2]));
                dp[r] = s[r] * (dp[r] - (e < 2 ? lo : hi)[e % 2 * 2 + 1]);
            }
        }
        if (i0 < k0 + 31) {  // the diagonal: queries before the key do not attend it
            const int least = opaque(k0 + c - i0 - 4 * half);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (8 * (r / 4) + r % 4 < least) s[r] = dp[r] = 0.f;
        }
        if constexpr (kWin) {
            if (i0 + kQ > k0 + a.window && k0 + 32 > a.sinks) {  // queries whose window begins behind the key, unless it is a first one
                const int most = opaque(k0 + c < a.sinks ? INT32_MAX : k0 + c + a.window - i0 - 4 * half);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r / 4) + r % 4 >= most) s[r] = dp[r] = 0.f;
            }
        }
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            const u32x4 b = as_operand<T>(s, p), d = as_operand<T>(dp, p);
#pragma unroll
            for (int i = 0; i < kVTiles; ++i) gv[i] = mma<T>(ro.columns(sO, i, p), b, gv[i]);
#pragma unroll
            for (int i = 0; i < kKTiles; ++i) gk[i] = mma<T>(rq.columns(sQ, i, p), d, gk[i]);
        }
        if constexpr (sizeof(T) == 2) lookahead<(kVTiles + kKTiles) * kP, 3, 1, 2>();
    };
    if constexpr (kKeep) arrive(kf);
    if constexpr (kVKeep) arrive(vf);
    if (n < n_end) {
        fetch();
        put(smem);
    }
    for (; n < n_end; n += 2) {
        tile_barrier();
        if (n + 1 < n_end) fetch();
        work(smem);
        if (n + 1 >= n_end) break;
        put(smem + Sz::kBuf);
        tile_barrier();
        if (n + 2 < n_end) fetch();
        work(smem + Sz::kBuf);
        if (n + 2 < n_end) put(smem);
    }
    if constexpr (kFar) {
        if (c < rows && k0 + c < a.sinks) {
            float* to = far_row(a, 1 + part, bucket, k0 + c, kvh, DK + DV);
            store_rows<float, DK>(to, gk, a.scale, half);
            store_rows<float, DV>(to + DK, gv, 1.f, half);
        }
        return;
    }
    const BwdK b = kWin ? again() : a;
    if (kWin && b.parts == 1 && b.far_parts > 0 && k_first < b.sinks && far_from<kQ>(b, k_first, t.len) < t.len) {
        if (c < rows && k0 + c < b.sinks) {
            float* to = far_row(b, 0, far_bucket(b, t.start), k0 + c, kvh, DK + DV);
            store_rows<float, DK>(to, gk, b.scale, half);
            store_rows<float, DV>(to + DK, gv, 1.f, half);
            return;
        }
    }
    if (c < rows) {
        const int64_t at = (t.start + k0 + c) * b.Hkv + kvh;
        if (b.parts > 1) {
            float* to = b.part + (static_cast<int64_t>(part) * b.T * b.Hkv + at) * (DK + DV);
            store_rows<float, DK>(to, gk, b.scale, half);
            store_rows<float, DV>(to + DK, gv, 1.f, half);
        } else {
            store_rows<T, DK>(static_cast<T*>(b.dk) + at * DK, gk, b.scale, half);
            store_rows<T, DV>(static_cast<T*>(b.dv) + at * DV, gv, 1.f, half);
        }
    }
}

// Both in one launch, the key gradients' workgroups first: they are the longer
// ones, and the query gradients' fill the chip behind them (one after the
// other, each launch ends with most of the chip idle: the small fp32 batch
// takes 55 + 59 us so).  Rows of up to 256 bytes leave registers for two
// workgroups a CU (fp32 at 64 channels: 4,000 tokens 1,900 us, 2,180 with one;
// the ragged batch of up to 1,000 tokens 301 us, 355 with one).
template <typename T, int DK, int DV, bool kWin, int kTileRows>
__global__ __launch_bounds__(kThreads, (DK * sizeof(T) <= 256 ? 2 : 1)) void attn_bwd_kernel(BwdK a, unsigned key_groups, unsigned far_groups) {
    extern __shared__ __align__(16) char smem[];
    unsigned block = blockIdx.x;
    if constexpr (kWin) {
        if (block < far_groups) return key_gradients<T, DK, DV, true, true>(a, block, smem);
        block -= far_groups;
    }
    if (block < key_groups) key_gradients<T, DK, DV, kWin, false>(a, block, smem);
    else query_gradients<T, DK, DV, kWin, kTileRows>(a, block - key_groups, smem);
}

// Adds four channels of `parts` rows `step` apart, in their order, eight in flight.
__device__ __forceinline__ void add_parts(const float* from, int64_t step, int parts, float (&sum)[4]) {
    constexpr int kEach = 8;
    for (int p0 = 0; p0 < parts; p0 += kEach) {
        float x[kEach][4];
#pragma unroll
        for (int p = 0; p < kEach; ++p)
            if (p0 + p < parts) ld4(from + (p0 + p) * step, x[p]);
#pragma unroll
        for (int p = 0; p < kEach; ++p)
            if (p0 + p < parts) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += x[p][e];
            }
    }
}

template <typename T, int DK, int DV>
__device__ __forceinline__ void store_sum(const BwdK& a, int64_t row, int ch, const float (&sum)[4]) {
    if (ch < DK) st4(static_cast<T*>(a.dk) + row * DK + ch, sum);
    else st4(static_cast<T*>(a.dv) + row * DV + ch - DK, sum);
}

// Adds what far queries gave to a first token; false: there are none.
template <typename T, int DK, int DV>
__device__ __forceinline__ bool add_far(const BwdK& a, int64_t bucket, int key, int len, int kvh, int ch, int first, float (&sum)[4]) {
    if (far_from<DkvSizes<T, DK, DV>::kQ>(a, key / kRows * kRows, len) >= len) return false;
    const int64_t step = a.far_buckets * a.sinks * a.Hkv * (DK + DV);
    add_parts(far_row(a, first, bucket, key, kvh, DK + DV) + ch, step, 1 + a.far_parts - first, sum);
    return true;
}

// Adds the parts in their order, four channels per thread: first the rows of
// the key heads (dk and dv together), then those of the query heads.  Bound by
// memory: four parts of 4,096 tokens of 8 heads, 151 MB, in 23 us (6.6 TB/s,
// a part of it from the caches).
template <typename T, int DK, int DV, bool kWin>
__global__ __launch_bounds__(kThreads) void attn_bwd_sum_kernel(BwdK a) {
    constexpr int kKv = (DK + DV) / 4, kQ = DK / 4;
    const int64_t tokens = a.cu == nullptr ? a.T : min(static_cast<int64_t>(max(a.cu[a.N], 0)), a.T);
    const int64_t kv_all = a.parts > 1 ? tokens * a.Hkv * kKv : 0, q_all = a.q_parts > 1 ? tokens * a.H * kQ : 0;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < kv_all) {
        const int64_t row = i / kKv;
        const int ch = static_cast<int>(i % kKv) * 4;
        add_parts(a.part + row * (DK + DV) + ch, a.T * a.Hkv * (DK + DV), a.parts, sum);
        if (kWin && a.far_parts > 0) {
            const int64_t token = row / a.Hkv;
            int64_t start;
            int len;
            seq_bounds(a.cu, a.cu == nullptr ? 0 : find_seq(a.cu, a.N, token), a.T, start, len);
            if (token - start < a.sinks && len >= reach(a))
                add_far<T, DK, DV>(a, far_bucket(a, start), static_cast<int>(token - start), len, static_cast<int>(row % a.Hkv), ch, 1, sum);
        }
        store_sum<T, DK, DV>(a, row, ch, sum);
        return;
    }
    i -= kv_all;
    if (i >= q_all) return;
    add_parts(a.q_part + i * 4, a.T * a.H * DK, a.q_parts, sum);
    st4(static_cast<T*>(a.dq) + i * 4, sum);
}

// The first tokens' gradients where no tile is cut into parts: what their own
// tile's workgroup summed, then the far parts.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void attn_bwd_far_sum_kernel(BwdK a) {
    constexpr int kKv = (DK + DV) / 4;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int ch = static_cast<int>(i % kKv) * 4;
    i /= kKv;
    const int kvh = static_cast<int>(i % a.Hkv);
    i /= a.Hkv;
    const int key = static_cast<int>(i % a.sinks);
    const int64_t bucket = i / a.sinks;
    int64_t start;
    int len;
    if (bucket >= a.far_buckets || !far_sequence(a, bucket, start, len)) return;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (add_far<T, DK, DV>(a, bucket, key, len, kvh, ch, 0, sum)) store_sum<T, DK, DV>(a, (start + key) * a.Hkv + kvh, ch, sum);
}

// Into how many parts the work of a tile is cut: key tiles so that their
// workgroups, which differ in length, fill the chip several times; query tiles
// where they and the key tiles' together leave it half empty.
constexpr int kKeyWant = 1024, kQueryWant = 384;  // workgroups below which tiles are cut
struct BwdParts {
    int key, query;
};
// With a window the workgroups of key tiles are equally long but for a sequence's
// last ones, and short: about one round of them, none of fewer than kLeast of its
// steps (32 queries of a key tile, 32 keys of a query tile).  fp32, whose steps
// are four times as long, is cut finer.  bf16 (8 heads over 2, six sequences of
// up to 500 tokens): 8 key parts 38 us, 3 parts 30; 4,096 tokens of 4 heads under
// a window of 1,024: 62 us, for 512 workgroups 79; 16 sequences of up to 800
// tokens 140 and 157.  fp32: the same six sequences 62 us, of 8 steps at least 84,
// of 2 as long; 3 sequences of 4 heads of 128 104 us, of 2 steps at least 119.
constexpr int kKeyWantWindow = 256, kKeyWantWindowF32 = 512, kQueryWantWindow = 256;
constexpr int kLeastSteps = 8, kLeastKeyStepsF32 = 4, kLeastQueryStepsF32 = 2;

BwdParts bwd_parts(int64_t T, int N, int H, int Hkv, DT x, int window) {
    const int64_t tiles = attn_tiles(T, N, kRows), keys = tiles * Hkv, queries = tiles * H;
    if (tiles == 0) return {1, 1};
    auto parts = [](int64_t want, int64_t units, int64_t most) {
        const int64_t p = (want + units - 1) / units;
        return static_cast<int>(p < 1 || most < 1 ? 1 : p > most ? most : p);
    };
    if (window < 1) return {parts(kKeyWant, keys, kMostParts), parts(kQueryWant, queries, kMostParts / 2)};
    auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    const bool four = heads_share(H, Hkv), wide = x == DT::F32;
    const int64_t rows = four ? 32 : kRows, seen = least(window, T);
    const int64_t key_steps = (seen + kRows + 31) / 32 * (H / Hkv), query_steps = (seen + rows + 31) / 32;
    const int64_t units = four ? attn_tiles(T, N, 32) * (H / 4) : queries;
    return {parts(wide ? kKeyWantWindowF32 : kKeyWantWindow, keys, least(kMostParts, key_steps / (wide ? kLeastKeyStepsF32 : kLeastSteps))),
            parts(kQueryWantWindow, units, least(kMostParts / 2, query_steps / (wide ? kLeastQueryStepsF32 : kLeastSteps)))};
}

// The far queries' workgroups.  More first tokens than a tile's reach are
// balanced as they are.  Parts as long as the other workgroups', as far as their
// sums stay few (kFarRows rows of all heads).
constexpr int kMostFarParts = 64;
constexpr int64_t kFarRows = 16384, kFarGroups = 65536;
// Rows whose sums one launch adds, four channels a thread: below 2^32 threads.
// Calls of more (first tokens of a tile's reach in millions of tokens, whose tiles
// are many) are balanced as they are too.
int64_t most_far_rows(int Hkv, int width) { return ((int64_t(1) << 32) - kThreads) / (static_cast<int64_t>(Hkv) * (width / 4)); }
struct FarPlan {
    int64_t buckets = 0;
    int tiles = 0, parts = 0;
    int64_t rows(int sinks) const { return buckets * sinks; }
};
// width: channels of a key and a value.
FarPlan far_plan(int64_t T, int64_t N, int Hkv, int width, int window, int sinks, int near_parts) {
    FarPlan p;
    const int64_t reach = static_cast<int64_t>(window) + kRows;
    if (window < 1 || sinks < 1 || sinks > reach || T < reach) return p;
    const int64_t buckets = T / reach < N ? T / reach : N;
    if (buckets * sinks > most_far_rows(Hkv, width)) return p;
    p.buckets = buckets;
    p.tiles = (sinks + kRows - 1) / kRows;
    int64_t parts = ((T - reach) * near_parts + reach - 1) / reach;
    const int64_t groups = p.buckets * p.tiles * Hkv, rows = p.rows(sinks);
    if (parts > kMostFarParts) parts = kMostFarParts;
    if (parts * groups > kFarGroups) parts = kFarGroups / groups;
    if (parts * rows > kFarRows) parts = kFarRows / rows;
    p.parts = static_cast<int>(parts < 1 ? 1 : parts);
    return p;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// How a call is cut, and where its workspace holds what: the launch and the
// queries all go by this one.  A window and first tokens of more than there are
// tokens count as that many, so that calls of the same view have the same plan.
struct BwdPlan {
    int window, sinks;
    BwdParts parts;
    FarPlan far;
    size_t dog, part, q_part, far_sums, bytes;  // (the statistics come first)
};
BwdPlan bwd_plan(int64_t T, int N, int H, int Hkv, int dk, int dv, DT x, bool gate, int window, int sinks) {
    BwdPlan p;
    p.window = static_cast<int>(window < T ? window : T);
    p.sinks = static_cast<int>(sinks < T ? sinks : T);
    p.parts = bwd_parts(T, N, H, Hkv, x, p.window);
    p.far = far_plan(T, N, Hkv, dk + dv, p.window, p.sinks, p.parts.key);
    const size_t rows = static_cast<size_t>(T) * H, kv = static_cast<size_t>(Hkv) * (dk + dv) * 4;
    p.dog = up256(rows * 8);
    p.part = p.dog + (gate ? up256(rows * dv * (x == DT::BF16 ? 2 : 4)) : 0);
    p.q_part = p.part + (p.parts.key > 1 ? up256(p.parts.key * T * kv) : 0);
    p.far_sums = p.q_part + (p.parts.query > 1 ? up256(p.parts.query * rows * dk * 4) : 0);
    p.bytes = p.far_sums + (p.far.parts > 0 ? up256((1 + p.far.parts) * p.far.rows(p.sinks) * kv) : 0);
    return p;
}

template <typename F>
hipError_t allow_lds(F fn, int lds) {
    if (lds <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <typename T, int DK, int DV, bool kWin, int kTileRows>
hipError_t launch_bwd(const AttnBackwardArgs& a, hipStream_t s) {
    const AttnArgs& f = a.f;
    BwdK k{};
    k.T = f.T; k.H = f.H; k.Hkv = f.Hkv; k.N = f.N; k.cu = f.cu;
    k.q = f.q; k.k = f.k; k.v = f.v; k.z = f.z; k.out = f.out; k.dy = a.dy; k.lse = f.lse;
    k.dq = a.dq; k.dk = a.dk; k.dv = a.dv; k.dz = a.dz; k.scale = f.scale;
    const BwdPlan p = bwd_plan(f.T, f.N, f.H, f.Hkv, DK, DV, f.x, f.z != nullptr, f.window, f.sinks);
    k.window = p.window;
    k.sinks = p.sinks;
    char* ws = static_cast<char*>(a.ws);
    k.stats = reinterpret_cast<float2*>(ws);
    k.dog = f.z != nullptr ? static_cast<void*>(ws + p.dog) : const_cast<void*>(a.dy);
    k.parts = p.parts.key;
    k.q_parts = p.parts.query;
    k.part = reinterpret_cast<float*>(ws + p.part);
    k.q_part = reinterpret_cast<float*>(ws + p.q_part);
    if constexpr (kWin) {
        k.far_buckets = p.far.buckets;
        k.far_tiles = p.far.tiles;
        k.far_parts = p.far.parts;
        k.far = reinterpret_cast<float*>(ws + p.far_sums);
    }
    constexpr int lds = DqSizes<T, DK, DV>::kLds > DkvSizes<T, DK, DV>::kLds ? DqSizes<T, DK, DV>::kLds : DkvSizes<T, DK, DV>::kLds;
    hipError_t e = allow_lds(attn_bwd_kernel<T, DK, DV, kWin, kTileRows>, lds);
    if (e != hipSuccess) return e;
    {
        LaunchTimer timer("attn_bwd_rows", s);
        const int64_t blocks = (f.T * f.H + kThreads / 16 - 1) / (kThreads / 16);
        attn_bwd_rows_kernel<T, DV><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s>>>(k);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t tiles = attn_tiles(f.T, f.N, kRows);
    {
        LaunchTimer timer(kWin ? "attn_window_bwd" : "attn_bwd", s);
        const int64_t key_groups = tiles * f.Hkv * k.parts, far_groups = k.far_buckets * k.far_tiles * f.Hkv * k.far_parts;
        const int64_t query_groups = attn_tiles(f.T, f.N, kTileRows) * (f.H / (kRows / kTileRows)) * k.q_parts;
        attn_bwd_kernel<T, DK, DV, kWin, kTileRows><<<dim3(static_cast<unsigned>(far_groups + key_groups + query_groups)), dim3(kThreads), lds, s>>>(
            k, static_cast<unsigned>(key_groups), static_cast<unsigned>(far_groups));
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (k.parts > 1 || k.q_parts > 1) {
        LaunchTimer timer("attn_bwd_sum", s);
        const int64_t threads = (k.parts > 1 ? f.T * f.Hkv * ((DK + DV) / 4) : 0) + (k.q_parts > 1 ? f.T * f.H * (DK / 4) : 0);
        attn_bwd_sum_kernel<T, DK, DV, kWin><<<dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(k);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if constexpr (kWin) {
        if (k.far_parts > 0 && k.parts == 1) {
            LaunchTimer timer("attn_window_bwd_far_sum", s);
            const int64_t threads = k.far_buckets * k.sinks * f.Hkv * ((DK + DV) / 4);
            attn_bwd_far_sum_kernel<T, DK, DV><<<dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(k);
        }
    }
    return hipGetLastError();
}

}  // namespace

size_t attn_backward_workspace_bytes(int64_t T, int N, int H, int Hkv, int dk, int dv, DT x, bool gate, int window, int sinks) {
    return bwd_plan(T, N, H, Hkv, dk, dv, x, gate, window, sinks).bytes;
}

// More tokens have fewer parts, so what a call needs does not rise with its
// sizes (but for a window's, as far as it holds them all).  One sequence has the
// fewest tiles and so the most parts; of the lengths of as many tiles, of 32 rows
// or 128, the longest needs the most; from kKeyWant tiles on
// there is one part.  The far sums' parts fall as their rows rise: p parts of r
// rows are at most kMostFarParts r and at most kFarRows or r.  Of more first
// tokens than a tile's reach, the call of just that many tokens alone has far
// sums, in one part.
size_t attn_backward_max_workspace_bytes(int64_t T, int H, int Hkv, int dk, int dv, DT x, bool gate, int window, int sinks) {
    size_t most = attn_backward_workspace_bytes(T, 1, H, Hkv, dk, dv, x, gate, window, 0);
    for (int64_t t = 31; t < T && t < static_cast<int64_t>(kKeyWant) * kRows; t += 32) {
        const size_t need = attn_backward_workspace_bytes(t, 1, H, Hkv, dk, dv, x, gate, window, 0);
        most = need > most ? need : most;
    }
    const int64_t reach = static_cast<int64_t>(window) + kRows;
    if (window < 1 || sinks < 1 || T < reach) return most;
    int64_t rows = sinks > reach ? reach : T / reach * sinks;
    if (rows > most_far_rows(Hkv, dk + dv)) rows = most_far_rows(Hkv, dk + dv);
    const int64_t parts = sinks > reach || rows > kFarRows ? rows : rows * kMostFarParts < kFarRows ? rows * kMostFarParts : kFarRows;
    return most + up256(static_cast<size_t>(rows + parts) * Hkv * (dk + dv) * 4);
}

hipError_t launch_attn_prefill_backward(const AttnBackwardArgs& a, hipStream_t s) {
    if (a.f.T == 0) return hipSuccess;
    return attn_dispatch(a.f.x, a.f.dk, a.f.dv, [&](auto t, auto dk, auto dv) {
        using X = typename decltype(t)::type;
        constexpr int kDk = decltype(dk)::value, kDv = decltype(dv)::value;
        if (a.f.window > 0 && heads_share(a.f.H, a.f.Hkv)) return launch_bwd<X, kDk, kDv, true, 32>(a, s);
        return a.f.window > 0 ? launch_bwd<X, kDk, kDv, true, kRows>(a, s) : launch_bwd<X, kDk, kDv, false, kRows>(a, s);
    });
}

}  // namespace kda
