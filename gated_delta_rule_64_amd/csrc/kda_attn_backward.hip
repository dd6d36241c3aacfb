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
};

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
// keys); a wave's queries, output gradients and sums stay in its registers, the
// keys and values pass through LDS once for four waves.
template <typename T, int DK, int DV>
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
    const int64_t rank = block / (a.H * a.q_parts);
    const int slot = block % (a.H * a.q_parts) / a.q_parts, part = block % a.q_parts;
    const int kvh = slot % a.Hkv, h = kvh * G + slot / a.Hkv;
    const Tile t = find_tile<kRows>(a.cu, a.N, a.T, rank);
    if (!t.there) return;
    const int q0 = t.level * kRows + wave * 32;
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
    const int64_t steps = (min(t.level * kRows + kRows, t.len) + kKeys - 1) / kKeys;  // keys [0, steps kKeys) are attended by some row
    const int start = static_cast<int>(steps * part / a.q_parts) * kKeys;
    const int last = static_cast<int>(steps * (part + 1) / a.q_parts) * kKeys;
    const T* kbase = static_cast<const T*>(a.k) + kvh * DK;
    const T* vbase = static_cast<const T*>(a.v) + kvh * DV;
    auto fetch = [&](int j0) {
        ck.load(rows_of(kbase, t.start + j0, k_row, min(kKeys, t.len - j0)), k_row, tid);
        cv.load(rows_of(vbase, t.start + j0, v_row, min(kKeys, t.len - j0)), v_row, tid);
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
    for (int j0 = start; j0 < last; j0 += 2 * kKeys) {
        tile_barrier();
        if (j0 + kKeys < last) fetch(j0 + kKeys);
        work(smem, j0);
        if (j0 + kKeys >= last) break;
        put(smem + Sz::kBuf);
        tile_barrier();
        if (j0 + 2 * kKeys < last) fetch(j0 + 2 * kKeys);
        work(smem + Sz::kBuf, j0 + kKeys);
        if (j0 + 2 * kKeys < last) put(smem);
    }
    if (c >= rows) return;
    if (a.q_parts > 1)
        store_rows<float, DK>(a.q_part + (static_cast<int64_t>(part) * a.T * a.H + at) * DK, acc, a.scale, half);
    else
        store_rows<T, DK>(static_cast<T*>(a.dq) + at * DK, acc, a.scale, half);
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
template <typename T, int DK, int DV>
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
    const int64_t rank = block / (a.Hkv * a.parts);
    const int slot = block % (a.Hkv * a.parts);
    const int kvh = slot % a.Hkv, part = slot / a.Hkv;
    const Tile t = find_tile<kRows>(a.cu, a.N, a.T, rank);
    if (!t.there) return;
    // the first keys of a sequence have the most queries: levels from the end
    const int k_first = (t.tiles - 1 - t.level) * kRows;
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
    const int steps = (t.len - k_first + kQ - 1) / kQ;  // per head
    const int64_t all = static_cast<int64_t>(steps) * G;
    int n = static_cast<int>(all * part / a.parts);
    const int n_end = static_cast<int>(all * (part + 1) / a.parts);
    int f_head = uniform(kvh * G + n / steps), f_i0 = uniform(k_first + n % steps * kQ);  // the next step to fetch
    auto fetch = [&]() __attribute__((always_inline)) {
        const int here = min(kQ, t.len - f_i0);
        cq.load(rows_of(static_cast<const T*>(a.q) + f_head * DK, t.start + f_i0, q_row, here), q_row, tid);
        co.load(rows_of(static_cast<const T*>(a.dog) + f_head * DV, t.start + f_i0, o_row, here), o_row, tid);
        // rows behind the sequence's end are 0 in all three and add nothing
        if (wave == 0)
            stat = buffer_load8(rows_of(a.stats + f_head, t.start + f_i0, a.H * 8, here), c * a.H * 8);
        f_i0 += kQ;
        if (f_i0 >= t.len) {
            f_i0 = k_first;
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
        i0 = i0 + kQ < t.len ? i0 + kQ : k_first;
        if (i0 + kQ - 1 < k0) return;  // queries before this wave's keys
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
    if (c < rows) {
        const int64_t at = (t.start + k0 + c) * a.Hkv + kvh;
        if (a.parts > 1) {
            float* to = a.part + (static_cast<int64_t>(part) * a.T * a.Hkv + at) * (DK + DV);
            store_rows<float, DK>(to, gk, a.scale, half);
            store_rows<float, DV>(to + DK, gv, 1.f, half);
        } else {
            store_rows<T, DK>(static_cast<T*>(a.dk) + at * DK, gk, a.scale, half);
            store_rows<T, DV>(static_cast<T*>(a.dv) + at * DV, gv, 1.f, half);
        }
    }
}

// Both in one launch, the key gradients' workgroups first: they are the longer
// ones, and the query gradients' fill the chip behind them (one after the
// other, each launch ends with most of the chip idle: the small fp32 batch
// takes 55 + 59 us so).  Rows of up to 256 bytes leave registers for two
// workgroups a CU (fp32 at 64 channels: 4,000 tokens 1,900 us, 2,180 with one;
// the ragged batch of up to 1,000 tokens 301 us, 355 with one).
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads, (DK * sizeof(T) <= 256 ? 2 : 1)) void attn_bwd_kernel(BwdK a, unsigned key_groups) {
    extern __shared__ __align__(16) char smem[];
    if (blockIdx.x < key_groups) key_gradients<T, DK, DV>(a, blockIdx.x, smem);
    else query_gradients<T, DK, DV>(a, blockIdx.x - key_groups, smem);
}

// Adds the parts in their order, four channels per thread: first the rows of
// the key heads (dk and dv together), then those of the query heads.  Bound by
// memory: four parts of 4,096 tokens of 8 heads, 151 MB, in 23 us (6.6 TB/s,
// a part of it from the caches).
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void attn_bwd_sum_kernel(BwdK a) {
    constexpr int kKv = (DK + DV) / 4, kQ = DK / 4;
    const int64_t tokens = a.cu == nullptr ? a.T : min(static_cast<int64_t>(max(a.cu[a.N], 0)), a.T);
    const int64_t kv_all = a.parts > 1 ? tokens * a.Hkv * kKv : 0, q_all = a.q_parts > 1 ? tokens * a.H * kQ : 0;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    auto add = [&](const float* from, int64_t step, int parts, float (&sum)[4]) {
        for (int p = 0; p < parts; ++p) {
            float x[4];
            ld4(from + p * step, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += x[e];
        }
    };
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < kv_all) {
        const int64_t row = i / kKv;
        const int ch = static_cast<int>(i % kKv) * 4;
        add(a.part + row * (DK + DV) + ch, a.T * a.Hkv * (DK + DV), a.parts, sum);
        if (ch < DK) st4(static_cast<T*>(a.dk) + row * DK + ch, sum);
        else st4(static_cast<T*>(a.dv) + row * DV + ch - DK, sum);
        return;
    }
    i -= kv_all;
    if (i >= q_all) return;
    add(a.q_part + i * 4, a.T * a.H * DK, a.q_parts, sum);
    st4(static_cast<T*>(a.dq) + i * 4, sum);
}

// Into how many parts the work of a tile is cut: key tiles so that their
// workgroups, which differ in length, fill the chip several times; query tiles
// where they and the key tiles' together leave it half empty.
constexpr int kKeyWant = 1024, kQueryWant = 384;  // workgroups below which tiles are cut
struct BwdParts {
    int key, query;
};
BwdParts bwd_parts(int64_t T, int N, int H, int Hkv) {
    const int64_t tiles = attn_tiles(T, N, kRows), keys = tiles * Hkv, queries = tiles * H;
    if (tiles == 0) return {1, 1};
    auto parts = [](int64_t want, int64_t units, int64_t most) {
        const int64_t p = (want + units - 1) / units;
        return static_cast<int>(p < 1 ? 1 : p > most ? most : p);
    };
    return {parts(kKeyWant, keys, kMostParts), parts(kQueryWant, queries, kMostParts / 2)};
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename F>
hipError_t allow_lds(F fn, int lds) {
    if (lds <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <typename T, int DK, int DV>
hipError_t launch_bwd(const AttnBackwardArgs& a, hipStream_t s) {
    const AttnArgs& f = a.f;
    BwdK k{};
    k.T = f.T; k.H = f.H; k.Hkv = f.Hkv; k.N = f.N; k.cu = f.cu;
    k.q = f.q; k.k = f.k; k.v = f.v; k.z = f.z; k.out = f.out; k.dy = a.dy; k.lse = f.lse;
    k.dq = a.dq; k.dk = a.dk; k.dv = a.dv; k.dz = a.dz; k.scale = f.scale;
    char* ws = static_cast<char*>(a.ws);
    k.stats = reinterpret_cast<float2*>(ws);
    ws += up256(static_cast<size_t>(f.T) * f.H * 8);
    k.dog = f.z != nullptr ? static_cast<void*>(ws) : const_cast<void*>(a.dy);
    if (f.z != nullptr) ws += up256(static_cast<size_t>(f.T) * f.H * DV * sizeof(T));
    const BwdParts parts = bwd_parts(f.T, f.N, f.H, f.Hkv);
    k.parts = parts.key;
    k.q_parts = parts.query;
    k.part = reinterpret_cast<float*>(ws);
    if (k.parts > 1) ws += up256(static_cast<size_t>(k.parts) * f.T * f.Hkv * (DK + DV) * 4);
    k.q_part = reinterpret_cast<float*>(ws);
    constexpr int lds = DqSizes<T, DK, DV>::kLds > DkvSizes<T, DK, DV>::kLds ? DqSizes<T, DK, DV>::kLds : DkvSizes<T, DK, DV>::kLds;
    hipError_t e = allow_lds(attn_bwd_kernel<T, DK, DV>, lds);
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
        LaunchTimer timer("attn_bwd", s);
        const int64_t key_groups = tiles * f.Hkv * k.parts;
        attn_bwd_kernel<T, DK, DV><<<dim3(static_cast<unsigned>(key_groups + tiles * f.H * k.q_parts)), dim3(kThreads), lds, s>>>(
            k, static_cast<unsigned>(key_groups));
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (k.parts > 1 || k.q_parts > 1) {
        LaunchTimer timer("attn_bwd_sum", s);
        const int64_t threads = (k.parts > 1 ? f.T * f.Hkv * ((DK + DV) / 4) : 0) + (k.q_parts > 1 ? f.T * f.H * (DK / 4) : 0);
        attn_bwd_sum_kernel<T, DK, DV><<<dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(k);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipGetLastError();
}

}  // namespace

size_t attn_backward_workspace_bytes(int64_t T, int N, int H, int Hkv, int dk, int dv, DT x, bool gate) {
    const size_t rows = static_cast<size_t>(T) * H;
    const BwdParts parts = bwd_parts(T, N, H, Hkv);
    return up256(rows * 8) + (gate ? up256(rows * dv * (x == DT::BF16 ? 2 : 4)) : 0) +
           (parts.key > 1 ? up256(static_cast<size_t>(parts.key) * T * Hkv * (dk + dv) * 4) : 0) +
           (parts.query > 1 ? up256(static_cast<size_t>(parts.query) * rows * dk * 4) : 0);
}

// More tokens have fewer parts, so what a call needs does not rise with its
// sizes.  One sequence has the fewest tiles and so the most parts; of the
// lengths of as many tiles the longest needs the most; from kKeyWant tiles on
// there is one part.
size_t attn_backward_max_workspace_bytes(int64_t T, int H, int Hkv, int dk, int dv, DT x, bool gate) {
    size_t most = attn_backward_workspace_bytes(T, 1, H, Hkv, dk, dv, x, gate);
    for (int64_t t = kRows - 1; t < T && t < static_cast<int64_t>(kKeyWant) * kRows; t += kRows) {
        const size_t need = attn_backward_workspace_bytes(t, 1, H, Hkv, dk, dv, x, gate);
        most = need > most ? need : most;
    }
    return most;
}

hipError_t launch_attn_prefill_backward(const AttnBackwardArgs& a, hipStream_t s) {
    if (a.f.T == 0) return hipSuccess;
    return attn_dispatch(a.f.x, a.f.dk, a.f.dv, [&](auto t, auto dk, auto dv) {
        return launch_bwd<typename decltype(t)::type, decltype(dk)::value, decltype(dv)::value>(a, s);
    });
}

}  // namespace kda
