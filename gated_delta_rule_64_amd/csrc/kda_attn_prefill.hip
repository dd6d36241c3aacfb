// Causal attention over packed prompts, grouped heads, optional output gate.
//
//   s_ij = scale q_i . k_j (j <= i, same sequence),  m_i = max_j s_ij,
//   l_i = sum_j e^(s_ij - m_i),  o_i = (1 / l_i) sum_j e^(s_ij - m_i) v_j,
//   y_i = o_i * sigmoid(z_i),    lse_i = m_i + log l_i
//
// One pass over the keys with the running maximum and sum.  The scores are
// formed transposed, S^T = K Q^T, so that a lane holds one query's scores (its
// softmax statistics need one exchange between the wave's halves, no shuffle
// tree) and P^T is the B operand of O^T += V^T P^T as it stands in registers.
//
// 128 rows of one head a workgroup, 32 a wave: the queries and sums of a wave
// fill its registers so that two workgroups share a CU, and a key tile read
// into LDS once serves four waves.  16,384 tokens of 32 heads of 128 over 8, in
// bf16: 2,090 to 2,170 us, 1,010 to 1,050 TFLOP/s (a large bf16 product of the
// library reaches 1,390); the matrix cores work in 53 % of the cycles, the vector
// units' softmax in 47 %.  Twelve ragged sequences of up to 2,048 tokens at
// 192/128 channels, gated: 326 to 341 us, 650 to 680 TFLOP/s, matrix cores 36 %,
// waits 28 %: such a batch also moves 0.69 GB (125 us), of which the queries, the
// gate and the results are not under the products (without a gate: 22 us less).
#include "kda_attn_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kQ = 32 * kWaves;  // query rows of a workgroup, 32 a wave

struct FwdK {
    int64_t T;
    int H, Hkv, N;
    const int32_t* cu;
    const void *q, *k, *v, *z;
    void* out;
    float* lse;
    float scale;
};

template <typename T, int DK, int DV>
struct FwdSizes {
    static constexpr int kKeys = DK > 128 || (sizeof(T) == 4 && DK > 64) ? 32 : 64;  // keys of a tile
    static constexpr int kBuf = kKeys * (DK + DV) * static_cast<int>(sizeof(T));
    static constexpr int kTiles = 2 * kBuf + tr_slack(DV), kRows = kWaves * 32 * DV * 4;
    static constexpr int kLds = kTiles > kRows ? kTiles : kRows;  // the results pass through the tiles' space
};

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 ? 2 : 1)) void attn_fwd_kernel(FwdK a) {
    using Sz = FwdSizes<T, DK, DV>;
    constexpr int kKeys = Sz::kKeys, kSub = kKeys / 32;
    constexpr int kQPieces = DK / (2 * Elem<T>::kPer16);  // operand pieces per lane of a query or key row
    constexpr int kVTiles = (DV + 31) / 32;
    constexpr int kP = Elem<T>::kPieces;
    extern __shared__ __align__(16) char smem[];
    constexpr int kV = kKeys * DK * static_cast<int>(sizeof(T));  // the values, behind the keys

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int G = a.H / a.Hkv;
    const int64_t rank = blockIdx.x / a.H;
    const int slot = blockIdx.x % a.H;
    const int kvh = slot % a.Hkv, h = kvh * G + slot / a.Hkv;
    const Tile t = find_tile<kQ>(a.cu, a.N, a.T, rank);
    if (!t.there) return;
    const int q0 = t.level * kQ + wave * 32;  // this wave's first row, in the sequence

    const int q_row = a.H * DK * static_cast<int>(sizeof(T));
    const int k_row = a.Hkv * DK * static_cast<int>(sizeof(T)), v_row = a.Hkv * DV * static_cast<int>(sizeof(T));
    u32x4 qf[kQPieces];
    {
        const auto src = rows_of(static_cast<const T*>(a.q) + h * DK, t.start + q0, q_row, min(32, t.len - q0));
#pragma unroll
        for (int s = 0; s < kQPieces; ++s) qf[s] = buffer_load16(src, c * q_row + (2 * s + half) * 16);
    }

    const float sc = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;  // m in units of raw scores
    f32x16 acc[kVTiles];
#pragma unroll
    for (int i = 0; i < kVTiles; ++i) acc[i] = f32x16{};

    TileCopy<T, kKeys, DK, kThreads> ck;
    TileCopy<T, kKeys, DV, kThreads> cv;
    TileRead<T, DK> rk;
    TileRead<T, DV> rv;
    rk.init_rows(c, half);
    rv.init_columns(lane);
    const int last = min(t.level * kQ + kQ, t.len);  // keys [0, last) are attended by some row
    const T* kbase = static_cast<const T*>(a.k) + kvh * DK;
    const T* vbase = static_cast<const T*>(a.v) + kvh * DV;
    auto fetch = [&](int j0) {
        ck.load(rows_of(kbase, t.start + j0, k_row, min(kKeys, t.len - j0)), k_row, tid);
        cv.load(rows_of(vbase, t.start + j0, v_row, min(kKeys, t.len - j0)), v_row, tid);
    };
    // Two tiles in LDS: while one is worked on, the next one's rows arrive in
    // registers and are stored behind it; one barrier a tile.
    auto put = [&](char* buf) {
        ck.store(buf, tid);
        cv.store(buf + kV, tid);
    };
    auto work = [&](const char* sK, int j0) __attribute__((always_inline)) {
        if (j0 > q0 + 31) return;  // nothing of the tile is attended by this wave's rows
        const char* sV = sK + kV;
        f32x16 s[kSub];
        // the wave that multiplies goes before the one that exponentiates
        // (2,158 to 2,136 us at 16,384 tokens)
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < kSub; ++u) s[u] = f32x16{};
#pragma unroll
        for (int p = 0; p < kQPieces; ++p)
#pragma unroll
            for (int u = 0; u < kSub; ++u) s[u] = mma<T>(rk.rows(sK + 32 * u * rk.kRow, p), qf[p], s[u]);
        lookahead<kQPieces * kSub, 4, Elem<T>::kMfmas>();
        __builtin_amdgcn_s_setprio(0);
        if (j0 + kKeys - 1 > q0) {  // the diagonal: keys behind the row's own are not attended
            const int most = opaque(q0 + c - j0 - 4 * half);
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * u + 8 * (r / 4) + r % 4 > most) s[u][r] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
        top = xor32_max(top);
        if (__any((top - m) * sc > kRise)) {  // m is -infinity at first
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
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[u][r] -= off;
            ms = 0.f;
        }
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], sc, -ms));
                sum += s[u][r];
            }
        l += sum;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const u32x4 b = as_operand<T>(s[u], p);
#pragma unroll
                for (int i = 0; i < kVTiles; ++i)
                    acc[i] = mma<T>(rv.columns(sV + 32 * u * rv.kRow, i, p), b, acc[i]);
            }
    };
    fetch(0);
    arrive(qf);
    put(smem);
    for (int j0 = 0; j0 < last; j0 += 2 * kKeys) {
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

    const int row = q0 + c;
    const int64_t first = (t.start + q0) * a.H + h;  // this wave's first row in [T, H]
    constexpr int kPer = Elem<T>::kPer16, kOut = 32 * DV / (64 * kPer), kRowPieces = DV / kPer;
    // the gate's logits, in flight while the results are laid out by rows
    u32x4 z[kOut];
    if (a.z != nullptr) {
        const auto src = rows_of(static_cast<const T*>(a.z) + h * DV, t.start + q0, a.H * DV * static_cast<int>(sizeof(T)), min(32, t.len - q0));
#pragma unroll
        for (int n = 0; n < kOut; ++n)
            z[n] = buffer_load16(src, (lane + 64 * n) / kRowPieces * (a.H * DV * static_cast<int>(sizeof(T))) + (lane + 64 * n) % kRowPieces * 16);
    }
    l = xor32_add(l);
    // A row attends itself at least.  A sum of NaN, or of 0 (every score is
    // -infinity), makes it and its lse NaN.
    const float inv = l > 0.f ? 1.f / l : NAN;
    if (a.lse != nullptr && half == 0 && row < t.len)
        a.lse[first + static_cast<int64_t>(c) * a.H] = l > 0.f ? (m * sc + __builtin_amdgcn_logf(l)) * kLn2 : NAN;
#pragma unroll
    for (int i = 0; i < kVTiles; ++i) acc[i] *= inv;
    tile_barrier();  // every wave is done with the tiles
    int n = 0;
    by_rows<T, DV>(smem + wave * 32 * DV * 4, acc, lane, [&](int r, int ch, auto& y) __attribute__((always_inline)) {
        if (a.z != nullptr) {
            float g[kPer];
            unpack_piece(z[n], g);
#pragma unroll
            for (int e = 0; e < kPer; ++e) y[e] *= sigmoid_fast(g[e]);
        }
        ++n;
        if (q0 + r < t.len) store_piece(static_cast<T*>(a.out) + (first + static_cast<int64_t>(r) * a.H) * DV + ch, y);
    });
}

template <typename T, int DK, int DV>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t s) {
    constexpr int lds = FwdSizes<T, DK, DV>::kLds;
    static_assert(lds <= 160 * 1024, "one workgroup's LDS");
    auto fn = attn_fwd_kernel<T, DK, DV>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const FwdK k{a.T, a.H, a.Hkv, a.N, a.cu, a.q, a.k, a.v, a.z, a.out, a.lse, a.scale};
    LaunchTimer timer("attn_fwd", s);
    fn<<<dim3(static_cast<unsigned>(attn_tiles(a.T, a.N, kQ) * a.H)), dim3(kThreads), lds, s>>>(k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    return attn_dispatch(a.x, a.dk, a.dv, [&](auto t, auto dk, auto dv) {
        return launch_fwd<typename decltype(t)::type, decltype(dk)::value, decltype(dv)::value>(a, s);
    });
}

}  // namespace kda
