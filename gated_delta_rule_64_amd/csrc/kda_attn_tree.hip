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
};

template <typename T, int DK, int DV, int NQ>
struct TreeSizes {
    static constexpr int kTile = kKeys * (DK + DV) * static_cast<int>(sizeof(T)) + kTrSlack;
    static constexpr int kWaves = 4 * kTile <= 160 * 1024 ? 4 : 2;
    static constexpr int kVTiles = (DV + 31) / 32;
    static constexpr int kPart = NQ * kVTiles * 16 * 64 * 4;        // one wave's sums
    static constexpr int kJoin = kWaves / 2 * (kPart + NQ * 2 * 64 * 4);
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

__device__ __forceinline__ void wave_lds_fence() {
    // LDS operations of one wave complete in order; this keeps the compiler
    // from moving them past each other (lanes read what other lanes wrote)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename T, int DK, int DV, int NQ>
__global__ __launch_bounds__((64 * TreeSizes<T, DK, DV, NQ>::kWaves)) void attn_tree_kernel(TreeK a) {
    using Sz = TreeSizes<T, DK, DV, NQ>;
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
    int id = blockIdx.x;
    const int block = id % a.blocks;
    id /= a.blocks;
    const int split = id % a.splits;
    id /= a.splits;
    const int kvh = id % a.Hkv, b = id / a.Hkv;
    int slot, ctx = 0;
    const bool real = slot_of(a, b, slot, ctx);
    slot = uniform(slot);
    ctx = uniform(ctx);

    // this lane's rows (columns of the transposed scores)
    int row[NQ];
    int64_t q_at[NQ];  // index of the row in [B, T, H]
    bool mine[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        row[n] = (block * NQ + n) * 32 + c;
        mine[n] = row[n] < rows;
        const int r = mine[n] ? row[n] : 0;
        q_at[n] = (static_cast<int64_t>(b) * a.T + r / G) * a.H + kvh * G + r % G;
    }
    f32x16 acc[NQ][kVTiles];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int i = 0; i < kVTiles; ++i) acc[n][i] = f32x16{};
    }

    const int ctx_tiles = (ctx + kKeys - 1) / kKeys, tiles = ctx_tiles + (a.T + kKeys - 1) / kKeys;
    const int each = (tiles + a.splits - 1) / a.splits;
    const int t_end = real ? min(tiles, (split + 1) * each) : 0;
    int tile = split * each + wave;

    if (tile < t_end) {
        u32x4 qf[NQ][kQPieces];
        uint64_t seen[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const char* src = static_cast<const char*>(a.q) + q_at[n] * kKRow + half * 16;
#pragma unroll
            for (int p = 0; p < kQPieces; ++p) qf[n][p] = *reinterpret_cast<const u32x4*>(src + p * 32);
            const int t = (mine[n] ? row[n] : 0) / G;
            seen[n] = a.mask != nullptr ? static_cast<uint64_t>(a.mask[static_cast<int64_t>(b) * a.T + t])
                                        : ~0ull >> (63 - t);
        }
        const float sc = a.scale * kLog2e;

        // 16 rows of keys and of values in flight, as 16-byte pieces; twice a tile
        constexpr int kKEach = (16 * kKRow / 16 + 63) / 64, kVEach = (16 * kVRow / 16 + 63) / 64;
        u32x4 kr[2][kKEach], vr[2][kVEach];
        int there[2];  // rows of each half tile that hold a token (whole wave)
        auto fetch = [&](int n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                __amdgpu_buffer_rsrc_t ks, vs;
                int k_step = kKRow, v_step = kVRow;
                if (n < ctx_tiles) {
                    const int t0 = n * kKeys + 16 * x;
                    int got = min(16, max(0, ctx - t0));
                    int page = 0;
                    if (got > 0) {
                        page = a.table[static_cast<int64_t>(slot) * a.max_pages + (t0 >> a.page_shift)];
                        if (page < 0 || page >= a.pages) got = 0;  // no such page: its tokens are not there
                    }
                    got = uniform(got);
                    page = uniform(got > 0 ? page : 0);
                    const int64_t first = ((static_cast<int64_t>(page) * a.Hkv + kvh) << a.page_shift) + (t0 & ((1 << a.page_shift) - 1));
                    there[x] = got;
                    ks = rows_of(a.k_cache, first, kKRow, got);
                    vs = rows_of(a.v_cache, first, kVRow, got);
                } else {
                    const int t0 = (n - ctx_tiles) * kKeys + 16 * x;
                    there[x] = min(16, max(0, a.T - t0));
                    const int64_t first = static_cast<int64_t>(b) * a.T + t0;
                    k_step = kKRow * a.Hkv;
                    v_step = kVRow * a.Hkv;
                    // bounded to the rows of this head: the last one ends inside its token's row
                    const char* kb = static_cast<const char*>(a.k_new) + first * k_step + kvh * kKRow;
                    const char* vb = static_cast<const char*>(a.v_new) + first * v_step + kvh * kVRow;
                    ks = rows_of(kb, 0, k_step, there[x]);
                    vs = rows_of(vb, 0, v_step, there[x]);
                }
#pragma unroll
                for (int i = 0; i < kKEach; ++i) {
                    const int p = lane + 64 * i, r = p / (kKRow / 16);
                    kr[x][i] = r < there[x] ? buffer_load16(ks, r * k_step + p % (kKRow / 16) * 16) : u32x4{};
                }
#pragma unroll
                for (int i = 0; i < kVEach; ++i) {
                    const int p = lane + 64 * i, r = p / (kVRow / 16);
                    vr[x][i] = r < there[x] ? buffer_load16(vs, r * v_step + p % (kVRow / 16) * 16) : u32x4{};
                }
            }
        };
        // fp32 tiles are twice as large and do not fit beside the sums: they
        // are fetched when they are stored
        constexpr bool kAhead = kE == 2 && (NQ == 1 || DK < 128);
        if (kAhead) fetch(tile);
        for (; tile < t_end; tile += kWaves) {
            if (!kAhead) fetch(tile);
            wave_lds_fence();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int i = 0; i < kKEach; ++i) {
                    const int p = lane + 64 * i;
                    if (p < 16 * kKRow / 16)
                        *reinterpret_cast<u32x4*>(sK + (16 * x + p / (kKRow / 16)) * kKRow +
                                                  (p % (kKRow / 16) ^ turn<kKRow / 16>(p / (kKRow / 16))) * 16) = kr[x][i];
                }
#pragma unroll
                for (int i = 0; i < kVEach; ++i) {
                    const int p = lane + 64 * i;
                    if (p < 16 * kVRow / 16)
                        *reinterpret_cast<u32x4*>(sV + (16 * x + p / (kVRow / 16)) * kVRow +
                                                  (p % (kVRow / 16) ^ turn<kVRow / 16>(p / (kVRow / 16))) * 16) = vr[x][i];
                }
            }
            const int n0 = there[0], n1 = there[1];
            const bool draft = tile >= ctx_tiles;
            const int draft0 = (tile - ctx_tiles) * kKeys;
            if (kAhead && tile + kWaves < t_end) fetch(tile + kWaves);
            wave_lds_fence();

#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                f32x16 s{};
#pragma unroll
                for (int p = 0; p < kQPieces; ++p) s = mma<T>(rk.rows(sK, p), qf[n][p], s);
                if (draft) {
                    const uint64_t bits = seen[n] >> draft0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = 8 * (r / 4) + 4 * half + r % 4;
                        if (draft0 + key >= a.T || (bits >> key & 1) == 0) s[r] = -INFINITY;
                    }
                } else if (n0 + n1 < kKeys) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = 8 * (r / 4) + 4 * half + r % 4;
                        if (key - (r >= 8 ? 16 : 0) >= (r >= 8 ? n1 : n0)) s[r] = -INFINITY;
                    }
                }
                float top = s[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
                top = fmaxf(xor32_max(top), m[n]);
                const float alpha = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[n] - top) * sc);
                m[n] = top;
                const float ms = top == -INFINITY ? 0.f : top * sc;
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], sc, -ms));
                    sum += s[r];
                }
                l[n] = l[n] * alpha + sum;
#pragma unroll
                for (int i = 0; i < kVTiles; ++i) acc[n][i] *= alpha;
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const u32x4 x = as_operand<T>(s, p);
#pragma unroll
                    for (int i = 0; i < kVTiles; ++i)
                        acc[n][i] = mma<T>(rv.columns(sV, i, p), x, acc[n][i]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) l[n] = xor32_add(l[n]);

    // join the waves, the upper half of them into the lower, until one is left
    __syncthreads();
    const float sc = a.scale * kLog2e;
    for (int left = kWaves / 2; left >= 1; left /= 2) {
        char* at = smem + (wave % left) * (Sz::kPart + NQ * 2 * 64 * 4);
        float* stats = reinterpret_cast<float*>(at + Sz::kPart);
        if (wave >= left && wave < 2 * left) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4)
                        *reinterpret_cast<f32x4*>(at + (((n * kVTiles + i) * 4 + r4) * 64 + lane) * 16) =
                            f32x4{acc[n][i][4 * r4], acc[n][i][4 * r4 + 1], acc[n][i][4 * r4 + 2], acc[n][i][4 * r4 + 3]};
                stats[(2 * n) * 64 + lane] = m[n];
                stats[(2 * n + 1) * 64 + lane] = l[n];
            }
        }
        __syncthreads();
        if (wave < left) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float mo = stats[(2 * n) * 64 + lane], lo = stats[(2 * n + 1) * 64 + lane];
                const float top = fmaxf(m[n], mo);
                const float fa = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[n] - top) * sc);
                const float fb = mo == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((mo - top) * sc);
                m[n] = top;
                l[n] = l[n] * fa + lo * fb;
#pragma unroll
                for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) {
                        const f32x4 o = *reinterpret_cast<const f32x4*>(at + (((n * kVTiles + i) * 4 + r4) * 64 + lane) * 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[n][i][4 * r4 + e] = acc[n][i][4 * r4 + e] * fa + o[e] * fb;
                    }
            }
        }
        __syncthreads();
    }
    if (wave != 0) return;

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        if (!mine[n]) continue;
        if (a.splits > 1) {
            if (!real) continue;  // the joining kernel writes padding rows
            const int64_t at = ((static_cast<int64_t>(split) * a.B + b) * a.Hkv + kvh) * rows + row[n];
            if (half == 0) {
                a.stats[2 * at] = m[n];
                a.stats[2 * at + 1] = l[n];
            }
            if (l[n] > 0.f) {
#pragma unroll
                for (int i = 0; i < kVTiles; ++i)
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) {
                        const int ch = 32 * i + 8 * r4 + 4 * half;
                        if (ch < DV)
                            *reinterpret_cast<f32x4*>(a.part + at * DV + ch) =
                                f32x4{acc[n][i][4 * r4], acc[n][i][4 * r4 + 1], acc[n][i][4 * r4 + 2], acc[n][i][4 * r4 + 3]};
                    }
            }
            continue;
        }
        const float inv = l[n] > 0.f ? 1.f / l[n] : 0.f;
        if (a.lse != nullptr && half == 0)
            a.lse[q_at[n]] = l[n] > 0.f ? (m[n] * sc + __builtin_amdgcn_logf(l[n])) * kLn2 : -INFINITY;
        T* out = static_cast<T*>(a.out) + q_at[n] * DV;
        const T* z = a.z != nullptr && real ? static_cast<const T*>(a.z) + q_at[n] * DV : nullptr;
#pragma unroll
        for (int i = 0; i < kVTiles; ++i)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int ch = 32 * i + 8 * r4 + 4 * half;
                if (ch >= DV) continue;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = acc[n][i][4 * r4 + e] * inv;
                store4<T>(out + ch, z != nullptr ? z + ch : nullptr, y);
            }
    }
}

// Joins the parts of one row per wave: lanes of half h take the splits of
// that parity, four channels each.
template <typename T, int DV>
__global__ __launch_bounds__(256) void attn_tree_join_kernel(TreeK a) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + uniform(threadIdx.x >> 6);
    const int64_t total = static_cast<int64_t>(a.B) * a.T * a.H;
    if (r >= total) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, ch = (lane & 31) * 4;
    const int G = a.H / a.Hkv, rows = a.T * G;
    const int h = static_cast<int>(r % a.H), t = static_cast<int>(r / a.H % a.T), b = static_cast<int>(r / a.H / a.T);
    const int64_t at = (static_cast<int64_t>(b) * a.Hkv + h / G) * rows + t * G + h % G;
    const int64_t step = static_cast<int64_t>(a.B) * a.Hkv * rows;
    int slot, ctx;
    const bool real = slot_of(a, b, slot, ctx);
    const float sc = a.scale * kLog2e;
    float top = -INFINITY;
    if (real)
        for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.stats[2 * (at + s * step)]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
    if (top != -INFINITY) {
        for (int s = half; s < a.splits; s += 2) {
            const int64_t p = at + s * step;
            const float lp = a.stats[2 * p + 1];
            if (!(lp > 0.f)) continue;
            const float f = __builtin_amdgcn_exp2f((a.stats[2 * p] - top) * sc);
            l += lp * f;
            if (ch < DV) {
                const f32x4 o = *reinterpret_cast<const f32x4*>(a.part + p * DV + ch);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += o[e] * f;
            }
        }
    }
    l = xor32_add(l);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = xor32_add(y[e]);
    if (half != 0) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
    if (a.lse != nullptr && lane == 0) a.lse[r] = l > 0.f ? (top * sc + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    if (ch < DV)
        store4<T>(static_cast<T*>(a.out) + r * DV + ch,
                  a.z != nullptr && real ? static_cast<const T*>(a.z) + r * DV + ch : nullptr, y);
}

// Whether a wave can take two blocks of 32 rows: their sums and queries fit
// the registers beside a tile in flight.
constexpr bool two_blocks(int dk, DT x) { return x == DT::BF16 && dk <= 128; }

// Row blocks and splits of a call.
struct TreePlan {
    int nq, blocks, splits;
};
TreePlan tree_plan(int B, int T, int H, int Hkv, int dk, DT x, int64_t max_ctx) {
    const int64_t rows = static_cast<int64_t>(T) * (H / Hkv);
    TreePlan p;
    p.nq = rows > 32 && two_blocks(dk, x) ? 2 : 1;
    p.blocks = static_cast<int>((rows + 32 * p.nq - 1) / (32 * p.nq));
    const int64_t units = static_cast<int64_t>(B) * Hkv * p.blocks;
    const int64_t tiles = (max_ctx + kKeys - 1) / kKeys + (T + kKeys - 1) / kKeys;
    int64_t s = (1024 + units - 1) / units;
    if (s > tiles / 8) s = tiles / 8;  // two tiles a wave at least
    p.splits = static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    return p;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename T, int DK, int DV, int NQ>
hipError_t launch_nq(const TreeK& k, hipStream_t s) {
    using Sz = TreeSizes<T, DK, DV, NQ>;
    static_assert(Sz::kLds <= 160 * 1024, "one workgroup's LDS");
    auto fn = attn_tree_kernel<T, DK, DV, NQ>;
    if (Sz::kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, Sz::kLds);
        if (e != hipSuccess) return e;
    }
    LaunchTimer timer("attn_tree", s);
    const int64_t groups = static_cast<int64_t>(k.B) * k.Hkv * k.blocks * k.splits;
    fn<<<dim3(static_cast<unsigned>(groups)), dim3(64 * Sz::kWaves), Sz::kLds, s>>>(k);
    return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t launch_tree(const TreeArgs& a, hipStream_t s) {
    const TreePlan p = tree_plan(a.B, a.T, a.H, a.Hkv, DK, a.x, static_cast<int64_t>(a.max_pages) << a.page_shift);
    const size_t parts = static_cast<size_t>(p.splits) * a.B * a.T * a.H;
    float* part = static_cast<float*>(a.ws);
    float* stats = reinterpret_cast<float*>(static_cast<char*>(a.ws) + up256(parts * DV * 4));
    const TreeK k{a.B, a.T, a.H, a.Hkv, a.scale, a.q, a.k_new, a.v_new, a.z, a.mask, a.k_cache, a.v_cache,
                  a.pages, a.page_shift, a.table, a.slots, a.max_pages, a.lens, a.slot_indices, a.out, a.lse,
                  part, stats, p.splits, p.blocks};
    hipError_t e = hipErrorInvalidValue;
    if constexpr (two_blocks(DK, sizeof(T) == 2 ? DT::BF16 : DT::F32)) {
        if (p.nq == 2) e = launch_nq<T, DK, DV, 2>(k, s);
    }
    if (p.nq == 1) e = launch_nq<T, DK, DV, 1>(k, s);
    if (e != hipSuccess || p.splits == 1) return e;
    LaunchTimer timer("attn_tree_join", s);
    const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.H;
    attn_tree_join_kernel<T, DV><<<dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

size_t attn_tree_workspace_bytes(int B, int T, int H, int Hkv, int dk, int dv, DT x, int64_t max_ctx) {
    if (B == 0 || T == 0) return 0;
    const TreePlan p = tree_plan(B, T, H, Hkv, dk, x, max_ctx);
    if (p.splits == 1) return 0;
    const size_t parts = static_cast<size_t>(p.splits) * B * T * H;
    return up256(parts * dv * 4) + up256(parts * 8);
}

hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t s) {
    if (a.B == 0 || a.T == 0) return hipSuccess;
    return attn_dispatch(a.x, a.dk, a.dv, [&](auto t, auto dk, auto dv) {
        return launch_tree<typename decltype(t)::type, decltype(dk)::value, decltype(dv)::value>(a, s);
    });
}

}  // namespace kda
