// The attention weights that a sequence's last tokens give to its cached
// tokens, summed per cached token.
//
//   w_j += sum over queries i and heads h of e^(s_ijh - lse_ih),
//   s_ijh = scale q_ih . k_j(h / G), over the keys j that query i attends
//
// lse is what the attention call gave, so the weights need no statistics of
// their own: one pass over the keys, no values.  The scores are formed
// transposed (S^T = K Q^T, 32 keys by 32 rows of queries and heads), so that a
// lane's lse stays in one register and its 16 sums, one per key that it holds,
// are added over the lanes once per tile of keys, not once per product.
#include "kda_attn_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kKeys = 32;  // keys of a tile

struct WeighK {
    CacheArgs c;
    WeighArgs a;
    int splits;
};

// Sequence n's queries and its slot's tokens; false: nothing to do.
struct Weighed {
    int64_t first;  // its first query's index
    int count, slot, ctx;
};
__device__ __forceinline__ bool weighed(const WeighK& k, int n, Weighed& w) {
    seq_bounds(k.a.cu, n, k.a.tokens, w.first, w.count);
    w.slot = k.a.slot_indices != nullptr ? k.a.slot_indices[n] : n;
    if (w.count == 0 || w.slot < 0 || w.slot >= k.c.slots) return false;
    const int64_t most = static_cast<int64_t>(k.c.max_pages) << k.c.page_shift;
    const int len = k.c.lens[w.slot];
    w.ctx = len < 0 ? 0 : static_cast<int>(len > most ? most : len);
    w.slot = uniform(w.slot);
    w.ctx = uniform(w.ctx);
    w.count = uniform(w.count);
    w.first = uniform64(w.first);
    return w.ctx > 0;
}

// One workgroup per (sequence, part of its tiles): the waves share out the
// (key head, block of 32 rows) pairs of a tile, their sums are added in LDS.
template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void cache_weigh_kernel(WeighK k) {
    constexpr int kQPieces = DK / (2 * Elem<T>::kPer16);
    constexpr int kRow = DK * static_cast<int>(sizeof(T));
    __shared__ float sums[kWaves][kKeys];
    const CacheArgs& c = k.c;
    const WeighArgs& a = k.a;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int n = blockIdx.x / k.splits, split = blockIdx.x % k.splits;
    Weighed w;
    if (!weighed(k, n, w)) return;
    const int G = a.H / c.Hkv;
    const int64_t rows = static_cast<int64_t>(w.count) * G;  // of a key head
    const int p_first = w.ctx - w.count;  // the first query's place; below 0: it has no token
    const int low = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
    const int sinks = a.window > 0 ? min(a.sinks, w.ctx) : 0;
    const int sink_tiles = (sinks + kKeys - 1) / kKeys, skip = max(0, low / kKeys - sink_tiles);
    const int tiles = (w.ctx + kKeys - 1) / kKeys - skip;
    const int blocks = static_cast<int>((rows + 31) / 32);
    const int64_t items = static_cast<int64_t>(blocks) * c.Hkv;
    const int32_t* table = c.table + static_cast<int64_t>(w.slot) * c.max_pages;
    const float sc = a.scale * kLog2e;
    for (int tile = split; tile < tiles; tile += k.splits) {
        const int first = (tile >= sink_tiles ? tile + skip : tile) * kKeys;
        // the row of this lane's key
        const int pos = first + col;
        const int page = pos < w.ctx ? table[pos >> c.page_shift] : -1;
        const bool there = page >= 0 && page < c.pages;
        const int64_t at = ((static_cast<int64_t>(there ? page : 0) * c.Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
        f32x16 acc{};
        u32x4 kf[kQPieces];
        int kvh = -1;
        for (int64_t item = items * wave / kWaves; item < items * (wave + 1) / kWaves; ++item) {
            const int f = static_cast<int>(item / blocks), block = static_cast<int>(item % blocks);
            if (f != kvh) {
                kvh = f;
                const char* from = static_cast<const char*>(c.k_cache) + (at + (static_cast<int64_t>(kvh) << c.page_shift)) * kRow + half * 16;
#pragma unroll
                for (int p = 0; p < kQPieces; ++p) kf[p] = there ? *reinterpret_cast<const u32x4*>(from + p * 32) : u32x4{};
            }
            // this lane's row: a query and a head
            const int64_t r = static_cast<int64_t>(block) * 32 + col;
            const int token = static_cast<int>(min(r, rows - 1) / G), h = kvh * G + static_cast<int>(min(r, rows - 1) % G);
            const int64_t t = w.first + token;
            const int64_t src = a.rows != nullptr ? a.rows[t] : t;
            const int p_here = max(p_first + token, -1);
            bool on = r < rows && p_here >= 0 && src >= 0 && src < a.src_rows;
            const int64_t q_at = (on ? src : 0) * a.H + h;
            const float lse = on ? a.lse[q_at] : 0.f;
            on = on && fabsf(lse) < INFINITY;  // a row that attends nothing, or a broken one, weighs nothing
            const char* q_row = static_cast<const char*>(a.q) + q_at * kRow + half * 16;
            f32x16 s{};
#pragma unroll
            for (int p = 0; p < kQPieces; ++p) {
                const u32x4 q = on ? *reinterpret_cast<const u32x4*>(q_row + p * 32) : u32x4{};
                s = mma<T>(kf[p], q, s);
            }
            const float lse2 = lse * kLog2e;
            const int most = on ? p_here - first - 4 * half : INT32_MIN;
            const int least = a.window > 0 ? p_here - a.window + 1 - first - 4 * half : INT32_MIN, sink = sinks - first - 4 * half;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const int key = 8 * (x / 4) + x % 4;
                const float e = __builtin_amdgcn_exp2f(fmaf(s[x], sc, -lse2));
                acc[x] += key <= most && (key >= least || key < sink) ? e : 0.f;
            }
        }
        // over the lanes of a half: the rows of queries
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            float v = row_ror_add<1>(acc[x]);
            v = row_ror_add<2>(v);
            v = row_ror_add<4>(v);
            v = xor16_add(row_ror_add<8>(v));
            if (col == 0) sums[wave][8 * (x / 4) + 4 * half + x % 4] = v;
        }
        __syncthreads();
        if (threadIdx.x < kKeys && there) {  // (thread j holds key j's place)
            float v = 0.f;
#pragma unroll
            for (int x = 0; x < kWaves; ++x) v += sums[x][threadIdx.x];
            a.weights[(static_cast<int64_t>(w.slot) * c.max_pages << c.page_shift) + pos] += v;
        }
        __syncthreads();
    }
}

constexpr int kWantGroups = 2048;

template <typename T, int DK>
hipError_t launch_weigh(const CacheArgs& c, const WeighArgs& a, hipStream_t s) {
    const int64_t max_ctx = static_cast<int64_t>(c.max_pages) << c.page_shift;
    int64_t reach = max_ctx;
    if (a.window > 0) reach = window_reach(max_ctx, a.window, a.sinks) + a.tokens;
    if (reach > max_ctx) reach = max_ctx;
    const int64_t tiles = (reach + kKeys - 1) / kKeys, want = (kWantGroups + a.N - 1) / a.N;
    WeighK k{c, a, static_cast<int>(tiles < want ? tiles : want)};
    if (k.a.window >= max_ctx) k.a.window = 0;  // it holds every token
    LaunchTimer timer("cache_weigh", s);
    cache_weigh_kernel<T, DK><<<dim3(static_cast<unsigned>(static_cast<int64_t>(a.N) * k.splits)), dim3(kThreads), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

size_t cache_weigh_workspace_bytes(int64_t, int, int, int, int64_t) { return 0; }

hipError_t launch_cache_weigh(const CacheArgs& c, const WeighArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return attn_dispatch(c.x, c.dk, c.dk == 192 ? 128 : c.dk, [&](auto t, auto dk, auto) {
        return launch_weigh<typename decltype(t)::type, decltype(dk)::value>(c, a, s);
    });
}

}  // namespace kda
