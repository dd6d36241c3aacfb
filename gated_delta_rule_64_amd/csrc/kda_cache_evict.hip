// Slots of an attention cache cut down to their heaviest tokens.
//
// The tokens that stay are found by the value of the last one that stays (the
// m-th largest weight, digit by digit over the weights' bits), ties by a count
// in the tokens' order.  They then move to the front in that order: token d
// goes to a place that is not behind its own, so whoever walks them in order
// can move them where they are, as long as a step's reads come before its
// writes.
#include "kda_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

constexpr int kPlan = 1024;  // threads of a planning workgroup
constexpr int kMove = 256;   // threads of a moving workgroup

struct EvictK {
    CacheArgs c;
    EvictArgs a;
    int32_t* list;  // [n, keep]: places of the tokens that stay
    int32_t* plan;  // [n]: the first token that changes its place (-1: nothing to do)
};

__device__ __forceinline__ bool names_page(int32_t e, int pages) { return e >= 0 && e < pages; }

// A barrier behind loads whose places other threads write after it: every wave
// waits until its loads have arrived.
__device__ __forceinline__ void loaded_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// A weight as a whole number of the same order: NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (!(w == w)) return 0;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}

template <typename I>
__device__ __forceinline__ I block_scan(I x, I* sums, I& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    I inc = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const I y = __shfl_up(inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    I before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        const I s = sums[w];
        before += w < wave ? s : 0;
        all += s;
    }
    __syncthreads();
    total = all;
    return before + inc - x;
}

// One workgroup per entry: checks it, finds what stays, moves its weights.
__global__ __launch_bounds__(kPlan) void cache_evict_plan_kernel(EvictK k) {
    __shared__ int hist[256];
    __shared__ uint64_t sums[kPlan / 64];
    __shared__ int s_first, s_bad, s_digit, s_left;
    const CacheArgs& c = k.c;
    const EvictArgs& a = k.a;
    const int i = blockIdx.x, tid = threadIdx.x;
    const int slot = a.slot_list[i];
    int32_t* list = k.list + static_cast<int64_t>(i) * a.keep;
    int32_t* kept = a.kept != nullptr ? a.kept + static_cast<int64_t>(i) * a.keep : nullptr;
    if (tid == 0) {
        s_bad = slot < 0 || slot >= c.slots;
        s_first = INT32_MAX;
    }
    __syncthreads();
    // an earlier entry that names the slot has it
    for (int j = tid; j < i; j += kPlan)
        if (a.slot_list[j] == slot) s_bad = 1;
    __syncthreads();
    bool bad = s_bad != 0;
    int len = 0;
    const int32_t* table = nullptr;
    if (!bad) {
        const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
        const int n = c.lens[slot];
        len = n < 0 ? 0 : static_cast<int>(n > most ? most : n);
        table = c.table + static_cast<int64_t>(slot) * c.max_pages;
    }
    const bool cut = !bad && len > a.keep;
    if (cut) {  // every token has a page
        for (int j = tid; j < (len + (1 << c.page_shift) - 1) >> c.page_shift; j += kPlan)
            if (!names_page(table[j], c.pages)) s_bad = 1;
    }
    __syncthreads();
    bad = s_bad != 0;
    if (bad || !cut) {
        if (kept != nullptr)
            for (int d = tid; d < a.keep; d += kPlan) kept[d] = !bad && d < len ? d : -1;
        if (tid == 0) {
            k.plan[i] = -1;
            if (a.status != nullptr) a.status[i] = bad ? 2 : 0;
        }
        return;
    }
    float* w = a.weights + (static_cast<int64_t>(slot) * c.max_pages << c.page_shift);
    // the places between the first and the most recent ones, of which `left` stay
    const int from = a.first, to = len - a.recent;
    int left = a.keep - a.first - a.recent;
    uint32_t known = 0;
    if (left > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int b = tid; b < 256; b += kPlan) hist[b] = 0;
            __syncthreads();
            for (int p = from + tid; p < to; p += kPlan) {
                const uint32_t o = order_of(w[p]);
                if (shift == 24 || o >> (shift + 8) == known >> (shift + 8)) atomicAdd(&hist[o >> shift & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int rest = left, b = 255;
                while (b > 0 && hist[b] < rest) rest -= hist[b--];
                s_digit = b;
                s_left = rest;
            }
            __syncthreads();
            known |= static_cast<uint32_t>(s_digit) << shift;
            left = s_left;
        }
    }
    // `left` of those whose order is `known` stay, the first ones, and all above it
    const bool some = a.keep > a.first + a.recent;
    uint64_t before = 0;  // above it or protected (high half), equal to it (low half)
    for (int p0 = 0; p0 < len; p0 += kPlan) {
        const int p = p0 + tid;
        uint64_t x = 0;
        if (p < len) {
            if (p < from || p >= to) {
                x = 1ull << 32;
            } else if (some) {
                const uint32_t o = order_of(w[p]);
                x = o > known ? 1ull << 32 : o == known ? 1 : 0;
            }
        }
        uint64_t total;
        const uint64_t at = before + block_scan(x, sums, total);
        before += total;
        const int eq = static_cast<int>(at & 0xffffffffu);
        if (x >> 32 || (x && eq < left)) {
            const int d = static_cast<int>(at >> 32) + min(eq, left);
            list[d] = p;
            if (kept != nullptr) kept[d] = p;
            if (d != p) atomicMin(&s_first, d);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the list is read by other threads
    __syncthreads();
    const int d0 = min(s_first, a.keep);  // (a cut slot whose last tokens go keeps its places)
    // A page that is written must be this slot's alone, and so must a partly
    // filled last one, which the slot's next tokens are written to.
    for (int j = (d0 >> c.page_shift) + tid; j <= (a.keep - 1) >> c.page_shift; j += kPlan)
        if (c.refs[table[j]] > 1) s_bad = 1;
    __syncthreads();
    if (s_bad != 0) {
        if (kept != nullptr)
            for (int d = tid; d < a.keep; d += kPlan) kept[d] = -1;
        if (tid == 0) {
            k.plan[i] = -1;
            if (a.status != nullptr) a.status[i] = 2;
        }
        return;
    }
    if (tid == 0) {
        k.plan[i] = d0;
        if (a.status != nullptr) a.status[i] = 0;
    }
    for (int e0 = d0; e0 < a.keep; e0 += kPlan) {
        const int d = e0 + tid;
        const float x = d < a.keep ? w[__hip_atomic_load(list + d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)] : 0.f;
        loaded_barrier();
        if (d < a.keep) w[d] = x;
    }
    __syncthreads();
    for (int p = a.keep + tid; p < len; p += kPlan) w[p] = 0.f;
}

// One workgroup per (entry, key head, keys or values): its rows in order, a
// step's reads before its writes.  What a later step reads is behind all that
// an earlier one writes.
__global__ __launch_bounds__(kMove) void cache_evict_move_kernel(EvictK k) {
    const CacheArgs& c = k.c;
    const int i = blockIdx.x, d0 = k.plan[i];
    if (d0 < 0) return;
    const int keep = k.a.keep, kvh = blockIdx.y >> 1, e = c.x == DT::BF16 ? 2 : 4;
    const bool is_k = (blockIdx.y & 1) == 0;
    const int pieces = (is_k ? c.dk : c.dv) * e / 16;
    uint4* pool = static_cast<uint4*>(is_k ? c.k_cache : c.v_cache);
    const int32_t* table = c.table + static_cast<int64_t>(k.a.slot_list[i]) * c.max_pages;
    const int32_t* list = k.list + static_cast<int64_t>(i) * keep;
    const int mask = (1 << c.page_shift) - 1;
    auto row = [&](int p) {
        return (((static_cast<int64_t>(table[p >> c.page_shift]) * c.Hkv + kvh) << c.page_shift) + (p & mask)) * pieces;
    };
    const int64_t all = static_cast<int64_t>(keep - d0) * pieces;
    constexpr int kEach = 4;
    for (int64_t x0 = 0; x0 < all; x0 += kMove * kEach) {
        uint4 r[kEach];
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int64_t at = x0 + x * kMove + threadIdx.x;
            if (at < all) r[x] = pool[row(list[d0 + at / pieces]) + at % pieces];
        }
        loaded_barrier();
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int64_t at = x0 + x * kMove + threadIdx.x;
            if (at < all) pool[row(static_cast<int>(d0 + at / pieces)) + at % pieces] = r[x];
        }
    }
}

// The pages behind are given back, the length is set.
__global__ __launch_bounds__(kMove) void cache_evict_finish_kernel(EvictK k) {
    const CacheArgs& c = k.c;
    const int i = blockIdx.x;
    if (k.plan[i] < 0) return;
    const int slot = k.a.slot_list[i];
    int32_t* table = c.table + static_cast<int64_t>(slot) * c.max_pages;
    for (int j = ((k.a.keep + (1 << c.page_shift) - 1) >> c.page_shift) + threadIdx.x; j < c.max_pages; j += kMove) {
        const int page = table[j];
        if (page == -1) continue;
        table[j] = -1;
        if (names_page(page, c.pages)) atomicSub(c.refs + page, 1);
    }
    if (threadIdx.x == 0) c.lens[slot] = k.a.keep;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t cache_evict_workspace_bytes(int n, int keep) {
    return up256(static_cast<size_t>(n) * keep * 4) + up256(static_cast<size_t>(n) * 4);
}

hipError_t launch_cache_evict(const CacheArgs& c, const EvictArgs& a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    char* ws = static_cast<char*>(a.ws);
    EvictK k{c, a, reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + up256(static_cast<size_t>(a.n) * a.keep * 4))};
    {
        LaunchTimer timer("cache_evict_plan", s);
        cache_evict_plan_kernel<<<dim3(a.n), dim3(kPlan), 0, s>>>(k);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    {
        LaunchTimer timer("cache_evict_move", s);
        cache_evict_move_kernel<<<dim3(a.n, 2 * c.Hkv), dim3(kMove), 0, s>>>(k);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    LaunchTimer timer("cache_evict_finish", s);
    cache_evict_finish_kernel<<<dim3(a.n), dim3(kMove), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace kda
