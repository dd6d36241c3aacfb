// Slots of an attention cache cut down to their heaviest tokens.
//
// The tokens that stay are found by the value of the last one that stays (the
// m-th largest weight, digit by digit over the weights' bits), ties by a count
// in the tokens' order.  They then move to the front in that order: token d
// goes to a place that is not behind its own, so whoever walks them in order
// can move them where they are, as long as a step's reads come before its
// writes.  What a later step reads is behind all that an earlier one writes, so
// that its reads need not wait for those writes.
//
// 64 slots of 500 to 8,000 tokens cut to 2,048 (8 heads of 128, bf16): 204 us, of
// which the plan takes 14 and the rows 182 (0.86 GB, 4.8 TB/s, of the 5.1 that a
// large copy reaches); one of 5,000 cut to 1,024: 28 us, of which the plan takes 12.
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
    int64_t* from;  // [n, keep]: their rows in head 0 of the pools
    int32_t* plan;  // [n][2]: the first token that changes its place (-1: nothing to do), how many there were
    int splits;     // workgroups that share a head's rows, each some of the channels
};

__device__ __forceinline__ bool names_page(int32_t e, int pages) { return e >= 0 && e < pages; }

// A barrier behind loads whose places other threads write after it: every wave
// waits until its own are done.
__device__ __forceinline__ void done_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// A weight as a whole number of the same order: NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (!(w == w)) return 0;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* sums, uint64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t inc = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up(inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        const uint64_t s = sums[w];
        before += w < wave ? s : 0;
        all += s;
    }
    __syncthreads();
    total = all;
    return before + inc - x;
}

// One workgroup per entry: checks it, finds what stays.  The digits (of 11, 11
// and 10 bits: many bins, so that weights of one size do not wait for each other)
// are counted in LDS; no further ones once all of a bin stays.  A slot of up to kStep tokens is read once and its orders
// stay in registers: bound by the length of its chain of barriers.  A longer one
// is read once per digit, the next step's weights in flight: 100,000 tokens in 85
// us, 1.6 us a step and digit.  Weights that are all equal count into one bin of
// each digit: that slot cut to 4,096 tokens 318 us, with others 102.
constexpr int kPer = 8;  // neighbouring tokens of a thread
constexpr int kStep = kPlan * kPer;
constexpr int kDigits = 3, kBins = 2048;
static_assert(kBins == 2 * kPlan, "two bins a thread");

__global__ __launch_bounds__(kPlan) void cache_evict_plan_kernel(EvictK k) {
    __shared__ int hist[kDigits][kBins], stay[kStep];
    __shared__ uint64_t sums[kPlan / 64];
    __shared__ int s_first, s_bad, s_digit, s_left;
    const CacheArgs& c = k.c;
    const EvictArgs& a = k.a;
    const int i = blockIdx.x, tid = threadIdx.x;
    const int slot = a.slot_list[i];
    int32_t* list = k.list + static_cast<int64_t>(i) * a.keep;
    int64_t* rows = k.from + static_cast<int64_t>(i) * a.keep;
    int32_t* kept = a.kept != nullptr ? a.kept + static_cast<int64_t>(i) * a.keep : nullptr;
    const bool real = slot >= 0 && slot < c.slots;
    const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
    const int stored = real ? c.lens[slot] : 0;
    const int len = stored < 0 ? 0 : static_cast<int>(stored > most ? most : stored);
    const int32_t* table = c.table + static_cast<int64_t>(real ? slot : 0) * c.max_pages;
    const float* w = a.weights + ((static_cast<int64_t>(real ? slot : 0) * c.max_pages) << c.page_shift);
    const int mask = (1 << c.page_shift) - 1;

    uint32_t order[kPer];
    float next[kPer];
    const int steps = (len + kStep - 1) / kStep;
    const bool whole = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
    auto fetch = [&](int step) __attribute__((always_inline)) {  // behind the last token 0, which nothing looks at
        const int p = step * kStep + tid * kPer;
        if (whole && p + kPer <= len) {
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e) {
                const float4 v = reinterpret_cast<const float4*>(w + p)[e];
                next[4 * e] = v.x, next[4 * e + 1] = v.y, next[4 * e + 2] = v.z, next[4 * e + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) next[e] = p + e < len ? w[p + e] : 0.f;
        }
    };
    // the orders of a step, the next one's weights on their way (behind the last the first one's again)
    auto take = [&](int step) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) order[e] = order_of(next[e]);
        if (steps > 1) fetch(step + 1 < steps ? step + 1 : 0);
    };
    const bool cut = len > a.keep;
    if (cut) fetch(0);

    // an earlier entry that names the slot has it; every token of a slot that is cut has a page
    if (tid == 0) {
        s_bad = !real;
        s_first = a.keep;
    }
#pragma unroll
    for (int d = 0; d < kDigits; ++d) hist[d][tid] = hist[d][kPlan + tid] = 0;
    __syncthreads();
    for (int j = tid; j < i; j += kPlan)
        if (a.slot_list[j] == slot) s_bad = 1;
    if (cut) {
        for (int j = tid; j < (len + mask) >> c.page_shift; j += kPlan)
            if (!names_page(table[j], c.pages)) s_bad = 1;
    }
    __syncthreads();
    const bool bad = s_bad != 0;
    if (bad || !cut) {
        if (kept != nullptr)
            for (int d = tid; d < a.keep; d += kPlan) kept[d] = !bad && d < len ? d : -1;
        if (tid == 0) {
            k.plan[2 * i] = -1;
            if (a.status != nullptr) a.status[i] = bad ? 2 : 0;
        }
        return;
    }
    // the places between the first and the most recent ones, of which `left` stay
    const int from = a.first, to = len - a.recent;
    const bool some = a.keep > a.first + a.recent;
    int left = a.keep - a.first - a.recent;
    uint32_t known = 0;
    if (some) {
#pragma unroll
        for (int digit = 0; digit < kDigits; ++digit) {
            constexpr int kShift[kDigits] = {21, 10, 0}, kWidth[kDigits] = {11, 11, 10};
            const int shift = kShift[digit], bins = 1 << kWidth[digit];
            for (int step = 0; step < steps; ++step) {
                take(step);
                const int p = step * kStep + tid * kPer;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (p + e >= from && p + e < to && (digit == 0 || order[e] >> (shift + kWidth[digit]) == known >> (shift + kWidth[digit])))
                        atomicAdd(&hist[digit][order[e] >> shift & (bins - 1)], 1);
            }
            __syncthreads();
            // two bins a thread, the largest first
            const int n0 = hist[digit][kBins - 1 - 2 * tid], n1 = hist[digit][kBins - 2 - 2 * tid];
            uint64_t total;
            const int before = static_cast<int>(block_scan(static_cast<uint64_t>(n0 + n1), sums, total));
            if (before < left && left <= before + n0 + n1) {
                const bool second = left > before + n0;
                s_digit = kBins - 1 - 2 * tid - second;
                const int of_it = left - before - (second ? n0 : 0);
                s_left = of_it == (second ? n1 : n0) ? 0 : of_it;  // 0: the whole bin stays
            }
            __syncthreads();
            known |= static_cast<uint32_t>(s_digit) << shift;
            left = s_left;
            if (left == 0) {  // so does all from the bin's first value on, which is above 0: some token goes
                --known;
                break;
            }
        }
    }
    // `left` of those whose order is `known` stay, the first ones, and all above
    // it.  A step's are gathered in LDS and written from there side by side.
    int up_before = 0, eq_before = 0;  // above it or protected, equal to it
    for (int step = 0; step < steps; ++step) {
        take(step);
        const int p0 = step * kStep + tid * kPer;
        uint32_t above = 0, equal = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int p = p0 + e;
            if (p >= len) continue;
            if (p < from || p >= to || (some && order[e] > known)) above |= 1u << e;
            else if (some && order[e] == known) equal |= 1u << e;
        }
        uint64_t total;
        const uint64_t at = block_scan(static_cast<uint64_t>(__popc(above)) << 32 | __popc(equal), sums, total);
        const int base = up_before + min(eq_before, left);
        int up = up_before + static_cast<int>(at >> 32), eq = eq_before + static_cast<int>(at & 0xffffffffu);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const bool is_up = above >> e & 1, is_eq = equal >> e & 1;
            if (is_up || (is_eq && eq < left)) stay[up + min(eq, left) - base] = p0 + e;
            up += is_up;
            eq += is_eq;
        }
        up_before += static_cast<int>(total >> 32);
        eq_before += static_cast<int>(total & 0xffffffffu);
        __syncthreads();
        const int count = up_before + min(eq_before, left) - base;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int x = tid + e * kPlan, d = base + x;
            if (x >= count) break;
            const int p = stay[x];
            list[d] = p;
            rows[d] = ((static_cast<int64_t>(table[p >> c.page_shift]) * c.Hkv) << c.page_shift) + (p & mask);
            if (kept != nullptr) kept[d] = p;
            // tokens before the first one that goes keep their places
            if (p != d && (x == 0 || stay[x - 1] == d - 1)) atomicMin(&s_first, d);
        }
    }
    __syncthreads();  // s_first is whole (the list is for the next launch)
    const int d0 = s_first;
    // A page that is written must be this slot's alone, and so must a partly
    // filled last one, which the slot's next tokens are written to.
    for (int j = (d0 >> c.page_shift) + tid; j <= (a.keep - 1) >> c.page_shift; j += kPlan)
        if (c.refs[table[j]] > 1) s_bad = 1;
    __syncthreads();
    if (s_bad != 0) {
        if (kept != nullptr)
            for (int d = tid; d < a.keep; d += kPlan) kept[d] = -1;
        if (tid == 0) {
            k.plan[2 * i] = -1;
            if (a.status != nullptr) a.status[i] = 2;
        }
        return;
    }
    if (tid == 0) {
        k.plan[2 * i] = d0;
        k.plan[2 * i + 1] = len;
        if (a.status != nullptr) a.status[i] = 0;
    }
}

// One workgroup per (entry, key head, keys or values, part of the channels): its
// rows in order, a step's rows in flight while the one before is written.  One
// workgroup more of an entry moves its weights in the same way, and one gives
// the pages behind back and sets the length (the others read neither those
// entries, nor the counts, nor the length).
constexpr int kRowsEach = 8;  // rows of a thread in a step

__device__ __forceinline__ void move_weights(const EvictK& k, int i, int slot, int d0) {
    const int keep = k.a.keep, len = k.plan[2 * i + 1], tid = threadIdx.x;
    const int32_t* list = k.list + static_cast<int64_t>(i) * keep;
    float* w = k.a.weights + ((static_cast<int64_t>(slot) * k.c.max_pages) << k.c.page_shift);
    constexpr int kEach = 8, kStep = kMove * kEach;
    struct Step {
        float x[kEach];
    };
    auto load = [&](Step& s, int d) __attribute__((always_inline)) {
        int at[kEach];
#pragma unroll
        for (int n = 0; n < kEach; ++n) at[n] = list[min(d + n * kMove + tid, keep - 1)];
#pragma unroll
        for (int n = 0; n < kEach; ++n) s.x[n] = w[at[n]];
    };
    auto store = [&](Step& s, int d) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < kEach; ++n) asm volatile("" : "+v"(s.x[n]));
        lds_barrier();
#pragma unroll
        for (int n = 0; n < kEach; ++n)
            if (d + n * kMove + tid < keep) w[d + n * kMove + tid] = s.x[n];
    };
    Step a, b;
    load(a, d0);
    for (int d = d0; d < keep; d += 2 * kStep) {
        load(b, d + kStep);
        store(a, d);
        if (d + kStep >= keep) break;
        load(a, d + 2 * kStep);
        store(b, d + kStep);
    }
    done_barrier();  // the last loads
    for (int p = keep + tid; p < len; p += kMove) w[p] = 0.f;
}

__global__ __launch_bounds__(kMove) void cache_evict_move_kernel(EvictK k) {
    const CacheArgs& c = k.c;
    const int i = blockIdx.x, d0 = k.plan[2 * i], keep = k.a.keep;
    if (d0 < 0) return;
    const int slot = k.a.slot_list[i];
    int32_t* table = c.table + static_cast<int64_t>(slot) * c.max_pages;
    if (blockIdx.y == gridDim.y - 1) {
        for (int j = ((keep + (1 << c.page_shift) - 1) >> c.page_shift) + threadIdx.x; j < c.max_pages; j += kMove) {
            const int page = table[j];
            if (page == -1) continue;
            table[j] = -1;
            if (names_page(page, c.pages)) atomicSub(c.refs + page, 1);
        }
        if (threadIdx.x == 0) c.lens[slot] = keep;
        return;
    }
    if (blockIdx.y == gridDim.y - 2) return move_weights(k, i, slot, d0);
    const int share = blockIdx.y % k.splits, unit = blockIdx.y / k.splits;
    const int kvh = unit >> 1, e = c.x == DT::BF16 ? 2 : 4;
    const int pieces = ((unit & 1) == 0 ? c.dk : c.dv) * e / 16;
    const int mine = pieces / k.splits, at_once = kMove / mine;  // pieces of a row, rows of a step of one each
    const int row = threadIdx.x / mine;
    const bool on = row < at_once;
    uint4* pool = static_cast<uint4*>((unit & 1) == 0 ? c.k_cache : c.v_cache) + share * mine + threadIdx.x % mine;
    const int64_t* from = k.from + static_cast<int64_t>(i) * keep;
    const int64_t head = static_cast<int64_t>(kvh) << c.page_shift;
    const int mask = (1 << c.page_shift) - 1, step = at_once * kRowsEach;
    struct Step {
        uint4 r[kRowsEach];
        int page[kRowsEach];  // that they go to
    };
    auto load = [&](Step& x, int d) __attribute__((always_inline)) {
        int64_t at[kRowsEach];
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) {
            const int to = min(d + n * at_once + row, keep - 1);
            at[n] = from[to];
            x.page[n] = table[to >> c.page_shift];
        }
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) x.r[n] = pool[(at[n] + head) * pieces];
    };
    // The rows of a step have arrived in every wave before any of its places is written.
    auto store = [&](Step& x, int d) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) asm volatile("" : "+v"(x.r[n].x), "+v"(x.r[n].y), "+v"(x.r[n].z), "+v"(x.r[n].w));
        lds_barrier();
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) {
            const int to = d + n * at_once + row;
            if (on && to < keep) pool[(((static_cast<int64_t>(x.page[n]) * c.Hkv) << c.page_shift) + head + (to & mask)) * pieces] = x.r[n];
        }
    };
    Step a, b;
    load(a, d0);
    for (int d = d0; d < keep; d += 2 * step) {
        load(b, d + step);
        store(a, d);
        if (d + step >= keep) break;
        load(a, d + 2 * step);
        store(b, d + step);
    }
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t cache_evict_workspace_bytes(int n, int keep) {
    const size_t all = static_cast<size_t>(n) * keep;
    return up256(all * 4) + up256(all * 8) + up256(static_cast<size_t>(n) * 8);
}

hipError_t launch_cache_evict(const CacheArgs& c, const EvictArgs& a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    const size_t all = static_cast<size_t>(a.n) * a.keep;
    char* ws = static_cast<char*>(a.ws);
    EvictK k{c, a, nullptr, nullptr, nullptr, 1};
    k.list = reinterpret_cast<int32_t*>(ws);
    ws += up256(all * 4);
    k.from = reinterpret_cast<int64_t*>(ws);
    ws += up256(all * 8);
    k.plan = reinterpret_cast<int32_t*>(ws);
    {
        LaunchTimer timer("cache_evict_plan", s);
        cache_evict_plan_kernel<<<dim3(a.n), dim3(kPlan), 0, s>>>(k);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // few workgroups: each takes fewer channels of more rows, 64 bytes of a row at least
    const int row = (c.dk < c.dv ? c.dk : c.dv) * (c.x == DT::BF16 ? 2 : 4);
    while (k.splits < 4 && static_cast<int64_t>(a.n) * 2 * c.Hkv * k.splits < 512 && row / (2 * k.splits) >= 64) k.splits *= 2;
    LaunchTimer timer("cache_evict_move", s);
    cache_evict_move_kernel<<<dim3(a.n, 2 * c.Hkv * k.splits + 2), dim3(kMove), 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace kda
