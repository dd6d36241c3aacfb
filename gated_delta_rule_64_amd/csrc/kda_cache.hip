// The pages of an attention cache: rows written into them, sequences forked
// over them, pages freed, given out, moved together and copied.
//
// A page is free when refs[page], the number of table entries that name it,
// is not positive.  There is no list of free pages: whoever needs some takes
// the lowest-numbered ones, found by a scan over refs, so that the result
// does not depend on the order in which workgroups run, and freeing is one
// atomic subtraction per entry, in any order.
//
// What bounds them: the copies memory, the planning workgroups the length of
// their chains of dependent loads and scans.  Measured with pages of 8 heads of
// 128 in bf16; the sizes stand at each kernel.
#include "kda_common.h"
#include "kda_internal.h"
#include "kda_profile.h"

namespace kda {
namespace {

constexpr int kPlan = 1024;  // threads of the planning workgroup
constexpr int kCopy = 256;   // threads of a copying workgroup

__device__ __forceinline__ bool names_page(int32_t e, int pages) { return e >= 0 && e < pages; }

__device__ __forceinline__ int load_fresh(const int32_t* p) {  // past the vector L1
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_fresh(int32_t* p, int32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A barrier of the planning workgroup behind stores that its other threads
// read: every wave waits until the L2 has its stores, where load_fresh finds
// them.  (A device-wide fence would write the L2 back as well, for other dies
// that do not read here: kda_cache_reserve's kernel for 256 slots 17 us, so 8.)
__device__ __forceinline__ void stored_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// Exclusive scan of one value per thread of the planning workgroup; `total`
// gets the sum.  sums: kPlan / 64 words of LDS.  All threads call it.
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

// Counts of kEach neighbouring pages per thread and step.  The first step's
// can be put in flight long before they are looked at, and are kept: a pool of
// up to 8,192 pages is read once.
constexpr int kEach = 8;
struct PageCounts {
    int r[kEach];
    __device__ __forceinline__ void load(const int32_t* refs, int pages, int p0) {
        const int first = p0 + static_cast<int>(threadIdx.x) * kEach;
        if (first + kEach <= pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
            const int4 a = reinterpret_cast<const int4*>(refs + first)[0], b = reinterpret_cast<const int4*>(refs + first)[1];
            r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
            r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) r[i] = first + i < pages ? refs[first + i] : 1;
        }
    }
};

// The lowest `want` free pages in order, list[0 .. want); returns how many
// there are (at most want).  counts: the first step's.  All threads of the
// planning workgroup call it.
__device__ __forceinline__ int lowest_free(const int32_t* refs, int pages, PageCounts counts, int want, int32_t* list, int* sums) {
    int found = 0;
    for (int p0 = 0; p0 < pages && found < want; p0 += kPlan * kEach) {
        if (p0 > 0) counts.load(refs, pages, p0);
        const int first = p0 + static_cast<int>(threadIdx.x) * kEach;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) mine += counts.r[i] <= 0;
        int total;
        int at = found + block_scan(mine, sums, total);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (counts.r[i] <= 0) {
                if (at < want) store_fresh(list + at, first + i);
                ++at;
            }
        found += total;
    }
    stored_barrier();
    return min(found, want);
}

// Of the good entries of a call that name the same slot, the first keeps it.
// The claims stand in LDS where the cache has few slots, else in the
// workspace, a word per slot.
constexpr int kLdsSlots = 8192;
struct Claims {
    int* lds;
    int32_t* memory;
    bool in_lds;
    __device__ __forceinline__ void clear(int slots, const int32_t* slot_of, int n) const {
        if (in_lds) {
            for (int s = threadIdx.x; s < slots; s += kPlan) lds[s] = INT32_MAX;
        } else {
            for (int i = threadIdx.x; i < n; i += kPlan)
                if (slot_of[i] >= 0 && slot_of[i] < slots) store_fresh(memory + slot_of[i], INT32_MAX);
        }
        stored_barrier();
    }
    __device__ __forceinline__ void claim(int slot, int i) const {
        if (in_lds) atomicMin(lds + slot, i);
        else atomicMin(memory + slot, i);
    }
    __device__ __forceinline__ void settle() const {
        stored_barrier();
    }
    __device__ __forceinline__ int owner(int slot) const { return in_lds ? lds[slot] : load_fresh(memory + slot); }
};

// ------------------------------------------------------------------- append

struct AppendK {
    CacheArgs c;
    int64_t tokens, src_rows;
    int N;
    const int32_t *cu, *rows, *slot_indices;
    const void *k_new, *v_new;
};

// Eight tokens find their rows, then the workgroup copies them in pieces of 16
// bytes, a token's heads side by side.  33,256 prompt tokens, 273 MB moved: 50 us (5.4
// TB/s); four pieces in flight per thread were slower (62 to 69 us a call).
constexpr int kAppendTokens = 8;  // tokens of a workgroup

__global__ __launch_bounds__(kCopy) void cache_append_kernel(AppendK a) {
    __shared__ int64_t s_src[kAppendTokens], s_dst[kAppendTokens];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kAppendTokens;
    const CacheArgs& c = a.c;
    if (threadIdx.x < kAppendTokens) {
        const int64_t t = t0 + threadIdx.x;
        int64_t src = -1, dst = -1;
        if (t < a.tokens) {
            int n = 0;
            int64_t first = 0, end = a.tokens;
            if (a.cu != nullptr) {
                n = find_seq(a.cu, a.N, t);
                first = a.cu[n];
                end = a.cu[n + 1];
            }
            if (t >= first && t < end) {
                const int slot = a.slot_indices != nullptr ? a.slot_indices[n] : n;
                src = a.rows != nullptr ? a.rows[t] : t;
                if (slot >= 0 && slot < c.slots && src >= 0 && src < a.src_rows) {
                    const int64_t pos = static_cast<int64_t>(max(c.lens[slot], 0)) + (t - first);
                    const int64_t col = pos >> c.page_shift;
                    if (col < c.max_pages) {
                        const int page = c.table[static_cast<int64_t>(slot) * c.max_pages + col];
                        if (names_page(page, c.pages))
                            dst = ((static_cast<int64_t>(page) * c.Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
                    }
                }
            }
        }
        s_src[threadIdx.x] = src;
        s_dst[threadIdx.x] = dst;  // row of head 0; head h is h << page_shift rows on
    }
    __syncthreads();
    const int e = c.x == DT::BF16 ? 2 : 4;
    const int k_pieces = c.dk * e / 16, v_pieces = c.dv * e / 16, head = k_pieces + v_pieces;
    const int per_token = c.Hkv * head;
    const uint4* kn = static_cast<const uint4*>(a.k_new);
    const uint4* vn = static_cast<const uint4*>(a.v_new);
    uint4* kc = static_cast<uint4*>(c.k_cache);
    uint4* vc = static_cast<uint4*>(c.v_cache);
    for (int i = threadIdx.x; i < kAppendTokens * per_token; i += kCopy) {
        const int t = i / per_token, p = i - t * per_token;
        const int64_t dst = s_dst[t], src = s_src[t];
        if (dst < 0) continue;
        const int k_all = c.Hkv * k_pieces;
        if (p < k_all) {
            const int h = p / k_pieces, x = p - h * k_pieces;
            kc[(dst + (static_cast<int64_t>(h) << c.page_shift)) * k_pieces + x] = kn[src * k_all + p];
        } else {
            const int y = p - k_all, h = y / v_pieces, x = y - h * v_pieces;
            vc[(dst + (static_cast<int64_t>(h) << c.page_shift)) * v_pieces + x] = vn[src * (c.Hkv * v_pieces) + y];
        }
    }
}

// --------------------------------------------------------------------- free

// A thread per table entry: 256 slots in 3 us, a launch's latency.
__global__ __launch_bounds__(kCopy) void cache_free_kernel(CacheArgs c, const int32_t* slot_list) {
    const int slot = slot_list[blockIdx.x];
    if (slot < 0 || slot >= c.slots) return;
    int32_t* row = c.table + static_cast<int64_t>(slot) * c.max_pages;
    const int col = blockIdx.y * kCopy + threadIdx.x;
    // the exchange gives an entry to one workgroup only, also where a slot is
    // named twice
    if (col < c.max_pages) {
        const int page = atomicExch(row + col, -1);
        if (names_page(page, c.pages)) atomicSub(c.refs + page, 1);
    }
    if (col == 0) c.lens[slot] = 0;
}

// --------------------------------------------------------------------- fork

struct ForkK {
    CacheArgs c;
    int n;
    const int32_t *src, *dst;
    int32_t* status;
    int32_t* claim;  // [slots]
    int32_t* list;   // [n] free pages
    int32_t* plan;   // [n][2]: source length (-1: refused), the new last page (-1: none needed)
};

// One workgroup: every entry is checked, the destinations claimed, then one scan
// over refs finds the pages.  256 forks: 8 us.
__global__ __launch_bounds__(kPlan) void cache_fork_plan_kernel(ForkK a) {
    __shared__ int sums[kPlan / 64];
    __shared__ int claims[kLdsSlots];
    const CacheArgs& c = a.c;
    const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
    const int mask = (1 << c.page_shift) - 1;
    PageCounts counts;
    counts.load(c.refs, c.pages, 0);
    const Claims slots{claims, a.claim, c.slots <= kLdsSlots};
    slots.clear(c.slots, a.dst, a.n);
    // what an entry is, kept in the plan by the thread that reads it again:
    // the source's length (-1: refused), whether its last page is to be copied
    for (int i = threadIdx.x; i < a.n; i += kPlan) {
        const int s = a.src[i], d = a.dst[i];
        int len = -1, need = 0;
        if (s >= 0 && s < c.slots && d >= 0 && d < c.slots && s != d) {
            const int dst_len = c.lens[d], dst_first = c.table[static_cast<int64_t>(d) * c.max_pages];
            const int64_t n = c.lens[s];
            if (dst_len == 0 && !names_page(dst_first, c.pages)) {  // the destination is empty
                len = static_cast<int>(n < 0 ? 0 : n > most ? most : n);
                if ((len & mask) != 0)
                    need = names_page(c.table[static_cast<int64_t>(s) * c.max_pages + (len >> c.page_shift)], c.pages);
                slots.claim(d, i);
            }
        }
        a.plan[2 * i] = len;
        a.plan[2 * i + 1] = need;
    }
    slots.settle();
    int want = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        int total, need = 0;
        if (i < a.n) {
            need = a.plan[2 * i + 1];
            if (a.plan[2 * i] >= 0 && slots.owner(a.dst[i]) != i) {
                a.plan[2 * i] = -1;
                a.plan[2 * i + 1] = need = 0;
            }
        }
        block_scan<int>(need, sums, total);
        want += total;
    }
    const int have = lowest_free(c.refs, c.pages, counts, want, a.list, sums);
    int before = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        const int len = i < a.n ? a.plan[2 * i] : -1, need = i < a.n ? a.plan[2 * i + 1] : 0;
        int total;
        const int at = before + block_scan<int>(need, sums, total);
        before += total;
        if (i < a.n) {
            int status = len >= 0 ? 0 : 2, page = -1;
            if (need) {
                if (at < have) {
                    page = load_fresh(a.list + at);
                    c.refs[page] = 1;
                } else {
                    status = 1;
                    a.plan[2 * i] = -1;
                }
            }
            a.plan[2 * i + 1] = page;
            if (a.status != nullptr) a.status[i] = status;
        }
    }
}

// Workgroup (i, 0) writes entry i's table row, (i, 1 + y) copies its share of
// the rows of the last page: 256 forks, 58 MB moved, in 14.5 us (4.0 TB/s).
__global__ __launch_bounds__(kCopy) void cache_fork_apply_kernel(ForkK a) {
    const CacheArgs& c = a.c;
    const int i = blockIdx.x;
    const int len = a.plan[2 * i], page = a.plan[2 * i + 1];
    if (len < 0) return;
    const int full = len >> c.page_shift, part = len & ((1 << c.page_shift) - 1);
    const int32_t* from = c.table + static_cast<int64_t>(a.src[i]) * c.max_pages;
    if (blockIdx.y == 0) {
        int32_t* to = c.table + static_cast<int64_t>(a.dst[i]) * c.max_pages;
        for (int j = threadIdx.x; j < full; j += kCopy) {
            const int p = from[j];
            to[j] = p;
            if (names_page(p, c.pages)) atomicAdd(c.refs + p, 1);
        }
        if (threadIdx.x == 0) {
            if (part > 0) to[full] = page;
            c.lens[a.dst[i]] = len;
        }
        return;
    }
    if (page < 0) return;
    const int e = c.x == DT::BF16 ? 2 : 4;
    const int64_t old = from[full];
    const int k_pieces = c.dk * e / 16, v_pieces = c.dv * e / 16;
    // a head's rows of a page are contiguous: part * k_pieces, then part * v_pieces
    const int per_head = part * (k_pieces + v_pieces), step = (gridDim.y - 1) * kCopy;
    uint4* kc = static_cast<uint4*>(c.k_cache);
    uint4* vc = static_cast<uint4*>(c.v_cache);
    for (int64_t w = static_cast<int64_t>(blockIdx.y - 1) * kCopy + threadIdx.x; w < static_cast<int64_t>(c.Hkv) * per_head; w += step) {
        const int h = static_cast<int>(w / per_head), x = static_cast<int>(w - static_cast<int64_t>(h) * per_head);
        const int64_t r0 = (old * c.Hkv + h) << c.page_shift, r1 = (static_cast<int64_t>(page) * c.Hkv + h) << c.page_shift;
        if (x < part * k_pieces) kc[r1 * k_pieces + x] = kc[r0 * k_pieces + x];
        else vc[r1 * v_pieces + x - part * k_pieces] = vc[r0 * v_pieces + x - part * k_pieces];
    }
}

// ------------------------------------------------------------------ reserve

struct ReserveK {
    CacheArgs c;
    int n;
    const int32_t *slot_list, *new_lens;
    int32_t* status;
    int32_t* claim;  // [slots]
    int32_t* counts; // [n] pages wanted, then the first one's place in `list`
    int32_t* list;   // [pages]
};

// One workgroup.  Every entry's columns that lack a page are counted, a scan
// gives every entry its place, and the lowest free pages go out in that order.
// An entry of few columns (a decode step's) is one thread's, so that the
// entries' dependent loads overlap (256 entries with a wave each: 49 us where threads took 20); one
// of many columns (a prompt's) a wave's.
constexpr int kFewColumns = 16;

__global__ __launch_bounds__(kPlan) void cache_reserve_kernel(ReserveK a) {
    __shared__ int sums[kPlan / 64];
    __shared__ int64_t sums64[kPlan / 64];  // the counts of a bad call may add up to more than 2^31
    __shared__ int claims[kLdsSlots];
    __shared__ int many;  // whether any entry has many columns
    if (threadIdx.x == 0) many = 0;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mask = (1 << c.page_shift) - 1;
    PageCounts pages;
    pages.load(c.refs, c.pages, 0);
    const Claims slots{claims, a.claim, c.slots <= kLdsSlots};
    slots.clear(c.slots, a.slot_list, a.n);
    struct Entry {
        int slot, first, end;  // the columns [first, end) are looked at; slot -1: refused
    };
    auto entry = [&](int i) {
        Entry e;
        e.slot = a.slot_list[i];
        const int64_t n = (static_cast<int64_t>(max(a.new_lens[i], 0)) + mask) >> c.page_shift;
        if (e.slot < 0 || e.slot >= c.slots || n > c.max_pages) return Entry{-1, 0, 0};
        e.end = static_cast<int>(n);
        // (only the columns behind the length: a missing page in front of it had
        // tokens, and a new page's stale contents would be attended as them)
        e.first = min(static_cast<int>((static_cast<int64_t>(max(c.lens[e.slot], 0)) + mask) >> c.page_shift), e.end);
        return e;
    };
    // a thread's first entry stays in its registers
    const Entry mine = static_cast<int>(threadIdx.x) < a.n ? entry(threadIdx.x) : Entry{-1, 0, 0};
    auto my_entry = [&](int i) { return i < kPlan ? mine : entry(i); };  // of a loop from threadIdx.x on
    for (int i = threadIdx.x; i < a.n; i += kPlan) {
        const Entry e = my_entry(i);
        if (e.slot >= 0) slots.claim(e.slot, i);
    }
    slots.settle();
    auto owned = [&](int i, const Entry& e) { return e.slot >= 0 && slots.owner(e.slot) == i; };
    for (int i = threadIdx.x; i < a.n; i += kPlan) {
        const Entry e = my_entry(i);
        int count = -1;
        if (owned(i, e)) {
            count = 0;
            if (e.end - e.first <= kFewColumns) {
                const int32_t* row = c.table + static_cast<int64_t>(e.slot) * c.max_pages;
                for (int j = e.first; j < e.end; ++j) count += !names_page(row[j], c.pages);
            } else {
                many = 1;
            }
        }
        store_fresh(a.counts + i, count);
    }
    stored_barrier();
    for (int i = wave; many != 0 && i < a.n; i += kPlan / 64) {
        const Entry e = entry(i);
        if (e.end - e.first <= kFewColumns || !owned(i, e)) continue;
        const int32_t* row = c.table + static_cast<int64_t>(e.slot) * c.max_pages;
        int count = 0;
        for (int j0 = e.first; j0 < e.end; j0 += 64) {
            const int j = j0 + lane;
            count += __popcll(__ballot(j < e.end && !names_page(row[j < e.end ? j : 0], c.pages)));
        }
        if (lane == 0) store_fresh(a.counts + i, count);
    }
    stored_barrier();
    int64_t want = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        int64_t total;
        block_scan<int64_t>(i < a.n ? max(load_fresh(a.counts + i), 0) : 0, sums64, total);
        want += total;
    }
    const int have = lowest_free(c.refs, c.pages, pages, static_cast<int>(min(want, static_cast<int64_t>(c.pages))), a.list, sums);
    int64_t before = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        const int count = i < a.n ? load_fresh(a.counts + i) : 0;
        int64_t total;
        const int64_t at = before + block_scan<int64_t>(max(count, 0), sums64, total);
        before += total;
        if (i < a.n) {
            const bool fits = count == 0 || (count > 0 && at + count <= have);
            if (a.status != nullptr) a.status[i] = count < 0 ? 2 : fits ? 0 : 1;
            int place = count > 0 && fits ? static_cast<int>(at) : -1;
            if (place >= 0) {
                const Entry e = my_entry(i);
                if (e.end - e.first <= kFewColumns) {
                    int32_t* row = c.table + static_cast<int64_t>(e.slot) * c.max_pages;
                    for (int j = e.first; j < e.end; ++j)
                        if (!names_page(row[j], c.pages)) {
                            const int page = load_fresh(a.list + place++);
                            row[j] = page;
                            c.refs[page] = 1;
                        }
                    place = -1;
                }
            }
            store_fresh(a.counts + i, place);
        }
    }
    if (many == 0) return;
    stored_barrier();
    for (int i = wave; i < a.n; i += kPlan / 64) {
        int at = load_fresh(a.counts + i);
        if (at < 0) continue;
        const Entry e = entry(i);
        int32_t* row = c.table + static_cast<int64_t>(e.slot) * c.max_pages;
        for (int j0 = e.first; j0 < e.end; j0 += 64) {
            const int j = j0 + lane;
            const bool lacks = j < e.end && !names_page(row[j < e.end ? j : 0], c.pages);
            const unsigned long long all = __ballot(lacks);
            if (lacks) {
                const int page = load_fresh(a.list + at + __popcll(all & ((1ull << lane) - 1)));
                row[j] = page;
                c.refs[page] = 1;
            }
            at += __popcll(all);
        }
    }
}

// ------------------------------------------------------------------ compact

struct CompactK {
    CacheArgs c;
    int32_t* live;    // [1]
    int32_t* moves;   // [1] pages to move
    int32_t* to;      // [pages] where a page goes
    int32_t *from_list, *to_list;  // [pages]
};

// One workgroup, two scans over refs.  8,192 pages: 12 us.
__global__ __launch_bounds__(kPlan) void cache_compact_plan_kernel(CompactK a) {
    __shared__ int sums[kPlan / 64];
    __shared__ int64_t sums64[kPlan / 64];
    const CacheArgs& c = a.c;
    PageCounts counts;
    int live = 0;
    for (int p0 = 0; p0 < c.pages; p0 += kPlan * kEach) {
        counts.load(c.refs, c.pages, p0);
        const int first = p0 + static_cast<int>(threadIdx.x) * kEach;
        int mine = 0, total;
#pragma unroll
        for (int i = 0; i < kEach; ++i) mine += first + i < c.pages && counts.r[i] > 0;
        block_scan(mine, sums, total);
        live += total;
    }
    // the k-th free page below `live` takes the k-th page in use behind it
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < c.pages; p0 += kPlan * kEach) {
        if (c.pages > kPlan * kEach) counts.load(c.refs, c.pages, p0);  // else they are still there
        const int first = p0 + static_cast<int>(threadIdx.x) * kEach;
        bool hole[kEach], mover[kEach];
        int64_t both = 0, all;  // holes in the low word, movers in the high one
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = first + i;
            const bool used = p < c.pages && counts.r[i] > 0;
            hole[i] = p < live && !used;
            mover[i] = p >= live && used;
            both += static_cast<int64_t>(hole[i]) + (static_cast<int64_t>(mover[i]) << 32);
        }
        const int64_t at = block_scan(both, sums64, all);
        int ah = holes + static_cast<int>(at), am = movers + static_cast<int>(at >> 32);
        holes += static_cast<int>(all);
        movers += static_cast<int>(all >> 32);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (first + i < c.pages) store_fresh(a.to + first + i, first + i);
            if (hole[i]) store_fresh(a.to_list + ah++, first + i);
            if (mover[i]) store_fresh(a.from_list + am++, first + i);
        }
    }
    stored_barrier();
    for (int k = threadIdx.x; k < movers; k += kPlan) {
        const int s = load_fresh(a.from_list + k), d = load_fresh(a.to_list + k);
        store_fresh(a.to + s, d);
        c.refs[d] = c.refs[s];
        c.refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        *a.live = live;
        *a.moves = movers;
    }
}

// One 16-byte piece per thread and step, four in flight.
__device__ __forceinline__ void copy_pieces(const uint4* src, uint4* dst, int64_t n) {
    constexpr int kFlight = 4;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += kCopy * kFlight) {
        uint4 r[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (i0 + i * kCopy < n) r[i] = src[i0 + i * kCopy];
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (i0 + i * kCopy < n) dst[i0 + i * kCopy] = r[i];
    }
}

constexpr int64_t kSegment = 1024;  // 16-byte pieces that a workgroup copies at a time

// The first table_blocks workgroups rewrite the table, the others move pages, a
// segment of 16 KiB at a time so that few pages still fill the chip: 969 MB in
// 175 to 203 us (4.8 to 5.5 TB/s; a large copy measured 5.1).
__global__ __launch_bounds__(kCopy) void cache_compact_move_kernel(CompactK a, int table_blocks) {
    const CacheArgs& c = a.c;
    if (static_cast<int>(blockIdx.x) < table_blocks) {
        const int64_t entries = static_cast<int64_t>(c.slots) * c.max_pages;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopy + threadIdx.x; i < entries; i += static_cast<int64_t>(table_blocks) * kCopy) {
            const int p = c.table[i];
            if (names_page(p, c.pages)) c.table[i] = a.to[p];
        }
        return;
    }
    const int e = c.x == DT::BF16 ? 2 : 4;
    const int64_t kp = (static_cast<int64_t>(c.Hkv) << c.page_shift) * (c.dk * e / 16);
    const int64_t vp = (static_cast<int64_t>(c.Hkv) << c.page_shift) * (c.dv * e / 16);
    const int64_t ks = (kp + kSegment - 1) / kSegment, vs = (vp + kSegment - 1) / kSegment;
    const int64_t work = static_cast<int64_t>(*a.moves) * (ks + vs);
    for (int64_t w = blockIdx.x - table_blocks; w < work; w += gridDim.x - table_blocks) {
        const int64_t k = w / (ks + vs);
        int64_t x = w - k * (ks + vs);
        const bool is_k = x < ks;
        const int64_t size = is_k ? kp : vp;
        if (!is_k) x -= ks;
        uint4* pool = static_cast<uint4*>(is_k ? c.k_cache : c.v_cache);
        const int64_t at = x * kSegment;
        copy_pieces(pool + a.from_list[k] * size + at, pool + a.to_list[k] * size + at, min(kSegment, size - at));
    }
}

// --------------------------------------------------------------------- copy

// Segments of rows in turn: 256 KDA states of 2 MB, 1.07 GB moved, in 217 us (5.0
// TB/s), 2,000 pages of 128 KB in 116 us (4.5).
__global__ __launch_bounds__(kCopy) void cache_copy_kernel(uint4* pool, int64_t row_pieces, int rows, const int32_t* src, const int32_t* dst,
                                                           int n) {
    const int64_t segments = (row_pieces + kSegment - 1) / kSegment;
    for (int64_t w = blockIdx.x; w < segments * n; w += gridDim.x) {
        const int64_t i = w / segments, at = (w - i * segments) * kSegment;
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= rows || d < 0 || d >= rows || s == d) continue;
        copy_pieces(pool + s * row_pieces + at, pool + d * row_pieces + at, min(kSegment, row_pieces - at));
    }
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kMoveBlocks = 2048;

}  // namespace

hipError_t launch_cache_append(const CacheArgs& c, int64_t tokens, int N, const int32_t* cu, int64_t src_rows, const int32_t* rows,
                               const void* k_new, const void* v_new, const int32_t* slot_indices, hipStream_t s) {
    if (tokens == 0) return hipSuccess;
    const AppendK a{c, tokens, src_rows, N, cu, rows, slot_indices, k_new, v_new};
    LaunchTimer timer("cache_append", s);
    cache_append_kernel<<<dim3(static_cast<unsigned>((tokens + kAppendTokens - 1) / kAppendTokens)), dim3(kCopy), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_free(const CacheArgs& c, int n, const int32_t* slot_list, hipStream_t s) {
    if (n == 0) return hipSuccess;
    LaunchTimer timer("cache_free", s);
    cache_free_kernel<<<dim3(n, (c.max_pages + kCopy - 1) / kCopy), dim3(kCopy), 0, s>>>(c, slot_list);
    return hipGetLastError();
}

size_t cache_workspace_bytes(int pages, int slots, int n) {
    const size_t fork = up256(static_cast<size_t>(slots) * 4) + up256(static_cast<size_t>(n) * 4) + up256(static_cast<size_t>(n) * 8);
    const size_t reserve = up256(static_cast<size_t>(slots) * 4) + up256(static_cast<size_t>(n) * 4) + up256(static_cast<size_t>(pages) * 4);
    const size_t compact = 256 + 3 * up256(static_cast<size_t>(pages) * 4);
    const size_t a = fork > reserve ? fork : reserve;
    return a > compact ? a : compact;
}

hipError_t launch_cache_fork(const CacheArgs& c, int n, const int32_t* src, const int32_t* dst, int32_t* status, void* ws, hipStream_t s) {
    if (n == 0) return hipSuccess;
    char* w = static_cast<char*>(ws);
    ForkK a{c, n, src, dst, status, nullptr, nullptr, nullptr};
    a.claim = reinterpret_cast<int32_t*>(w);
    w += up256(static_cast<size_t>(c.slots) * 4);
    a.list = reinterpret_cast<int32_t*>(w);
    w += up256(static_cast<size_t>(n) * 4);
    a.plan = reinterpret_cast<int32_t*>(w);
    {
        LaunchTimer timer("cache_fork_plan", s);
        cache_fork_plan_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t page_bytes = (static_cast<int64_t>(c.Hkv) << c.page_shift) * (c.dk + c.dv) * (c.x == DT::BF16 ? 2 : 4);
    int64_t shares = page_bytes / (16 * kCopy * 8);  // eight pieces a thread of a full page
    shares = shares < 1 ? 1 : shares > 64 ? 64 : shares;
    LaunchTimer timer("cache_fork_apply", s);
    cache_fork_apply_kernel<<<dim3(n, static_cast<unsigned>(1 + shares)), dim3(kCopy), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_reserve(const CacheArgs& c, int n, const int32_t* slot_list, const int32_t* new_lens, int32_t* status, void* ws,
                                hipStream_t s) {
    if (n == 0) return hipSuccess;
    char* w = static_cast<char*>(ws);
    ReserveK a{c, n, slot_list, new_lens, status, nullptr, nullptr, nullptr};
    a.claim = reinterpret_cast<int32_t*>(w);
    w += up256(static_cast<size_t>(c.slots) * 4);
    a.counts = reinterpret_cast<int32_t*>(w);
    w += up256(static_cast<size_t>(n) * 4);
    a.list = reinterpret_cast<int32_t*>(w);
    LaunchTimer timer("cache_reserve", s);
    cache_reserve_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const CacheArgs& c, int32_t* live, void* ws, hipStream_t s) {
    char* w = static_cast<char*>(ws);
    CompactK a{c, live, nullptr, nullptr, nullptr, nullptr};
    a.moves = reinterpret_cast<int32_t*>(w);
    w += 256;
    const size_t list = up256(static_cast<size_t>(c.pages) * 4);
    a.to = reinterpret_cast<int32_t*>(w);
    a.from_list = reinterpret_cast<int32_t*>(w + list);
    a.to_list = reinterpret_cast<int32_t*>(w + 2 * list);
    {
        LaunchTimer timer("cache_compact_plan", s);
        cache_compact_plan_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t entries = static_cast<int64_t>(c.slots) * c.max_pages;
    const int64_t want = (entries + 4 * kCopy - 1) / (4 * kCopy);
    const int table_blocks = static_cast<int>(want < 1 ? 1 : want > 256 ? 256 : want);
    LaunchTimer timer("cache_compact_move", s);
    cache_compact_move_kernel<<<dim3(table_blocks + kMoveBlocks), dim3(kCopy), 0, s>>>(a, table_blocks);
    return hipGetLastError();
}

hipError_t launch_cache_copy(void* pool, int64_t row_bytes, int rows, const int32_t* src, const int32_t* dst, int n, hipStream_t s) {
    if (n == 0 || row_bytes == 0) return hipSuccess;
    const int64_t pieces = row_bytes / 16, work = (pieces + kSegment - 1) / kSegment * n;
    LaunchTimer timer("cache_copy", s);
    cache_copy_kernel<<<dim3(static_cast<unsigned>(work < 4096 ? work : 4096)), dim3(kCopy), 0, s>>>(static_cast<uint4*>(pool), pieces, rows,
                                                                                                 src, dst, n);
    return hipGetLastError();
}

}  // namespace kda
