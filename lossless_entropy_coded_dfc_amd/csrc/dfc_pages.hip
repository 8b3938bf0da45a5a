// dfc_pages.hip - pages of the cache given back, shared, moved and copied.
//
// shared[p] is the number of requests that hold page p beyond the first.
//
// dfc_paged_release.  A request gives up entries of its row; every one takes a
// holder off its page, and a page whose count passes below zero is free.  The
// counts are atomic sums, so which pages are free does not depend on any
// order; they go to the ring in ascending order of their numbers, so their
// places do not either.
//
// dfc_paged_fork.  Full pages of the parent's first tokens gain a holder, the
// one that the tokens fill in part gets a new page off the ring: the i-th such
// copy of the call takes the i-th free page.
//
// dfc_paged_compact.  With the held and the free pages in ascending order
// a_0 < a_1 < ..., U of them held, page a_i stays if i < U and is held, is a
// place to move to if i < U and is free, and is on the ring afterwards if
// i >= U: all of it prefix sums of two flags over the pages.
//
// Bounds (one MI355X).  Tables, counts and rings are a few bytes: what these
// kernels take is launches and chains of dependent loads (lengths, entry, holder's
// count, ring), so the small sizes are one launch each, by one workgroup, and the
// large ones as few as their order allows without workgroups that wait for
// others.  Pages copied are bound by HBM: 4,200 pages of 16 tokens of 8 heads of
// 128 in four layers (2.2 GB read and written) 415-422 us, 5.2-5.3 TB/s, where a
// device copy reaches 5.05; 300 of 128 tokens in eight layers (2.5 GB) 503, 5.0.  A
// page of one K or V is one workgroup's however large it is, so few large ones take
// its time: one page of 16, 64 and 128 tokens in one layer 3.9, 6.3 and 9.8 us,
// seven in eight layers 4.3, 7.9 and 14.2 (1.7, 3.7 and 4.1 TB/s).
//
// Times of single kernels below are medians of calls that the host waits for, 1 us
// above those in a full queue.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "dfc.h"
#include "dfc_decode_core.h"
#include "dfc_paged.h"

namespace {

constexpr uint32_t kRowThreads = 256;    // of a workgroup that walks a request's row
constexpr uint32_t kPageThreads = 1024;  // of one that walks a slab of pages
constexpr uint32_t kPageWaves = kPageThreads / kWave;
constexpr uint32_t kMostSlabs = DFC_RELEASE_WORKSPACE / 4;
constexpr uint32_t kMostRequests = 65536;

__device__ __forceinline__ void tell(uint32_t *status, uint32_t bad) {
    if (bad && status) atomicOr(status, bad);
}

__device__ __forceinline__ uint64_t lanes_below() { return (uint64_t(1) << (threadIdx.x % kWave)) - 1u; }

// A cursor's free entries; none where it does not fit the ring.
struct Ring {
    uint32_t head, size, length;  // the head in the ring
    bool ok;
    // the place of entry i < length from the head on
    __device__ __forceinline__ uint32_t at(uint32_t i) const {
        return i < length - head ? head + i : i - (length - head);
    }
};
__device__ __forceinline__ Ring ring_of(const int64_t *cursor, uint32_t n_ring) {
    const int64_t head = cursor[0], tail = cursor[1];
    const bool ok = head >= 0 && tail >= head && uint64_t(tail - head) <= n_ring;
    return Ring{ok ? uint32_t(uint64_t(head) % n_ring) : 0u, ok ? uint32_t(tail - head) : 0u, n_ring, ok};
}

// The sum of a value over the workgroup, for every thread.  `part` is LDS for
// one value a wavefront.
template <uint32_t NT>
__device__ __forceinline__ uint32_t sum_of(uint32_t x, uint32_t *part) {
    const uint32_t w = __builtin_amdgcn_readlane(wave_inclusive_scan(x), kWave - 1);
    __syncthreads();  // the part before has been read
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = w;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (uint32_t k = 0; k < NT / kWave; ++k) all += part[k];
    return all;
}

// Exclusive prefix sum over the workgroup, the sum in `all`.  `part` as in sum_of.
__device__ __forceinline__ uint32_t before_of(uint32_t x, uint32_t *part, uint32_t &all) {
    const uint32_t inc = wave_inclusive_scan(x), wave = threadIdx.x / kWave;
    __syncthreads();  // the part before has been read
    if (threadIdx.x % kWave == kWave - 1) part[wave] = inc;
    __syncthreads();
    uint32_t before = inc - x;
    all = 0;
#pragma unroll
    for (uint32_t k = 0; k < kPageWaves; ++k) {
        if (k < wave) before += part[k];
        all += part[k];
    }
    return before;
}

// ------------------------------------------------------- slabs of pages

// The pages are cut into equal slabs, one a workgroup, and those into equal
// runs, one a wavefront: consecutive lanes have consecutive pages, kAtOnce
// loads are under way together.
constexpr uint32_t kAtOnce = 8;
constexpr uint32_t kSlab = kPageThreads * kAtOnce;

struct Slabs {
    uint32_t count, rounds;  // slabs; rounds of kSlab pages in each
};
Slabs slabs_of(uint32_t n_pages) {
    const uint32_t least = uint32_t(dfc::ceil_div(uint64_t(n_pages), uint64_t(kSlab)));
    const uint32_t rounds = uint32_t(dfc::ceil_div(uint64_t(least), uint64_t(kMostSlabs)));
    return Slabs{uint32_t(dfc::ceil_div(uint64_t(least), uint64_t(std::max(rounds, 1u)))), std::max(rounds, 1u)};
}

// f(page, there, value of the page) for the pages of the calling wavefront's
// run, in order, all lanes at a time.
template <typename F>
__device__ __forceinline__ void each_page(const int32_t *of, uint32_t n_pages, uint32_t rounds, F &&f) {
    const uint32_t run = rounds * kAtOnce * kWave;
    const uint64_t first = (uint64_t(blockIdx.x) * kPageWaves + threadIdx.x / kWave) * run + threadIdx.x % kWave;
    for (uint32_t r = 0; r < rounds; ++r) {
        int32_t v[kAtOnce];
        const uint64_t base = first + uint64_t(r) * kAtOnce * kWave;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) v[i] = base + i * kWave < n_pages ? of[base + i * kWave] : 0;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) f(uint32_t(base + i * kWave), base + i * kWave < n_pages, v[i]);
    }
}

// ---------------------------------------------------------------- release

struct ReleaseArgs {
    dfc_release_args a;
    uint32_t shift, slabs, rounds;
};

// The entries that a request gives up: [hole, hole + n_hole), behind the window,
// and [begin, end), behind what it keeps.
struct Given {
    uint32_t hole, n_hole, begin, n;  // n: of all
    __device__ __forceinline__ uint32_t at(uint32_t j) const { return j < n_hole ? hole + j : begin + (j - n_hole); }
};
__device__ __forceinline__ Given given_of(const ReleaseArgs &p, uint32_t r, uint32_t &bad) {
    const dfc_release_args &a = p.a;
    const uint32_t P = a.page_size;
    const int32_t held = a.held_lens[r], keep = a.keep_lens[r];
    Given g{0u, 0u, 0u, 0u};
    if (held < 0 || keep < 0 || keep > held) {
        bad |= kStatusCorrupt;
        return g;
    }
    uint32_t end = (uint32_t(held) + P - 1u) >> p.shift;
    if (end > a.max_pages) {
        bad |= uint32_t(DFC_ESIZE);
        end = a.max_pages;
    }
    g.begin = min((uint32_t(keep) + P - 1u) >> p.shift, end);
    g.hole = uint32_t((uint64_t(a.sinks) + P - 1u) >> p.shift);
    if (a.window && uint32_t(keep) + 1u > a.window) {
        const uint32_t passed = min((uint32_t(keep) + 1u - a.window) >> p.shift, g.begin);
        g.n_hole = passed > g.hole ? passed - g.hole : 0u;
    }
    g.n = g.n_hole + (end - g.begin);
    return g;
}

__device__ __forceinline__ int32_t *entry_of(const ReleaseArgs &p, uint32_t r, uint32_t i) {
    return p.a.block_table + int64_t(r) * p.a.table_stride + i;
}

// The page of an entry that is given up, -1 if it is none.
__device__ __forceinline__ int32_t given_up(const ReleaseArgs &p, int32_t *entry, int32_t page, uint32_t &bad) {
    if (page < 0) return -1;
    *entry = -1;
    if (uint32_t(page) < p.a.n_pages) return page;
    bad |= kStatusCorrupt;
    return -1;
}

// A request that is cut inside a page that others hold after the call.
__device__ __forceinline__ void look_at_cut(const ReleaseArgs &p, uint32_t r, uint32_t &bad) {
    const dfc_release_args &a = p.a;
    const int32_t held = a.held_lens[r], keep = a.keep_lens[r];
    if (keep <= 0 || keep >= held || !(uint32_t(keep) & (a.page_size - 1u))) return;
    const uint32_t i = uint32_t(keep) >> p.shift;
    if (i >= a.max_pages) return;
    const int32_t page = a.block_table[int64_t(r) * a.table_stride + i];
    if (page < 0 || uint32_t(page) >= a.n_pages) return;
    // (as the atomics left it, not as a load before them found it)
    if (__hip_atomic_load(a.shared + page, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0) bad |= uint32_t(DFC_EUNSUPPORTED);
}

// A workgroup takes a request at a time and its lanes the entries.  300 requests,
// 97 of which give up all of up to 2,048 pages, 5.2 us.
__global__ __launch_bounds__(kRowThreads) void release_kernel(ReleaseArgs p) {
    uint32_t bad = 0;
    for (uint32_t r = blockIdx.x; r < p.a.n_requests; r += gridDim.x) {
        const Given g = given_of(p, r, bad);
        for (uint32_t j = threadIdx.x; j < g.n; j += kRowThreads) {
            int32_t *entry = entry_of(p, r, g.at(j));
            const int32_t page = given_up(p, entry, *entry, bad);
            if (page >= 0 && atomicSub(p.a.shared + page, 1) < 0) bad |= kStatusCorrupt;  // more often than held
        }
    }
    tell(p.a.status_dev, bad);
}

// Free pages of every slab.  (307,000 pages 4.7 us, and 6.5 to write those that
// are free: a chain of loads, sums and stores each.)
__global__ __launch_bounds__(kPageThreads) void freed_count_kernel(ReleaseArgs p) {
    __shared__ uint32_t part[kPageWaves];
    uint32_t n = 0;
    each_page(p.a.shared, p.a.n_pages, p.rounds, [&](uint32_t, bool, int32_t v) { n += v < 0; });
    const uint32_t all = sum_of<kPageThreads>(n, part);
    if (threadIdx.x == 0) p.a.workspace_dev[blockIdx.x] = all;
}

// The free pages to the ring, their counts to 0, and the cursor.  One slab
// counts its pages itself.
__global__ __launch_bounds__(kPageThreads) void freed_write_kernel(ReleaseArgs p) {
    __shared__ uint32_t part[kPageWaves], of_wave[kPageWaves];
    const dfc_release_args &a = p.a;
    const uint32_t tid = threadIdx.x, wave = tid / kWave;
    uint32_t bad = 0, before = 0, total = 0;
    if (p.slabs > 1) {
        uint32_t mine = 0, all = 0;
        for (uint32_t k = tid; k < p.slabs; k += kPageThreads) {
            const uint32_t n = a.workspace_dev[k];
            all += n;
            if (k < blockIdx.x) mine += n;
        }
        before = sum_of<kPageThreads>(mine, part);
        total = sum_of<kPageThreads>(all, part);
    }
    uint32_t n = 0;
    each_page(a.shared, a.n_pages, p.rounds, [&](uint32_t, bool, int32_t v) { n += uint32_t(__popcll(__ballot(v < 0))); });
    if (tid % kWave == 0) of_wave[wave] = n;
    __syncthreads();
    uint32_t here = 0;
#pragma unroll
    for (uint32_t k = 0; k < kPageWaves; ++k) {
        if (k < wave) before += of_wave[k];
        here += of_wave[k];
    }
    if (p.slabs == 1) total = here;
    const Ring ring = ring_of(a.cursor, a.n_ring);
    const bool fits = ring.ok && total <= a.n_ring - ring.size;
    if (!fits) bad |= kStatusCorrupt;
    if (n) {  // (of the wavefront)
        uint32_t to = ring.size + before;  // the entry of the wavefront's next page
        each_page(a.shared, a.n_pages, p.rounds, [&](uint32_t page, bool, int32_t v) {
            const uint64_t who = __ballot(v < 0);
            if (v < 0) {
                if (fits) a.free_pages[ring.at(to + uint32_t(__popcll(who & lanes_below())))] = int32_t(page);
                a.shared[page] = 0;
            }
            to += uint32_t(__popcll(who));
        });
    }
    for (uint32_t r = blockIdx.x * kPageThreads + tid; r < a.n_requests; r += gridDim.x * kPageThreads)
        look_at_cut(p, r, bad);
    if (blockIdx.x == 0 && tid == 0) {
        const int64_t head = a.cursor[0], tail = a.cursor[1];
        a.cursor_out[0] = head;
        a.cursor_out[1] = fits ? tail + int64_t(total) : tail;
    }
    tell(a.status_dev, bad);
}

// All of it by one workgroup, for few requests: the pages that become free are
// bits in LDS, so that nothing is looked through.  A page without other holders
// becomes free at once; one with others counts one less, and whoever finds none
// left frees it and puts the count back to 0.  Both may happen to one page, whose
// bit then is set by one of them: which one makes no difference.  A lane reads a
// request's lengths and gives up a few entries by itself, as after refused drafts;
// longer runs are taken by the wavefront, eight entries a lane at a time.
//
// The call's own time here and in three launches, pages of 16 tokens, in a graph: 64
// requests of up to 8191 cut by up to five 4 and 11 us, eight of 8191 that end 6 and
// 8, a window's pages of 64 8 and 11, of 16 with 32768 8 and 12; but 32 of up to 8191
// that end 16 and 12, and 64 of 8191 37 and 13: the freed pages are written two words
// a wavefront at a time.  No size on the host tells these from the first, which a
// program makes at every step, and few of its requests end at once.
constexpr uint32_t kFewRequests = 64, kFreedWords = 4, kFewFreed = 32u * kPageThreads * kFreedWords, kFewGiven = 65536;
__global__ __launch_bounds__(kPageThreads) void release_few_kernel(ReleaseArgs p) {
    constexpr uint32_t kAlone = 2, kEach = kFewRequests / kPageWaves;
    __shared__ uint32_t freed[kPageThreads * kFreedWords], rank[kPageThreads * kFreedWords], part[kPageWaves];
    const dfc_release_args &a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const Ring ring = ring_of(a.cursor, a.n_ring);
    uint32_t bad = 0;
    Given g{0u, 0u, 0u, 0u};
    const uint32_t mine = wave + lane * kPageWaves;
    if (lane < kEach && mine < a.n_requests) g = given_of(p, mine, bad);
#pragma unroll
    for (uint32_t i = 0; i < kFreedWords; ++i) freed[i * kPageThreads + tid] = 0;
    __syncthreads();
    auto drop = [&](int32_t page, int32_t others) {
        if (page < 0) return;
        if (others > 0) {
            if (atomicSub(a.shared + page, 1) > 0) return;
            atomicAdd(a.shared + page, 1);
        }
        const uint32_t bit = 1u << (page & 31);
        if ((atomicOr(&freed[page >> 5], bit) & bit) || others < 0) bad |= kStatusCorrupt;  // more often than held
    };
    if (g.n <= kAlone)
        for (uint32_t j = 0; j < g.n; ++j) {
            int32_t *entry = entry_of(p, mine, g.at(j));
            const int32_t page = given_up(p, entry, *entry, bad);
            drop(page, page < 0 ? 0 : a.shared[page]);
        }
#pragma unroll
    for (uint32_t k = 0; k < kEach; ++k) {
        const uint32_t n = __builtin_amdgcn_readlane(g.n, k);
        if (n <= kAlone) continue;
        const Given o{uint32_t(__builtin_amdgcn_readlane(g.hole, k)), uint32_t(__builtin_amdgcn_readlane(g.n_hole, k)),
                      uint32_t(__builtin_amdgcn_readlane(g.begin, k)), n};
        for (uint32_t j0 = 0; j0 < n; j0 += kAtOnce * kWave) {
            int32_t *entry[kAtOnce], page[kAtOnce], others[kAtOnce];
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
                const uint32_t j = j0 + i * kWave + lane;
                entry[i] = entry_of(p, wave + k * kPageWaves, o.at(min(j, n - 1u)));
                page[i] = j < n ? *entry[i] : -1;
            }
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
                page[i] = given_up(p, entry[i], page[i], bad);
                others[i] = page[i] < 0 ? 0 : a.shared[page[i]];
            }
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) drop(page[i], others[i]);
        }
    }
    __syncthreads();
    uint32_t n[kFreedWords], sum = 0, total;
#pragma unroll
    for (uint32_t i = 0; i < kFreedWords; ++i) sum += n[i] = uint32_t(__popc(freed[tid * kFreedWords + i]));
    uint32_t before = before_of(sum, part, total);
#pragma unroll
    for (uint32_t i = 0; i < kFreedWords; ++i) {
        rank[tid * kFreedWords + i] = before;
        before += n[i];
    }
    __syncthreads();
    const bool fits = ring.ok && total <= a.n_ring - ring.size;
    if (!fits) bad |= kStatusCorrupt;
    // a wavefront takes every 16th word, 64 of them at once and, of those that are
    // not 0, two at a time
#pragma unroll
    for (uint32_t i = 0; i < kFreedWords; ++i) {
        const uint32_t first = wave + i * kWave * kPageWaves;
        for (uint64_t words = __ballot(freed[first + lane * kPageWaves] != 0); words;) {
            const uint32_t one = uint32_t(__builtin_ctzll(words));
            words &= words - 1u;
            const uint32_t two = words ? uint32_t(__builtin_ctzll(words)) : one;
            const uint32_t word = first + (lane < 32u ? one : two) * kPageWaves, bit = lane % 32u, x = freed[word];
            if (!words && lane >= 32u) break;  // an odd one
            words &= words - 1u;
            if (!(x >> bit & 1u)) continue;
            const uint32_t page = 32u * word + bit;
            const uint32_t at = ring.size + rank[word] + uint32_t(__popc(x & ((1u << bit) - 1u)));
            if (fits) a.free_pages[ring.at(at)] = int32_t(page);
        }
    }
    // (pages that others hold are none of those)
    if (lane < kEach && mine < a.n_requests) look_at_cut(p, mine, bad);
    if (tid == 0) {
        const int64_t tail = a.cursor[1];
        a.cursor_out[0] = a.cursor[0];
        a.cursor_out[1] = fits ? tail + int64_t(total) : tail;
    }
    tell(a.status_dev, bad);
}

// ------------------------------------------------------------------- fork

struct ForkArgs {
    dfc_fork_args a;
    uint32_t shift;
};

// What becomes of request r: whether it is forked (if the ring has its page),
// how many tokens it gets, and the page to copy (-1: none).
struct Child {
    int32_t parent, tokens, page;
    bool forked;
};
__device__ __forceinline__ Child child_of(const dfc_fork_args &a, uint32_t shift, uint32_t r, uint32_t &bad) {
    Child c{a.parents[r], 0, -1, false};
    if (c.parent == -1) return c;
    if (c.parent < 0 || uint32_t(c.parent) >= a.n_requests || a.parents[c.parent] != -1 || a.context_lens[r] != 0) {
        bad |= kStatusCorrupt;
        return c;
    }
    const int32_t has = a.context_lens[c.parent];
    c.tokens = a.fork_lens ? a.fork_lens[r] : has;
    if (c.tokens < 0 || c.tokens > has) {
        bad |= kStatusCorrupt;
        return c;
    }
    const uint32_t full = uint32_t(c.tokens) >> shift;
    const bool ends = uint32_t(c.tokens) & (a.page_size - 1u);
    if (full + ends > a.max_pages) {
        bad |= uint32_t(DFC_ESIZE);
        return c;
    }
    if (ends) {
        c.page = a.block_table[int64_t(c.parent) * a.table_stride + full];
        if (c.page < 0 || uint32_t(c.page) >= a.n_pages) {
            bad |= kStatusCorrupt;
            return c;
        }
    }
    c.forked = true;
    return c;
}

// A workgroup a request.  Those that are forked, and the last one for the
// cursor, count the pages that the requests before them take: each for itself,
// which costs a few loads a thread for some hundred requests and saves a second
// launch.  7 children of one request of 8191 tokens 5.3 us, 112 of 16 requests 5.8.
// The work grows with the square of the requests: as many children as parents, 64 of
// each 4.5 us in a graph, 512 6, 2,048 18, 8,192 133, 32,768 1,700.
__global__ __launch_bounds__(kRowThreads) void fork_kernel(ForkArgs p) {
    __shared__ uint32_t part[kRowThreads / kWave];
    const dfc_fork_args &a = p.a;
    const uint32_t r = blockIdx.x, tid = threadIdx.x;
    const Ring ring = ring_of(a.cursor, a.n_ring);
    uint32_t bad = ring.ok ? 0u : kStatusCorrupt, unused = 0;
    if (!a.n_requests) {
        if (tid == 0) a.cursor_out[0] = a.cursor[0], a.cursor_out[1] = a.cursor[1], tell(a.status_dev, bad);
        return;
    }
    Child c = child_of(a, p.shift, r, bad);
    const bool last = r == a.n_requests - 1u;
    uint32_t before = 0;
    if (last || (c.forked && c.page >= 0)) {
        for (uint32_t k = tid; k < r; k += kRowThreads) {
            const Child o = child_of(a, p.shift, k, unused);
            before += o.forked && o.page >= 0;
        }
        before = sum_of<kRowThreads>(before, part);
    }
    if (last && tid == 0) {
        const uint64_t taken = min(uint64_t(before) + (c.forked && c.page >= 0), ring.size);
        a.cursor_out[0] = a.cursor[0] + int64_t(taken);
        a.cursor_out[1] = a.cursor[1];
    }
    int32_t page = -1;
    if (c.forked && c.page >= 0) {
        if (before >= ring.size) {
            bad |= uint32_t(DFC_ESIZE);
            c.forked = false;
        } else {
            page = a.free_pages[ring.at(before)];
            if (page < 0 || uint32_t(page) >= a.n_pages) {
                bad |= kStatusCorrupt;
                c.forked = false;
            }
        }
    }
    if (tid == 0) {
        a.context_out[r] = c.parent == -1 ? a.context_lens[r] : c.forked ? c.tokens : max(a.context_lens[r], 0);
        a.src[r] = c.forked ? c.page : -1;
        a.dst[r] = c.forked ? page : -1;
    }
    if (c.forked) {
        const int32_t *from = a.block_table + int64_t(c.parent) * a.table_stride;
        int32_t *to = a.block_table + int64_t(r) * a.table_stride;
        const uint32_t full = uint32_t(c.tokens) >> p.shift;
        for (uint32_t i = tid; i < full; i += kRowThreads) {
            int32_t x = from[i];
            if (x >= 0 && uint32_t(x) >= a.n_pages) {
                bad |= kStatusCorrupt;
                x = -1;
            }
            to[i] = x;
            if (x >= 0) atomicAdd(a.shared + x, 1);
        }
        if (tid == 0 && page >= 0) to[full] = page;
    }
    tell(a.status_dev, bad);
}

// ---------------------------------------------------------------- compact

constexpr int32_t kHeld = 1, kFree = 2;

struct CompactArgs {
    dfc_compact_args a;
    uint32_t shift, slabs, rounds;
    int32_t *flags;              // per page: kHeld | kFree
    int32_t *place;              // its own number, -1 if it is not held, -2 - k if it is the k-th held one and moves
    uint32_t *held, *either;     // per slab
    uint32_t *wrong;             // ring and tables contradict each other
    uint32_t *stay;              // held pages that do not move
};

__global__ __launch_bounds__(kRowThreads) void compact_clear_kernel(CompactArgs p) {
    const dfc_compact_args &a = p.a;
    for (uint32_t i = blockIdx.x * kRowThreads + threadIdx.x; i < a.n_pages; i += gridDim.x * kRowThreads) {
        p.flags[i] = 0;
        if (i < a.n_pages / 2u) a.src[i] = a.dst[i] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.wrong = *p.stay = 0;
}

// Workgroups go through the requests' rows, then through the ring.
__global__ __launch_bounds__(kRowThreads) void compact_mark_kernel(CompactArgs p) {
    const dfc_compact_args &a = p.a;
    uint32_t bad = 0;
    bool wrong = false;
    for (uint32_t r = blockIdx.x; r < a.n_requests; r += gridDim.x) {
        const int32_t n = a.context_lens[r];
        if (n < 0) {
            bad |= kStatusCorrupt;
            continue;
        }
        uint32_t end = (uint32_t(n) + a.page_size - 1u) >> p.shift;
        if (end > a.max_pages) {
            bad |= uint32_t(DFC_ESIZE);
            end = a.max_pages;
        }
        const int32_t *row = a.block_table + int64_t(r) * a.table_stride;
        for (uint32_t i = threadIdx.x; i < end; i += kRowThreads) {
            const int32_t page = row[i];
            if (page < 0) continue;
            if (uint32_t(page) < a.n_pages)
                atomicOr(p.flags + page, kHeld);
            else
                wrong = true;
        }
    }
    const Ring ring = ring_of(a.cursor, a.n_ring);
    wrong |= !ring.ok;
    for (uint32_t i = blockIdx.x * kRowThreads + threadIdx.x; i < ring.size; i += gridDim.x * kRowThreads) {
        const int32_t page = a.free_pages[ring.at(i)];
        if (page >= 0 && uint32_t(page) < a.n_pages)
            wrong |= (atomicOr(p.flags + page, kFree) & kFree) != 0;  // twice on the ring
        else
            wrong = true;
    }
    if (wrong) atomicOr(p.wrong, 1u);
    tell(a.status_dev, bad | (wrong ? kStatusCorrupt : 0u));
}

__global__ __launch_bounds__(kPageThreads) void compact_count_kernel(CompactArgs p) {
    __shared__ uint32_t part[kPageWaves];
    uint32_t held = 0, either = 0;
    bool both = false;
    each_page(p.flags, p.a.n_pages, p.rounds, [&](uint32_t, bool, int32_t v) {
        held += (v & kHeld) != 0;
        either += v != 0;
        both |= v == (kHeld | kFree);
    });
    held = sum_of<kPageThreads>(held, part);
    either = sum_of<kPageThreads>(either, part);
    if (threadIdx.x == 0) p.held[blockIdx.x] = held, p.either[blockIdx.x] = either;
    if (both) atomicOr(p.wrong, 1u);
    tell(p.a.status_dev, both ? kStatusCorrupt : 0u);
}

__global__ __launch_bounds__(kPageThreads) void compact_place_kernel(CompactArgs p) {
    __shared__ uint32_t part[kPageWaves], held_of[kPageWaves], either_of[kPageWaves];
    const dfc_compact_args &a = p.a;
    const uint32_t tid = threadIdx.x, wave = tid / kWave;
    uint32_t held = 0, h = 0, e = 0;  // held pages; held, and either, in the slabs before this one
    {
        uint32_t all = 0, mh = 0, me = 0;
        for (uint32_t k = tid; k < p.slabs; k += kPageThreads) {
            const uint32_t x = p.held[k], y = p.either[k];
            all += x;
            if (k < blockIdx.x) mh += x, me += y;
        }
        held = sum_of<kPageThreads>(all, part);
        h = sum_of<kPageThreads>(mh, part);
        e = sum_of<kPageThreads>(me, part);
    }
    if (blockIdx.x == 0 && tid == 0) *a.used = int32_t(held);
    if (*p.wrong) {
        each_page(p.flags, a.n_pages, p.rounds, [&](uint32_t page, bool there, int32_t) {
            if (there) p.place[page] = int32_t(page);
        });
        return;
    }
    uint32_t nh = 0, ne = 0;
    each_page(p.flags, a.n_pages, p.rounds, [&](uint32_t, bool, int32_t v) {
        nh += uint32_t(__popcll(__ballot(v & kHeld)));
        ne += uint32_t(__popcll(__ballot(v != 0)));
    });
    if (tid % kWave == 0) held_of[wave] = nh, either_of[wave] = ne;
    __syncthreads();
    for (uint32_t k = 0; k < wave; ++k) h += held_of[k], e += either_of[k];
    const Ring ring = ring_of(a.cursor, a.n_ring);
    const uint64_t below = lanes_below();
    each_page(p.flags, a.n_pages, p.rounds, [&](uint32_t page, bool there, int32_t v) {
        const uint64_t hs = __ballot(v & kHeld), es = __ballot(v != 0);
        const uint32_t rank = e + uint32_t(__popcll(es & below)), before = h + uint32_t(__popcll(hs & below));
        if (there) {
            int32_t to = -1;
            if (v == kHeld) to = rank < held ? int32_t(page) : -2 - int32_t(before);
            p.place[page] = to;
            if (v == kFree && rank < held) a.dst[rank - before] = int32_t(page);
            // (the first `stay` held pages are those up to a_{U-1})
            if (v && rank + 1u == held) *p.stay = before + (v == kHeld);
            if (v && rank >= held) a.free_pages[ring.at(rank - held)] = int32_t(page);
        }
        h += uint32_t(__popcll(hs));
        e += uint32_t(__popcll(es));
    });
}

// The pages that move: the lists and their holders; and the rows.
__global__ __launch_bounds__(kRowThreads) void compact_finish_kernel(CompactArgs p) {
    const dfc_compact_args &a = p.a;
    if (*p.wrong) return;
    const uint32_t stay = *p.stay;
    for (uint32_t i = blockIdx.x * kRowThreads + threadIdx.x; i < a.n_pages; i += gridDim.x * kRowThreads) {
        const int32_t k = p.place[i];
        if (k > -2) continue;
        const uint32_t move = uint32_t(-2 - k) - stay;
        const int32_t to = a.dst[move];
        a.src[move] = int32_t(i);
        a.shared[to] = a.shared[i];
        a.shared[i] = 0;
    }
    for (uint32_t r = blockIdx.x; r < a.n_requests; r += gridDim.x) {
        const int32_t n = a.context_lens[r];
        if (n < 0) continue;
        const uint32_t end = min((uint32_t(n) + a.page_size - 1u) >> p.shift, a.max_pages);
        int32_t *row = a.block_table + int64_t(r) * a.table_stride;
        for (uint32_t i = threadIdx.x; i < end; i += kRowThreads) {
            const int32_t page = row[i];
            if (page < 0 || uint32_t(page) >= a.n_pages) continue;
            const int32_t k = p.place[page];
            if (k <= -2) row[i] = a.dst[uint32_t(-2 - k) - stay];
        }
    }
}

// All of it by one workgroup, where pages and rows' entries are a few for each of
// its threads: two bits a page in LDS, from whose sums a page's rank is read.  64
// requests of up to 500 tokens among 512 free pages take 4.5 us in a graph, and 13.5
// in five launches;
// 17,000 entries over 16,700 pages took 23 in place of 20, since one compute unit
// did all of it.
constexpr uint32_t kFewPages = kSlab, kEntries = 8, kFewEntries = kEntries * kPageThreads, kFewRows = 1024;
static_assert(kFewPages <= 32u * kPageThreads && kFewPages <= 65536u, "a word a thread, a page in 16 bits");

__global__ __launch_bounds__(kPageThreads) void compact_few_kernel(CompactArgs p) {
    __shared__ uint32_t held[kPageThreads], free[kPageThreads];
    __shared__ uint16_t pages_of[kFewRows], held_before[kPageThreads], before[kPageThreads];
    __shared__ uint16_t from[kFewPages / 2], to[kFewPages / 2];
    __shared__ uint32_t part[kPageWaves], wrong, stay;
    const dfc_compact_args &a = p.a;
    const uint32_t tid = threadIdx.x;
    const uint32_t entries = a.n_requests * a.max_pages;
    const Ring ring = ring_of(a.cursor, a.n_ring);
    uint32_t bad = 0;
    held[tid] = free[tid] = 0;
    if (tid == 0) wrong = !ring.ok, stay = 0;
    if (tid < a.n_requests) {
        const int32_t n = a.context_lens[tid];
        const uint32_t end = (uint32_t(max(n, 0)) + a.page_size - 1u) >> p.shift;
        if (n < 0) bad |= kStatusCorrupt;
        if (end > a.max_pages) bad |= uint32_t(DFC_ESIZE);
        pages_of[tid] = uint16_t(min(end, a.max_pages));
    }
    for (uint32_t i = tid; i < a.n_pages / 2u; i += kPageThreads) a.src[i] = a.dst[i] = -1;
    __syncthreads();
    // f(k, entry) for the thread's entries of the rows, kPageThreads apart
    const uint32_t width = max(a.max_pages, 1u), rows = kPageThreads / width, rest = kPageThreads - rows * width;
    auto each_entry = [&](auto &&f) {
        uint32_t r = tid / width, at = tid - r * width;
#pragma unroll
        for (uint32_t k = 0; k < kEntries; ++k) {
            if (k * kPageThreads >= entries) continue;
            f(k, r < a.n_requests && at < pages_of[r] ? a.block_table + int64_t(r) * a.table_stride + at : nullptr);
            r += rows;
            at += rest;
            if (at >= width) at -= width, ++r;
        }
    };
    int32_t page[kEntries];  // -1: none
    each_entry([&](uint32_t k, const int32_t *e) { page[k] = e ? *e : -1; });
    bool odd = false;
#pragma unroll 8
    for (uint32_t i = tid; i < ring.size; i += kPageThreads) {
        const int32_t x = a.free_pages[ring.at(i)];
        if (x >= 0 && uint32_t(x) < a.n_pages)
            odd |= atomicOr(&free[x >> 5], 1u << (x & 31)) >> (x & 31) & 1u;  // twice on the ring
        else
            odd = true;
    }
#pragma unroll
    for (uint32_t k = 0; k < kEntries; ++k) {
        if (k * kPageThreads >= entries || page[k] < 0) continue;
        if (uint32_t(page[k]) < a.n_pages)
            atomicOr(&held[page[k] >> 5], 1u << (page[k] & 31));
        else
            odd = true;
    }
    __syncthreads();
    const uint32_t h = held[tid], f = free[tid];
    if (odd || (h & f)) wrong = 1u;
    uint32_t n_held, n_either;
    held_before[tid] = uint16_t(before_of(uint32_t(__popc(h)), part, n_held));
    before[tid] = uint16_t(before_of(uint32_t(__popc(h | f)), part, n_either));
    __syncthreads();
    if (tid == 0) *a.used = int32_t(n_held);
    if (wrong) {  // (written before the barriers of the sums)
        tell(a.status_dev, bad | kStatusCorrupt);
        return;
    }
    // a page's rank among the held ones and all, from its word's
    auto place = [&](uint32_t x, uint32_t &h_rank, uint32_t &rank) {
        const uint32_t word = x >> 5, below = (1u << (x & 31)) - 1u, hw = held[word];
        h_rank = held_before[word] + uint32_t(__popc(hw & below));
        rank = before[word] + uint32_t(__popc((hw | free[word]) & below));
        return hw >> (x & 31) & 1u;
    };
    for (uint32_t x = tid; x < a.n_pages; x += kPageThreads) {
        if (!((held[x >> 5] | free[x >> 5]) >> (x & 31) & 1u)) continue;
        uint32_t h_rank, rank;
        const bool is_held = place(x, h_rank, rank);
        if (!is_held && rank < n_held) to[rank - h_rank] = uint16_t(x);
        if (rank >= n_held) a.free_pages[ring.at(rank - n_held)] = int32_t(x);
        if (rank + 1u == n_held) stay = h_rank + is_held;
    }
    __syncthreads();
    for (uint32_t x = tid; x < a.n_pages; x += kPageThreads) {
        uint32_t h_rank, rank;
        if (place(x, h_rank, rank) && rank >= n_held) from[h_rank - stay] = uint16_t(x);
    }
    __syncthreads();
    for (uint32_t i = tid; i < n_held - stay; i += kPageThreads) {
        const int32_t s = from[i], d = to[i];
        a.src[i] = s;
        a.dst[i] = d;
        a.shared[d] = a.shared[s];
        a.shared[s] = 0;
    }
    each_entry([&](uint32_t k, int32_t *e) {
        uint32_t h_rank, rank;
        if (!e || page[k] < 0) return;
        place(uint32_t(page[k]), h_rank, rank);
        if (rank >= n_held) *e = to[h_rank - stay];
    });
    tell(a.status_dev, bad);
}

// ------------------------------------------------------------------- copy

using U4 = __attribute__((ext_vector_type(4))) uint32_t;
constexpr uint32_t kCopyThreads = 256, kCopyCaches = 64, kCopyList = 1024;

struct CopyArgs {
    U4 *base[2 * kCopyCaches];  // K and V of every cache
    const int32_t *src, *dst;
    uint32_t *status;
    uint32_t n, n_pages;
    uint32_t parts;                // bases
    uint32_t groups;               // pair i belongs to group i mod groups
    uint32_t pieces;               // 16-byte pieces of a page
    uint32_t step_pairs, step_pieces;  // kCopyThreads = step_pairs pieces + step_pieces
    uint32_t heads, row;           // for pages that are not one run: heads; pieces of a head
    uint32_t k_stride[3], v_stride[3];  // in pieces
};

// A workgroup copies the pages of one group of pairs in one K or V: the pairs
// that are none are passed over first, and the threads then go through the
// others' pieces, eight loads of 16 bytes under way each.  Consecutive pairs are
// dealt out to different groups, since a list is often filled in front only.
template <bool Run>
__global__ __launch_bounds__(kCopyThreads) void copy_kernel(CopyArgs a) {
    __shared__ int2 list[kCopyList];
    __shared__ uint32_t filled;
    const uint32_t part = blockIdx.x % a.parts, group = blockIdx.x / a.parts, tid = threadIdx.x;
    if (tid == 0) filled = 0;
    __syncthreads();
    bool bad = false;
    for (uint64_t i = group + uint64_t(tid) * a.groups; i < a.n; i += uint64_t(kCopyThreads) * a.groups) {
        const int32_t from = a.src[i], to = a.dst[i];
        if (from < 0 || to < 0) continue;
        if (uint32_t(from) >= a.n_pages || uint32_t(to) >= a.n_pages) {
            bad = true;
            continue;
        }
        list[atomicAdd(&filled, 1u)] = int2{from, to};
    }
    __syncthreads();
    tell(a.status, bad ? kStatusCorrupt : 0u);
    const uint32_t n = filled;
    U4 *base = a.base[part];
    const uint32_t page_stride = part & 1u ? a.v_stride[0] : a.k_stride[0];
    const uint32_t place_stride = part & 1u ? a.v_stride[1] : a.k_stride[1];
    const uint32_t head_stride = part & 1u ? a.v_stride[2] : a.k_stride[2];
    uint32_t pair = tid / a.pieces, piece = tid % a.pieces;
    auto next = [&]() {
        pair += a.step_pairs;
        piece += a.step_pieces;
        if (piece >= a.pieces) piece -= a.pieces, ++pair;
    };
    while (pair < n) {
        constexpr uint32_t kLoads = 8;
        U4 x[kLoads];
        uint64_t to[kLoads];
        bool there[kLoads];
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) {
            // (past the last pair, its piece again, not stored)
            there[i] = pair < n;
            const int2 l = list[min(pair, n - 1u)];
            uint64_t in_page = piece;
            if constexpr (!Run) {
                const uint32_t head = piece / a.row;
                in_page = uint64_t(head / a.heads) * place_stride + uint64_t(head % a.heads) * head_stride + piece % a.row;
            }
            x[i] = base[uint64_t(uint32_t(l.x)) * page_stride + in_page];
            to[i] = uint64_t(uint32_t(l.y)) * page_stride + in_page;
            next();
        }
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i)
            if (there[i]) base[to[i]] = x[i];
    }
}

// ----------------------------------------------------------------- launch

bool pool_ok(uint32_t n_requests, uint32_t max_pages, uint32_t page_size, uint32_t n_ring, uint32_t n_pages,
             const void *table, int64_t stride, const void *lens, const void *ring, const void *cursor,
             const void *shared) {
    if (!dfc::is_pow2(page_size) || !n_ring || n_ring > 0x7fffffffu || !n_pages || n_pages > (1u << 30)) return false;
    if (!ring || !cursor || !shared) return false;
    return !n_requests || (table && lens && max_pages && max_pages <= 0x7fffffffu && stride >= int64_t(max_pages));
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) == 0; }

dfc_status launched() { return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP; }

}  // namespace

extern "C" {

dfc_status dfc_paged_release(const dfc_release_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_release_args &a = *args;
    if (!pool_ok(a.n_requests, a.max_pages, a.page_size, a.n_ring, a.n_pages, a.block_table, a.table_stride, a.held_lens,
                 a.free_pages, a.cursor, a.shared))
        return DFC_EINVAL;
    if ((a.n_requests && !a.keep_lens) || !a.cursor_out || a.cursor_out == a.cursor) return DFC_EINVAL;
    if (!a.workspace_dev || !aligned(a.workspace_dev, 16)) return DFC_EINVAL;
    if (a.window > 0x7fffffffu || a.sinks > 0x7fffffffu) return DFC_EINVAL;
    if (a.n_requests > kMostRequests) return DFC_EUNSUPPORTED;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Slabs s = slabs_of(a.n_pages);
    const ReleaseArgs p{a, dfc::log2_of(a.page_size), s.count, s.rounds};
    if (a.n_requests <= kFewRequests && a.n_pages <= kFewFreed && uint64_t(a.n_requests) * a.max_pages <= kFewGiven) {
        hipLaunchKernelGGL(release_few_kernel, dim3(1), dim3(kPageThreads), 0, st, p);
        return launched();
    }
    if (a.n_requests) hipLaunchKernelGGL(release_kernel, dim3(std::min(a.n_requests, 4096u)), dim3(kRowThreads), 0, st, p);
    if (s.count > 1) hipLaunchKernelGGL(freed_count_kernel, dim3(s.count), dim3(kPageThreads), 0, st, p);
    hipLaunchKernelGGL(freed_write_kernel, dim3(s.count), dim3(kPageThreads), 0, st, p);
    return launched();
}

dfc_status dfc_paged_fork(const dfc_fork_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_fork_args &a = *args;
    if (!pool_ok(a.n_requests, a.max_pages, a.page_size, a.n_ring, a.n_pages, a.block_table, a.table_stride, a.context_lens,
                 a.free_pages, a.cursor, a.shared))
        return DFC_EINVAL;
    if (!a.cursor_out || a.cursor_out == a.cursor) return DFC_EINVAL;
    // every workgroup reads the lengths and the parents while others write
    if (a.n_requests && (!a.parents || !a.context_out || !a.src || !a.dst || a.src == a.dst)) return DFC_EINVAL;
    for (const int32_t *out : {a.context_out, a.src, a.dst})
        if (a.n_requests && (out == a.context_lens || out == a.parents || out == a.fork_lens)) return DFC_EINVAL;
    if (a.n_requests > kMostRequests) return DFC_EUNSUPPORTED;
    const ForkArgs p{a, dfc::log2_of(a.page_size)};
    hipLaunchKernelGGL(fork_kernel, dim3(std::max(a.n_requests, 1u)), dim3(kRowThreads), 0, static_cast<hipStream_t>(stream),
                       p);
    return launched();
}

uint64_t dfc_paged_compact_workspace(uint32_t n_pages) {
    return uint64_t(n_pages) * 8u + 2u * kMostSlabs * 4u + 16u;
}

dfc_status dfc_paged_compact(const dfc_compact_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_compact_args &a = *args;
    if (!pool_ok(a.n_requests, a.max_pages, a.page_size, a.n_ring, a.n_pages, a.block_table, a.table_stride, a.context_lens,
                 a.free_pages, a.cursor, a.shared))
        return DFC_EINVAL;
    if (!a.used || (a.n_pages > 1 && (!a.src || !a.dst || a.src == a.dst))) return DFC_EINVAL;
    if (!a.workspace_dev || !aligned(a.workspace_dev, 16)) return DFC_EINVAL;
    if (a.n_requests > kMostRequests) return DFC_EUNSUPPORTED;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Slabs s = slabs_of(a.n_pages);
    CompactArgs p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    p.shift = dfc::log2_of(a.page_size);
    p.slabs = s.count;
    p.rounds = s.rounds;
    uint32_t *work = a.workspace_dev;
    p.wrong = work;
    p.stay = work + 1;
    p.held = work + 4;
    p.either = p.held + kMostSlabs;
    p.flags = reinterpret_cast<int32_t *>(p.either + kMostSlabs);
    p.place = p.flags + a.n_pages;
    if (a.n_pages <= kFewPages && a.n_requests <= kFewRows && uint64_t(a.n_requests) * a.max_pages <= kFewEntries) {
        hipLaunchKernelGGL(compact_few_kernel, dim3(1), dim3(kPageThreads), 0, st, p);
        return launched();
    }
    const uint32_t pages = std::min(uint32_t(dfc::ceil_div(uint64_t(a.n_pages), uint64_t(kRowThreads))), 2048u);
    const uint32_t ring = std::min(uint32_t(dfc::ceil_div(uint64_t(a.n_ring), uint64_t(kRowThreads))), 2048u);
    const uint32_t rows = std::min(a.n_requests, 4096u);
    hipLaunchKernelGGL(compact_clear_kernel, dim3(pages), dim3(kRowThreads), 0, st, p);
    hipLaunchKernelGGL(compact_mark_kernel, dim3(std::max(rows, ring)), dim3(kRowThreads), 0, st, p);
    hipLaunchKernelGGL(compact_count_kernel, dim3(s.count), dim3(kPageThreads), 0, st, p);
    hipLaunchKernelGGL(compact_place_kernel, dim3(s.count), dim3(kPageThreads), 0, st, p);
    hipLaunchKernelGGL(compact_finish_kernel, dim3(std::max(rows, pages)), dim3(kRowThreads), 0, st, p);
    return launched();
}

dfc_status dfc_paged_copy(const dfc_paged_cache *caches, uint32_t n_caches, const int32_t *src, const int32_t *dst,
                          uint32_t n, uint32_t *status_dev, void *stream) {
    if (n_caches && !caches) return DFC_EINVAL;
    for (uint32_t i = 0; i < n_caches; ++i) {
        const dfc_paged_cache &c = caches[i], &first = caches[0];
        const dfc_status cs = dfc::check_cache(c);
        if (cs != DFC_OK) return cs;
        if (c.n_pages != first.n_pages || c.page_size != first.page_size || c.kv_heads != first.kv_heads ||
            c.head_dim != first.head_dim || c.dtype != first.dtype)
            return DFC_EINVAL;
        for (int k = 0; k < 3; ++k) {
            if (c.k_stride[k] != first.k_stride[k] || c.v_stride[k] != first.v_stride[k]) return DFC_EINVAL;
            if (c.k_stride[k] >> 34 || c.v_stride[k] >> 34) return DFC_EUNSUPPORTED;
        }
    }
    if (!n || !n_caches) return DFC_OK;
    if (!src || !dst || src == dst || n > 0x7fffffffu) return DFC_EINVAL;
    const dfc_paged_cache &c = caches[0];
    CopyArgs a;
    std::memset(&a, 0, sizeof(a));
    a.src = src;
    a.dst = dst;
    a.status = status_dev;
    a.n = n;
    a.n_pages = c.n_pages;
    a.row = c.head_dim / 8u;
    a.heads = c.kv_heads;
    const uint64_t pieces = uint64_t(c.page_size) * c.kv_heads * a.row;
    if (pieces > 0x3fffffffull) return DFC_EUNSUPPORTED;
    a.pieces = uint32_t(pieces);
    a.step_pairs = kCopyThreads / a.pieces;
    a.step_pieces = kCopyThreads % a.pieces;
    for (int k = 0; k < 3; ++k) {
        a.k_stride[k] = uint32_t(c.k_stride[k] / 8);
        a.v_stride[k] = uint32_t(c.v_stride[k] / 8);
    }
    // a page is one run of memory, in whichever order
    auto run = [&](const int64_t (&s)[3]) {
        const int64_t dim = c.head_dim, heads = c.kv_heads, places = c.page_size;
        return (s[2] == dim && s[1] == heads * dim) || (s[1] == dim && s[2] == places * dim) ||
               (heads == 1 && s[1] == dim) || (places == 1 && s[2] == dim);
    };
    const bool whole = run(c.k_stride) && run(c.v_stride);
    hipStream_t st = static_cast<hipStream_t>(stream);
    for (uint32_t first = 0; first < n_caches; first += kCopyCaches) {
        const uint32_t here = std::min(n_caches - first, kCopyCaches);
        a.parts = 2u * here;
        for (uint32_t i = 0; i < here; ++i) {
            a.base[2 * i] = static_cast<U4 *>(caches[first + i].k_dev);
            a.base[2 * i + 1] = static_cast<U4 *>(caches[first + i].v_dev);
        }
        // pairs of a group: a workgroup's loads at least, no more than 16,384
        // workgroups, and no more pairs than its list holds
        const uint64_t fill = dfc::ceil_div(uint64_t(8u * kCopyThreads), uint64_t(a.pieces));
        const uint64_t few = dfc::ceil_div(uint64_t(n) * a.parts, uint64_t(16384));
        const uint64_t pairs = std::min<uint64_t>(std::max(fill, few), kCopyList);
        a.groups = uint32_t(dfc::ceil_div(uint64_t(n), pairs));
        const uint64_t blocks = uint64_t(a.groups) * a.parts;
        if (blocks > 0xffffffffu / kCopyThreads) return DFC_EUNSUPPORTED;  // threads of a launch, in 32 bits
        if (whole)
            hipLaunchKernelGGL((copy_kernel<true>), dim3(uint32_t(blocks)), dim3(kCopyThreads), 0, st, a);
        else
            hipLaunchKernelGGL((copy_kernel<false>), dim3(uint32_t(blocks)), dim3(kCopyThreads), 0, st, a);
    }
    return launched();
}

}  // extern "C"
