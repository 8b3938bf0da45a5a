// dfc_paged.hip - the paged key/value cache of a serving program: the plan of
// a step (pages, slots and positions from request lengths) and the append of
// a step's keys and values (with the rotary embedding).
//
// dfc_paged_plan.  Request r holds c_r tokens and brings n_r: with pages of P
// tokens it has ceil(c_r / P) pages and needs ceil((c_r + n_r) / P).  The
// missing ones come off the ring of free pages in request order, so request
// r's first new page is the exclusive sum of the missing pages before it, and
// its first new token is the exclusive sum of the new tokens before it.
//
// dfc_paged_append.  Token t's keys and values go to row slots[t] of the
// cache, rounded to its type; q and k are first rotated by the angles of
// their position: (a, b) -> (a cos - b sin, b cos + a sin) over the pairs
// (i, i + half) or (2i, 2i + 1).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dfc.h"
#include "dfc_decode_core.h"
#include "dfc_paged.h"

namespace {

// ------------------------------------------------------------------- plan

constexpr uint32_t kPlanThreads = 256;
constexpr uint32_t kPlanWaves = kPlanThreads / kWave;

struct PlanArgs {
    dfc_plan_args a;
    uint32_t page_shift;
};

// Inclusive prefix sum of 32-bit values across the wavefront, in 64 bits: the
// halves of a value add up apart from each other.
__device__ __forceinline__ uint64_t wave_scan64(uint32_t x) {
    return wave_inclusive_scan(x & 0xffffu) + (uint64_t(wave_inclusive_scan(x >> 16)) << 16);
}

// Exclusive prefix sums of (x, y) over the workgroup; the totals come back in
// sum_x and sum_y.  `part` is 2 * kPlanWaves values of LDS.
__device__ __forceinline__ void scan2(uint32_t x, uint32_t y, uint64_t &before_x, uint64_t &before_y, uint64_t &sum_x,
                                      uint64_t &sum_y, uint64_t *part) {
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint64_t ix = wave_scan64(x), iy = wave_scan64(y);
    __syncthreads();  // the previous scan's part has been read
    if (lane == kWave - 1) {
        part[wave] = ix;
        part[kPlanWaves + wave] = iy;
    }
    __syncthreads();
    before_x = ix - x;
    before_y = iy - y;
    sum_x = sum_y = 0;
#pragma unroll
    for (uint32_t w = 0; w < kPlanWaves; ++w) {
        const uint64_t px = part[w], py = part[kPlanWaves + w];
        if (w < wave) {
            before_x += px;
            before_y += py;
        }
        sum_x += px;
        sum_y += py;
    }
}

// The last j in [0, n) with key[j] <= t (key ascending, key[0] <= t).
__device__ __forceinline__ uint32_t last_at_most(const uint64_t *key, uint32_t n, uint64_t t) {
    uint32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (key[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Every workgroup scans all requests (256 at a time) and then writes its share
// of the step's tokens and new pages, in groups of 256 dealt out in turn: no
// workgroup waits for another, and one launch does it all.  Tokens and pages
// find their request by binary search in the scanned starts.  What bounds it
// is the chain of latencies (lengths, scan, search, page, store), not the
// few bytes: 64 requests of one token 4.9 us a call, 300 requests with 97
// chunks of 333 6.9 us, of which a launch that does nothing is about half.
// (Shuffles in place of the DPP scans, and workgroups of 1,024: 8.4 and 15.4.)
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs p) {
    __shared__ uint64_t part[2 * kPlanWaves];
    __shared__ uint64_t tok_start[kPlanThreads], page_start[kPlanThreads];
    __shared__ uint32_t ctx_of[kPlanThreads], have_of[kPlanThreads], need_of[kPlanThreads];
    const dfc_plan_args &a = p.a;
    const uint32_t tid = threadIdx.x, b = blockIdx.x, nb = gridDim.x;
    const uint32_t P = a.page_size, shift = p.page_shift;
    uint32_t bad = 0;
    const int64_t head0 = a.cursor[0], tail0 = a.cursor[1];
    const bool ring_ok = head0 >= 0 && tail0 >= head0 && uint64_t(tail0 - head0) <= a.n_ring;
    const uint64_t avail = ring_ok ? uint64_t(tail0 - head0) : 0;
    const uint64_t head = ring_ok ? uint64_t(head0) : 0;
    if (!ring_ok) bad |= kStatusCorrupt;
    // the page a ring rank stands for, or -1
    auto ring_page = [&](uint64_t rank) -> int32_t {
        if (rank >= avail) return -1;
        const int32_t page = a.free_pages[(head + rank) % a.n_ring];
        return page < 0 ? -1 : page;
    };
    // the first of this workgroup's groups that holds rank x or later ones
    auto first_group = [&](uint64_t x) -> uint64_t {
        const uint64_t g = x / kPlanThreads;
        return g + (b + nb - uint32_t(g % nb)) % nb;
    };
    uint64_t tok_base = 0, page_base = 0;
    for (uint32_t r0 = 0; r0 < a.n_requests; r0 += kPlanThreads) {
        const uint32_t r = r0 + tid, n_here = min(kPlanThreads, a.n_requests - r0);
        int32_t ctx = 0, n_new = 0;
        if (r < a.n_requests) {
            ctx = a.context_lens[r];
            n_new = a.new_lens[r];
            if (ctx < 0 || n_new < 0 || int64_t(ctx) + n_new > INT32_MAX) {
                bad |= kStatusCorrupt;
                ctx = max(ctx, 0);
                n_new = min(max(n_new, 0), INT32_MAX - ctx);
            }
        }
        const uint32_t total = uint32_t(ctx) + uint32_t(n_new);
        const uint32_t have0 = (uint32_t(ctx) + P - 1) >> shift, need0 = (total + P - 1) >> shift;
        if (need0 > a.max_pages) bad |= uint32_t(DFC_ESIZE);
        const uint32_t have = min(have0, a.max_pages), need = min(need0, a.max_pages);
        uint64_t ts, ps, t_sum, p_sum;
        scan2(uint32_t(n_new), need - have, ts, ps, t_sum, p_sum, part);
        ts += tok_base;
        ps += page_base;
        tok_start[tid] = ts;
        page_start[tid] = ps;
        ctx_of[tid] = uint32_t(ctx);
        have_of[tid] = have;
        need_of[tid] = need;
        if (b == 0 && r < a.n_requests) {
            a.seq_lens[r] = int32_t(total);
            a.cu_q[r] = int32_t(min(ts, a.tokens));
        }
        __syncthreads();
        // new pages of these requests
        for (uint64_t g = first_group(page_base); g * kPlanThreads < page_base + p_sum; g += nb) {
            const uint64_t j = g * kPlanThreads + tid;
            if (j < page_base || j >= page_base + p_sum) continue;
            const uint32_t k = last_at_most(page_start, n_here, j);
            const int32_t page = ring_page(j);
            if (page < 0) bad |= uint32_t(DFC_ESIZE);
            a.block_table[int64_t(r0 + k) * a.table_stride + have_of[k] + (j - page_start[k])] = page;
        }
        // new tokens of these requests
        const uint64_t t_end = min(tok_base + t_sum, a.tokens);
        for (uint64_t g = first_group(tok_base); g * kPlanThreads < t_end; g += nb) {
            const uint64_t t = g * kPlanThreads + tid;
            if (t < tok_base || t >= t_end) continue;
            const uint32_t k = last_at_most(tok_start, n_here, t);
            const uint32_t pos = ctx_of[k] + uint32_t(t - tok_start[k]);
            const uint32_t pi = pos >> shift;
            int32_t page = -1;
            if (pi < have_of[k]) {
                page = a.block_table[int64_t(r0 + k) * a.table_stride + pi];
                if (page < 0) bad |= kStatusCorrupt;
            } else if (pi < need_of[k]) {
                page = ring_page(page_start[k] + (pi - have_of[k]));
            }
            a.slots[t] = page < 0 ? -1 : (int64_t(page) << shift) + (pos & (P - 1));
            a.positions[t] = int32_t(pos);
        }
        tok_base += t_sum;
        page_base += p_sum;
        __syncthreads();  // the starts have been read
    }
    if (tok_base > a.tokens) bad |= uint32_t(DFC_ESIZE);
    // what is left of the capacity is padding
    for (uint64_t t = tok_base + uint64_t(b) * kPlanThreads + tid; t < a.tokens; t += uint64_t(nb) * kPlanThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (b == 0 && tid == 0) {
        a.cu_q[a.n_requests] = int32_t(min(tok_base, a.tokens));
        a.cursor_out[0] = head0 + int64_t(min(page_base, avail));
        a.cursor_out[1] = tail0;
    }
    if (bad && a.status_dev) atomicOr(a.status_dev, bad);
}

// ----------------------------------------------------------------- append

struct AppendArgs {
    dfc_append_args a;
    uint32_t page_shift;
    uint32_t chunks, units;      // 8-value chunks of a head; threads per head
    uint32_t per_token;          // threads per token
    uint64_t threads;
};

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 lo = *reinterpret_cast<const float4 *>(p), hi = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
    x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
}

template <typename S>
__device__ __forceinline__ void load8(const S *p, float (&x)[8]) {
    using S8 = __attribute__((ext_vector_type(8))) S;
    const S8 v = *reinterpret_cast<const S8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = float(v[i]);
}

// The pairs (x, y) of 8 turned by their angles.
__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float *cosines, const float *sines) {
    float c[8], s[8];
    load8(cosines, c);
    load8(sines, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = x[i], w = y[i];
        x[i] = u * c[i] - w * s[i];
        y[i] = w * c[i] + u * s[i];
    }
}

__device__ __forceinline__ void turn_inside(float (&x)[8], const float *cosines, const float *sines) {
    const float4 co = *reinterpret_cast<const float4 *>(cosines), si = *reinterpret_cast<const float4 *>(sines);
    const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], w = x[2 * i + 1];
        x[2 * i] = u * c[i] - w * s[i];
        x[2 * i + 1] = w * c[i] + u * s[i];
    }
}

// Eight values.  Past: they pass the L2 cache by, since nothing here reads them
// again and what is left dirty in it is written back when the kernel ends
// (300 tokens 4.0 us so and 4.2 otherwise, 1,000 6.7 and 7.6, 3,500 16.8 and
// 18.5, 8,192 35.3-39.2 and 39.3-39.8; but 64 tokens 6.6 and 6.2).
template <bool Past, typename E8, typename E>
__device__ __forceinline__ void store8(E *at, const E8 &v) {
    using U4 = __attribute__((ext_vector_type(4))) uint32_t;
    U4 *to = reinterpret_cast<U4 *>(at);
    if constexpr (Past)
        __builtin_nontemporal_store(__builtin_bit_cast(U4, v), to);
    else
        *to = __builtin_bit_cast(U4, v);
}

// One thread takes two chunks of 8 values of one head of one token: those that
// pair up half a rotation apart, elsewhere two that lie as far from each other
// as the head's other threads reach.  Every value is read and written once.
// Memory bound: 8,192 tokens of 32 + 8 heads of 128 in bfloat16 move 206 MB, in
// 35.5-39 us (5.3-5.8 TB/s; one chunk a thread, and with it every rotated value
// read twice, took 52).  64 tokens from float32 take 6 us, a launch and one chain of
// loads.
template <typename S, typename E, bool Past>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs p) {
    using E8 = __attribute__((ext_vector_type(8))) E;
    const dfc_append_args &a = p.a;
    const uint64_t base = uint64_t(blockIdx.x) * 256u;
    if (base + threadIdx.x >= p.threads) return;
    // the block's first token by one uniform division, the rest in 32 bits
    const uint64_t t_base = base / p.per_token;
    const uint32_t rest = uint32_t(base - t_base * p.per_token) + threadIdx.x;
    const uint64_t t = t_base + rest / p.per_token;
    const uint32_t in_token = rest % p.per_token;
    const uint32_t row = in_token / p.units, u = in_token % p.units;
    const uint32_t nk = a.cache.kv_heads;
    // rows of a token: k heads, v heads, q heads
    const uint32_t which = row < nk ? 0u : row < 2u * nk ? 1u : 2u;
    const uint32_t h = row - (which == 0u ? 0u : which == 1u ? nk : 2u * nk);
    const S *src;
    E *dst;
    if (which == 2u) {
        src = static_cast<const S *>(a.q_dev) + int64_t(t) * a.q_stride[0] + int64_t(h) * a.q_stride[1];
        dst = static_cast<E *>(a.q_out_dev) + int64_t(t) * a.q_out_stride[0] + int64_t(h) * a.q_out_stride[1];
    } else {
        const int64_t slot = a.slots[t];
        const uint64_t page = uint64_t(slot) >> p.page_shift;
        if (slot < 0) return;
        if (page >= a.cache.n_pages) {
            if (a.status_dev) atomicOr(a.status_dev, kStatusCorrupt);
            return;
        }
        const int64_t in_page = slot & int64_t(a.cache.page_size - 1u);
        const int64_t *st = which == 0u ? a.cache.k_stride : a.cache.v_stride;
        dst = static_cast<E *>(which == 0u ? a.cache.k_dev : a.cache.v_dev) + int64_t(page) * st[0] + in_page * st[1] +
              int64_t(h) * st[2];
        src = which == 0u ? static_cast<const S *>(a.k_dev) + int64_t(t) * a.k_src_stride[0] + int64_t(h) * a.k_src_stride[1]
                          : static_cast<const S *>(a.v_dev) + int64_t(t) * a.v_src_stride[0] + int64_t(h) * a.v_src_stride[1];
    }
    const uint32_t turned = which == 1u ? 0u : a.rot_dim / 8u;  // chunks that are rotated, an even number
    const uint32_t c0 = u < turned / 2u ? u : u + turned / 2u;
    const uint32_t c1 = u < turned / 2u ? u + turned / 2u : c0 + p.units - turned / 2u;
    const bool two = c1 < p.chunks;
    float x[8], y[8] = {};
    load8(src + 8u * c0, x);
    if (two) load8(src + 8u * c1, y);
    if (c0 < turned) {
        int32_t pos = a.positions[t];
        if (pos < 0 || uint32_t(pos) >= a.max_positions) {
            if (a.status_dev) atomicOr(a.status_dev, kStatusCorrupt);
            pos = 0;
        }
        const float *cosines = a.rotary_dev + int64_t(pos) * a.rot_dim, *sines = cosines + a.rot_dim / 2u;
        if (a.interleaved) {
            turn_inside(x, cosines + 4u * c0, sines + 4u * c0);
            turn_inside(y, cosines + 4u * c1, sines + 4u * c1);
        } else {
            turn(x, y, cosines + 8u * c0, sines + 8u * c0);
        }
    }
    E8 out;
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = E(x[i]);
    store8<Past>(dst + 8u * c0, out);
    if (two) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = E(y[i]);
        store8<Past>(dst + 8u * c1, out);
    }
}

template <typename S, typename E>
void launch_append(const AppendArgs &p, uint32_t blocks, hipStream_t stream) {
    // 32 bytes a thread
    if (p.threads * 32u > (2u << 20))
        hipLaunchKernelGGL((append_kernel<S, E, true>), dim3(blocks), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((append_kernel<S, E, false>), dim3(blocks), dim3(256), 0, stream, p);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" {

dfc_status dfc_paged_plan(const dfc_plan_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_plan_args &a = *args;
    if (!dfc::is_pow2(a.page_size) || a.tokens > 0x7fffffffull || a.n_requests > 0x7fffffffu) return DFC_EINVAL;
    if (!a.cursor || !a.cursor_out || a.cursor == a.cursor_out || !a.cu_q) return DFC_EINVAL;
    if (a.n_requests && (!a.context_lens || !a.new_lens || !a.seq_lens || !a.block_table || !a.max_pages ||
                         a.table_stride < int64_t(a.max_pages)))
        return DFC_EINVAL;
    // every workgroup reads the lengths while one writes seq_lens and cu_q
    if (a.n_requests && (a.seq_lens == a.context_lens || a.seq_lens == a.new_lens || a.cu_q == a.context_lens ||
                         a.cu_q == a.new_lens))
        return DFC_EINVAL;
    if (a.tokens && (!a.slots || !a.positions)) return DFC_EINVAL;
    if (!a.n_ring || !a.free_pages) return DFC_EINVAL;
    PlanArgs p{a, dfc::log2_of(a.page_size)};
    const uint32_t groups = uint32_t(dfc::ceil_div(a.tokens, uint64_t(kPlanThreads)));
    const uint32_t blocks = std::min(std::max(groups, 1u), 256u);
    hipLaunchKernelGGL(plan_kernel, dim3(blocks), dim3(kPlanThreads), 0, static_cast<hipStream_t>(stream), p);
    return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP;
}

dfc_status dfc_paged_append(const dfc_append_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_append_args &a = *args;
    const dfc_status cs = dfc::check_cache(a.cache);
    if (cs != DFC_OK) return cs;
    if (a.tokens > 0x7fffffffull) return DFC_EINVAL;
    if (a.source_dtype != DFC_BF16 && a.source_dtype != DFC_F16 && a.source_dtype != DFC_F32) return DFC_EUNSUPPORTED;
    if (a.source_dtype != DFC_F32 && a.source_dtype != a.cache.dtype) return DFC_EUNSUPPORTED;
    if (a.rot_dim % 16u || a.rot_dim > a.cache.head_dim) return DFC_EINVAL;
    if (a.rot_dim && (!a.rotary_dev || !a.max_positions || !aligned16(a.rotary_dev))) return DFC_EINVAL;
    if (a.q_heads > 65536u) return DFC_EINVAL;
    if (!a.tokens) return DFC_OK;
    if (!a.k_dev || !a.v_dev || !a.slots || (a.rot_dim && !a.positions)) return DFC_EINVAL;
    if (a.q_heads && (!a.q_dev || !a.q_out_dev)) return DFC_EINVAL;
    if (!aligned16(a.k_dev) || !aligned16(a.v_dev)) return DFC_EINVAL;
    // strides in whole 16-byte pieces
    const int64_t unit = a.source_dtype == DFC_F32 ? 4 : 8;
    for (int i = 0; i < 2; ++i)
        if (a.k_src_stride[i] % unit || a.v_src_stride[i] % unit) return DFC_EINVAL;
    if (a.q_heads) {
        if (!aligned16(a.q_dev) || !aligned16(a.q_out_dev)) return DFC_EINVAL;
        for (int i = 0; i < 2; ++i)
            if (a.q_stride[i] % unit || a.q_out_stride[i] % 8) return DFC_EINVAL;
        if (a.q_dev == a.q_out_dev && (a.rot_dim || a.source_dtype == DFC_F32)) return DFC_EINVAL;
    }
    AppendArgs p;
    p.a = a;
    p.page_shift = dfc::log2_of(a.cache.page_size);
    p.chunks = a.cache.head_dim / 8u;
    p.units = (p.chunks + 1u) / 2u;
    p.per_token = p.units * (a.q_heads + 2u * a.cache.kv_heads);
    p.threads = uint64_t(p.per_token) * a.tokens;
    const uint64_t blocks = dfc::ceil_div(p.threads, uint64_t(256));
    if (blocks > 0x7fffffffull) return DFC_EUNSUPPORTED;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool bf = a.cache.dtype == DFC_BF16;
    if (a.source_dtype == DFC_F32)
        bf ? launch_append<float, __bf16>(p, uint32_t(blocks), st) : launch_append<float, _Float16>(p, uint32_t(blocks), st);
    else
        bf ? launch_append<__bf16, __bf16>(p, uint32_t(blocks), st)
           : launch_append<_Float16, _Float16>(p, uint32_t(blocks), st);
    return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP;
}

}  // extern "C"
