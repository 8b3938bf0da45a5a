// dfc_attention_schedule.h - how a step's attention is cut into pieces of work
// (internal to dfc_attention.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "dfc.h"
#include "dfc_decode_core.h"

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = 4;

// One piece of work: a tile of rows of one request and a range of keys, for
// one cache head.  With sinks, keys are counted without those between the
// sinks and the window, which no row of the tile sees: see key_at.
struct Piece {
    uint32_t req, row0;     // request; first row of the tile
    int32_t q_start, q_len, kv_len;
    int32_t lo, hi;         // keys
    int32_t gap;            // left out behind the sinks
    uint32_t split, splits; // which piece of the tile, of how many
    uint32_t slot;          // first partial result of the tile (splits > 1)
};

// A tile of a request whose tiles are split, for the joining of its pieces.
struct alignas(16) Tile {
    uint32_t splits, slot;  // pieces; the first one's partial result
    int32_t token0;         // row of q of the request's first token
    uint32_t row0, rows;
    uint32_t pad[3];
};

struct AttnArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *cu_q, *seq_lens;
    int64_t q_stride[2], out_stride[2], table_stride;
    uint32_t k_units[3], v_units[3];  // strides of the cache in 16-byte pieces
    uint32_t n_pages, page_shift, kv_heads, group, heads, dim;
    uint32_t n_requests, tokens, max_pages, window;
    int32_t causal;
    float scale, scale_log2;   // scores by exp2: scale log2(e)
    uint32_t rows_per_tile, key_tile, rows_shift, key_shift;  // powers of two
    uint32_t min_piece;  // a piece has min_piece key tiles or more
    uint32_t resident;         // workgroups that run at once
    // in key tiles: what a piece costs beside its keys, one of several of a
    // tile more (its sums written and read again), and the joining
    float piece_cost, split_cost, join_cost;
    uint32_t extra;            // pieces there may be beyond one a tile
    uint32_t tile_cap;
    uint32_t join_shares;      // shares a tile's rows are joined in
    uint32_t *tile_count;      // tiles[] written
    Tile *tiles;               // null: no tile can be split
    float *part_o, *part_ml;
    uint32_t *status;
    int32_t sinks, sink_end;   // tokens that stay visible; the same up to a whole key tile
};

// The token of a piece's key.  Both ends of the gap are multiples of the key
// tile, so a tile of keys is a tile of tokens.
template <bool Sinks>
__device__ __forceinline__ int32_t key_at(const AttnArgs &a, const Piece &w, int32_t key) {
    return Sinks && key >= a.sink_end ? key + w.gap : key;
}
// The end of a piece's tokens.
template <bool Sinks>
__device__ __forceinline__ int32_t end_of(const AttnArgs &a, const Piece &w) {
    return Sinks && w.hi > a.sink_end ? w.hi + w.gap : w.hi;
}

// -------------------------------------------------------------- schedule
//
// Every workgroup finds its own piece from the step's lengths.  A request's
// tiles (n of them, the longest of c key tiles) are cut into S = ceil(c / L)
// pieces each, so the pieces before a request are a prefix sum of n S, and
// what all workgroups have to agree on is L.  Reading the lengths costs each
// workgroup about a microsecond; a kernel that lists the pieces first, and
// its launch, cost the step more than ten (700 keys: 23.9 us so, 12.5 this way).

struct Req {
    int32_t q_start, q_len, kv_len;
};

// A request's ranges, held inside the buffers whatever the lengths say.
__device__ __forceinline__ Req request(const AttnArgs &a, uint32_t r, uint32_t &bad) {
    Req q;
    const int32_t c0 = a.cu_q[r], c1 = a.cu_q[r + 1];
    q.q_start = min(max(c0, 0), int32_t(a.tokens));
    q.q_len = min(max(c1, q.q_start), int32_t(a.tokens)) - q.q_start;
    const int64_t room = int64_t(a.max_pages) << a.page_shift;
    const int32_t s = a.seq_lens[r];
    const int32_t most = int32_t(min(room, int64_t(0x7fffff00)));  // a key tile past it is still an int
    q.kv_len = min(max(s, 0), most);
    if (c0 < 0 || c1 < c0 || c1 > int32_t(a.tokens) || q.kv_len != s) bad |= kStatusCorrupt;
    return q;
}

// Keys [first, hi) that the rows row0 .. of a tile see between them, and lo,
// first rounded down to a multiple of the key tile.  With sinks, lo is 0, and
// lo and hi leave out the `gap` keys between the sinks' last tile and the
// window's first.
template <bool Sinks>
__device__ __forceinline__ void tile_keys(const AttnArgs &a, const Req &q, uint32_t row0, int32_t &lo, int32_t &hi,
                                          int32_t &first, int32_t &gap) {
    const int32_t t0 = int32_t(row0 / a.group);
    const int32_t rows = int32_t(min(a.rows_per_tile, uint32_t(q.q_len) * a.group - row0));
    const int32_t t1 = int32_t((row0 + uint32_t(rows) - 1) / a.group);
    const int64_t base = int64_t(q.kv_len) - q.q_len;
    const int64_t end = a.causal ? min(int64_t(q.kv_len), base + t1 + 1) : int64_t(q.kv_len);
    const int64_t begin = a.window ? max(int64_t(0), base + t0 + 1 - int64_t(a.window)) : 0;
    hi = int32_t(max(end, int64_t(0)));
    first = int32_t(min(begin, int64_t(hi)));
    lo = first >> a.key_shift << a.key_shift;
    gap = 0;
    if constexpr (Sinks) {
        gap = max(lo - a.sink_end, 0);
        lo = 0;
        hi -= gap;
    }
}

__device__ __forceinline__ uint32_t key_tiles(const AttnArgs &a, int32_t lo, int32_t hi) {
    return (uint32_t(hi - lo) + a.key_tile - 1u) >> a.key_shift;
}

__device__ __forceinline__ uint32_t ceil_of(uint32_t x, uint32_t y) { return (x + y - 1u) / y; }

// Tiles of rows of a request, and the key tiles of its last one (the longest
// but for a window's edge).
template <bool Sinks>
__device__ __forceinline__ void tiles_of(const AttnArgs &a, const Req &q, uint32_t &n, uint32_t &c) {
    n = (uint32_t(q.q_len) * a.group + a.rows_per_tile - 1u) >> a.rows_shift;
    c = 0;
    if (n) {
        int32_t lo, hi, first, gap;
        tile_keys<Sinks>(a, q, (n - 1u) * a.rows_per_tile, lo, hi, first, gap);
        c = key_tiles(a, lo, hi);
    }
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d; d /= 2) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// L for up to 64 requests, one a lane: every lane tries one value, counts the
// pieces p it makes and takes
//     rounds (L + piece_cost + split_cost) + join_cost,
//     rounds = ceil(p heads / resident),
// for its time (the last two costs where something is split); the least wins.
// Cutting one long request into as many equal pieces as run at once, cutting
// many ragged ones finer so that the last round is full, and not cutting where
// it does not pay all come out of it.
// The wavefronts count a share of the requests each: one that counts all of
// 64 takes 2 us, which the workgroups left without a piece spend as well.
template <uint32_t NT>
__device__ __forceinline__ uint32_t choose_piece(const AttnArgs &a, uint32_t n, uint32_t c, uint32_t *scratch) {
    constexpr uint32_t kShares = NT / kWave;
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    uint32_t longest = c;
#pragma unroll
    for (int d = 32; d; d /= 2) longest = max(longest, uint32_t(__shfl_xor(longest, d)));
    const float parts = lane < 32u ? float(lane + 1u) : 32.0f * __builtin_amdgcn_exp2f(float(lane - 31u) * 0.15625f);
    // (the first lane's leaves every tile whole)
    const uint32_t piece = max(a.min_piece, lane ? uint32_t(ceilf(float(longest) / parts)) : longest);
    const float inv = 1.0f / float(piece);
    const bool shared = a.n_requests > 4u;
    uint64_t more = 0;  // pieces beyond one a tile
    for (uint32_t r = shared ? wave : 0u; r < a.n_requests; r += shared ? kShares : 1u) {
        const uint32_t nr = __builtin_amdgcn_readlane(n, r), cr = __builtin_amdgcn_readlane(c, r);
        uint32_t s = uint32_t(float(cr) * inv);  // never below ceil(c / piece) after this
        s += s * piece < cr;
        s += s * piece < cr;
        more += uint64_t(nr) * (max(s, 1u) - 1u);
    }
    if (shared) {
        uint64_t *sums = reinterpret_cast<uint64_t *>(scratch);
        sums[threadIdx.x] = more;
        __syncthreads();
        more = 0;
#pragma unroll
        for (uint32_t k = 0; k < kShares; ++k) more += sums[k * kWave + lane];
        __syncthreads();  // read by all before the scratch is used again
    }
    const uint32_t tiles = __builtin_amdgcn_readlane(wave_inclusive_scan(n), 63);
    const float rounds = ceilf(float(more + tiles) * float(a.kv_heads) / float(a.resident));
    const bool split = piece < longest;
    float t = rounds * (float(piece) + a.piece_cost + (split ? a.split_cost : 0.0f));
    if (split) t += a.join_cost;
    if (more > a.extra) t = 3e38f;
    const float best = -wave_max(-t);
    const uint32_t who = __builtin_ctzll(__ballot(t == best));
    return __builtin_amdgcn_readlane(piece, who);
}

// The piece `index` of the step (for every cache head), false if there is
// none.  `scratch` is LDS that nothing else uses meanwhile.  Row ranges that
// overlap could make more tiles than q has room for: then there are none.
// Called by all NT threads of the workgroup.
template <uint32_t NT, bool Sinks>
__device__ __forceinline__ bool find_piece(const AttnArgs &a, uint32_t index, bool first, uint32_t *scratch, Piece &w) {
    const uint32_t tid = threadIdx.x, lane = tid % kWave;
    uint32_t bad = 0;
    uint32_t within = 0, parts = 1, n_tiles = 0, slot0 = 0, tile0 = 0, piece = 1;
    if (a.n_requests <= 64) {
        Req q{0, 0, 0};
        if (lane < a.n_requests) q = request(a, lane, bad);
        uint32_t n, c;
        tiles_of<Sinks>(a, q, n, c);
        piece = a.extra ? choose_piece<NT>(a, n, c, scratch) : 1u << 30;
        const uint32_t s = max(1u, ceil_of(c, piece)), x = n * s, y = s > 1u ? x : 0u, z = s > 1u ? n : 0u;
        const uint32_t ix = wave_inclusive_scan(x), iy = wave_inclusive_scan(y), iz = wave_inclusive_scan(z);
        const uint32_t in = wave_inclusive_scan(n);
        const bool fits = uint32_t(__builtin_amdgcn_readlane(in, 63)) <= a.tile_cap;
        if (!fits) bad |= kStatusCorrupt;
        if (first && tid == 63) *a.tile_count = fits ? iz : 0u;
        if (first && bad && a.status) atomicOr(a.status, bad);
        if (!fits || index >= uint32_t(__builtin_amdgcn_readlane(ix, 63))) return false;
        const uint32_t r = 63u - uint32_t(__builtin_clzll(__ballot(x > 0u && ix - x <= index)));
        within = index - uint32_t(__builtin_amdgcn_readlane(ix - x, r));
        parts = __builtin_amdgcn_readlane(s, r);
        n_tiles = __builtin_amdgcn_readlane(n, r);
        slot0 = __builtin_amdgcn_readlane(iy - y, r);
        tile0 = __builtin_amdgcn_readlane(iz - z, r);
        w.req = r;
        w.q_start = __builtin_amdgcn_readlane(q.q_start, r);
        w.q_len = __builtin_amdgcn_readlane(q.q_len, r);
        w.kv_len = __builtin_amdgcn_readlane(q.kv_len, r);
    } else {
        // more requests than lanes: L from the sum of their key tiles
        const uint32_t wave = tid / kWave;
        uint64_t *sums = reinterpret_cast<uint64_t *>(scratch);
        uint64_t all = 0, tiles = 0;
        for (uint32_t r = tid; r < a.n_requests; r += NT) {
            uint32_t n, c;
            tiles_of<Sinks>(a, request(a, r, bad), n, c);
            all += uint64_t(n) * c;
            tiles += n;
        }
#pragma unroll
        for (int d = 32; d; d /= 2) {
            all += __shfl_xor(all, d);
            tiles += __shfl_xor(tiles, d);
        }
        if (lane == 0) sums[wave] = all, sums[NT / 64u + wave] = tiles;
        __syncthreads();
        all = tiles = 0;
        for (uint32_t k = 0; k < NT / 64u; ++k) all += sums[k], tiles += sums[NT / 64u + k];
        all *= a.kv_heads;
        const bool fits = tiles <= a.tile_cap;
        if (!fits) bad |= kStatusCorrupt;
        const uint64_t target = uint64_t(a.extra) * a.kv_heads;
        // with about as many tiles as run at once, pieces are not worth
        // their joining below some length (80 requests of 5 tokens over 700:
        // 85 us cut in two, 58 whole)
        const uint32_t least = tiles * a.kv_heads >= a.resident ? 24u : a.min_piece;
        piece = a.extra ? uint32_t(min(uint64_t(1) << 30, max(uint64_t(least), (all + target - 1u) / target)))
                        : 1u << 30;
        uint32_t px = 0, py = 0, pz = 0;  // before this chunk of requests
        uint32_t *found = scratch + NT / 16u, *part = found + 16;
        if (tid == 0) found[0] = 0;
        for (uint32_t r0 = 0; r0 < a.n_requests; r0 += NT) {
            Req q{0, 0, 0};
            uint32_t unused = 0, n, c;
            if (r0 + tid < a.n_requests) q = request(a, r0 + tid, unused);
            tiles_of<Sinks>(a, q, n, c);
            const uint32_t s = max(1u, ceil_of(c, piece)), x = n * s, y = s > 1u ? x : 0u, z = s > 1u ? n : 0u;
            uint32_t ix = wave_inclusive_scan(x), iy = wave_inclusive_scan(y), iz = wave_inclusive_scan(z);
            __syncthreads();  // part has been read
            if (lane == 63u) part[3u * wave] = ix, part[3u * wave + 1u] = iy, part[3u * wave + 2u] = iz;
            __syncthreads();
            ix += px, iy += py, iz += pz;
            for (uint32_t k = 0; k < NT / 64u; ++k) {
                const uint32_t tx = part[3u * k], ty = part[3u * k + 1u], tz = part[3u * k + 2u];
                if (k < wave) ix += tx, iy += ty, iz += tz;
                px += tx, py += ty, pz += tz;
            }
            if (ix - x <= index && index < ix) {
                found[0] = 1;
                found[1] = r0 + tid, found[2] = uint32_t(q.q_start), found[3] = uint32_t(q.q_len);
                found[4] = uint32_t(q.kv_len), found[5] = index - (ix - x), found[6] = s, found[7] = n;
                found[8] = iy - y, found[9] = iz - z;
            }
            if (!first && px > index) break;  // this chunk had it
        }
        __syncthreads();
        if (first && tid == 0) *a.tile_count = fits ? pz : 0u;
        if (first && bad && a.status) atomicOr(a.status, bad);
        uint32_t f[10];
#pragma unroll
        for (int i = 0; i < 10; ++i) f[i] = __builtin_amdgcn_readfirstlane(found[i]);
        __syncthreads();  // read by all before the scratch is used again
        if (!f[0] || !fits) return false;
        w.req = f[1];
        w.q_start = int32_t(f[2]), w.q_len = int32_t(f[3]), w.kv_len = int32_t(f[4]);
        within = f[5], parts = f[6], n_tiles = f[7], slot0 = f[8], tile0 = f[9];
    }
    // the later tiles of a request see more keys: they come first
    const uint32_t tile = within / parts;
    w.split = within - tile * parts;
    w.row0 = (n_tiles - 1u - tile) * a.rows_per_tile;
    int32_t lo, hi, seen;
    tile_keys<Sinks>(a, Req{w.q_start, w.q_len, w.kv_len}, w.row0, lo, hi, seen, w.gap);
    const uint32_t c = key_tiles(a, lo, hi);
    w.splits = min(parts, max(1u, ceil_of(c, piece)));
    w.slot = slot0 + tile * parts;
    // even shares of the key tiles
    w.lo = lo + int32_t(uint32_t(uint64_t(c) * w.split / w.splits) * a.key_tile);
    w.hi = min(hi, lo + int32_t(uint32_t(uint64_t(c) * (w.split + 1u) / w.splits) * a.key_tile));
    if (parts > 1u && w.split == 0u && threadIdx.x == 0 && blockIdx.x % a.kv_heads == 0) {
        Tile t;
        t.splits = w.splits;
        t.slot = w.slot;
        t.token0 = w.q_start;
        t.row0 = w.row0;
        t.rows = min(a.rows_per_tile, uint32_t(w.q_len) * a.group - w.row0);
        a.tiles[tile0 + tile] = t;
    }
    return w.split < w.splits;
}

}  // namespace
