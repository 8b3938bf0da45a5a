// dfc_attention.hip - attention of a step's new tokens over the paged cache.
//
// Token i of request r (n_r new tokens, s_r tokens in all) stands at position
// p = s_r - n_r + i and sees the keys j < s_r with j <= p (causal) and
// j > p - window.  For each of its heads, which share the keys and values of
// one cache head in groups of G = heads / kv_heads,
//     o = sum_j exp(z_j - m) v_j / sum_j exp(z_j - m),  z_j = scale q . k_j,
// in one pass over the keys: m is a running reference no smaller than the
// running maximum less a slack, and the sums are rescaled when it moves.
//
// Rows.  The n_r G (token, head of the group) pairs of a request and cache
// head are its rows; a tile is 32 RW of them, 32 per wavefront.  A workgroup
// of four wavefronts takes one tile and one piece of its keys: RW wavefronts
// along the rows times 4 / RW groups along the keys, whose results it joins
// at the end.
//
// Layout.  Scores are computed transposed, S^T = K Q^T, with 32x32x16
// MFMA: lane l then holds, for the row l mod 32, the keys 8 (r / 4) +
// 4 (l / 32) + r mod 4 of each block of 32 (r = 0..15), so a row's maximum
// and sum are in-lane sums and one exchange with lane l ^ 32, and the
// rounded probabilities are, as they stand, the B operand of O^T = V^T P^T
// (the order of the keys within a step of 16 is free as long as V^T follows
// it: the transposing LDS read gives each lane those four keys at its
// column).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "dfc.h"
#include "dfc_decode_core.h"
#include "dfc_paged.h"

namespace {

using f32x16 = __attribute__((ext_vector_type(16))) float;
using s16x4 = __attribute__((ext_vector_type(4))) short;

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = 4;

// One piece of work: a tile of rows of one request and a range of keys, for
// one cache head.
struct Piece {
    uint32_t req, row0;     // request; first row of the tile
    int32_t q_start, q_len, kv_len;
    int32_t lo, hi;         // keys
    uint32_t split, splits; // which piece of the tile, of how many
    uint32_t slot;          // first partial result of the tile (splits > 1)
    uint32_t tile;          // number of the tile in the step
};

// A tile, for the joining of its pieces.
struct alignas(16) Tile {
    uint32_t splits, slot;
    int32_t token0;         // row of q of the request's first token
    uint32_t row0, rows;
    uint32_t pad[3];
};

struct AttnArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *cu_q, *seq_lens;
    int64_t q_stride[2], out_stride[2], k_stride[3], v_stride[3], table_stride;
    uint32_t n_pages, page_shift, kv_heads, group, heads, dim;
    uint32_t n_requests, tokens, max_pages, window;
    int32_t causal;
    int32_t simple_rows;       // K and V have one layout, and a load's rows lie in one page
    uint32_t page_units, slot_units;  // its strides in 16-byte pieces (simple_rows)
    float scale, scale_log2;   // scores by exp2: scale log2(e)
    uint32_t rows_per_tile, key_tile, min_piece;  // a piece has min_piece key tiles or more
    uint32_t resident;         // workgroups that run at once
    float piece_cost, join_cost;  // what a piece, and the joining, cost in key tiles
    uint32_t extra;            // pieces there may be beyond one a tile
    uint32_t tile_cap;
    uint32_t *tile_count;
    Tile *tiles;               // null: no tile can be split
    float *part_o, *part_ml;
    uint32_t *status;
};

// -------------------------------------------------------------- schedule
//
// Every workgroup finds its own piece from the step's lengths.  A request's
// tiles (n of them, the longest of c key tiles) are cut into S = ceil(c / L)
// pieces each, so the pieces before a request are a prefix sum of n S, and
// what all workgroups have to agree on is L.  Reading the lengths costs each
// workgroup about a microsecond; a kernel that lists the pieces first, and
// its launch, cost the step more than ten.

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

// Keys [lo, hi) that the rows row0 .. of a tile see between them, lo at a
// multiple of the key tile.
__device__ __forceinline__ void tile_keys(const AttnArgs &a, const Req &q, uint32_t row0, int32_t &lo, int32_t &hi) {
    const int32_t t0 = int32_t(row0 / a.group);
    const int32_t rows = int32_t(min(uint64_t(a.rows_per_tile), uint64_t(q.q_len) * a.group - row0));
    const int32_t t1 = int32_t((row0 + uint32_t(rows) - 1) / a.group);
    const int64_t base = int64_t(q.kv_len) - q.q_len;
    const int64_t end = a.causal ? min(int64_t(q.kv_len), base + t1 + 1) : int64_t(q.kv_len);
    int64_t begin = a.window ? max(int64_t(0), base + t0 + 1 - int64_t(a.window)) : 0;
    begin = begin / a.key_tile * a.key_tile;
    hi = int32_t(max(end, int64_t(0)));
    lo = int32_t(min(begin, int64_t(hi)));
}

__device__ __forceinline__ uint32_t key_tiles(const AttnArgs &a, int32_t lo, int32_t hi) {
    return (uint32_t(hi - lo) + a.key_tile - 1u) / a.key_tile;
}

__device__ __forceinline__ uint32_t ceil_of(uint32_t x, uint32_t y) { return (x + y - 1u) / y; }

// Tiles of rows of a request, and the key tiles of its last one (the longest
// but for a window's edge).
__device__ __forceinline__ void tiles_of(const AttnArgs &a, const Req &q, uint32_t &n, uint32_t &c) {
    n = uint32_t((uint64_t(uint32_t(q.q_len)) * a.group + a.rows_per_tile - 1u) / a.rows_per_tile);
    c = 0;
    if (n) {
        int32_t lo, hi;
        tile_keys(a, q, (n - 1u) * a.rows_per_tile, lo, hi);
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
//     rounds (L + piece_cost), rounds = ceil(p heads / resident),
// for its time; the least wins.  Cutting one long request into as many equal
// pieces as run at once, cutting many ragged ones finer so that the last
// round is full, and not cutting where it does not pay all come out of it.
__device__ __forceinline__ uint32_t choose_piece(const AttnArgs &a, uint32_t n, uint32_t c) {
    const uint32_t lane = threadIdx.x % kWave;
    const float longest = wave_max(float(c));
    const float parts = lane < 32u ? float(lane + 1u) : 32.0f * __builtin_amdgcn_exp2f(float(lane - 31u) * 0.15625f);
    const uint32_t piece = max(a.min_piece, uint32_t(ceilf(longest / parts)));
    const float inv = 1.0f / float(piece);
    uint64_t p = 0;
    uint32_t tiles = 0;
    for (uint32_t r = 0; r < a.n_requests; ++r) {
        const uint32_t nr = __builtin_amdgcn_readlane(n, r), cr = __builtin_amdgcn_readlane(c, r);
        uint32_t s = uint32_t(float(cr) * inv);  // never below ceil(c / piece) after this
        s += s * piece < cr;
        s += s * piece < cr;
        tiles += nr;
        p += uint64_t(nr) * max(s, 1u);
    }
    const float rounds = ceilf(float(p) * float(a.kv_heads) / float(a.resident));
    float t = rounds * (float(piece) + a.piece_cost);
    if (float(piece) < longest) t += a.join_cost;
    if (p - tiles > a.extra) t = 3e38f;
    const float best = -wave_max(-t);
    const uint32_t who = __builtin_ctzll(__ballot(t == best));
    return __builtin_amdgcn_readlane(piece, who);
}

// The piece `index` of the step (for every cache head), false if there is
// none.  `scratch` is LDS that nothing else uses meanwhile.  Row ranges that
// overlap could make more tiles than q has room for: then there are none.
__device__ __forceinline__ bool find_piece(const AttnArgs &a, uint32_t index, bool first, uint32_t *scratch, Piece &w) {
    const uint32_t tid = threadIdx.x, lane = tid % kWave;
    uint32_t bad = 0;
    uint32_t within = 0, parts = 1, n_tiles = 0, slot0 = 0, tile0 = 0, piece = 1;
    if (a.n_requests <= 64) {
        Req q{0, 0, 0};
        if (lane < a.n_requests) q = request(a, lane, bad);
        uint32_t n, c;
        tiles_of(a, q, n, c);
        piece = a.extra ? choose_piece(a, n, c) : 1u << 30;
        const uint32_t s = max(1u, ceil_of(c, piece)), x = n * s, y = s > 1u ? x : 0u;
        const uint32_t ix = wave_inclusive_scan(x), iy = wave_inclusive_scan(y), in = wave_inclusive_scan(n);
        const bool fits = uint32_t(__builtin_amdgcn_readlane(in, 63)) <= a.tile_cap;
        if (!fits) bad |= kStatusCorrupt;
        if (first && tid == 63) *a.tile_count = fits ? in : 0u;
        if (first && bad && a.status) atomicOr(a.status, bad);
        if (!fits || index >= uint32_t(__builtin_amdgcn_readlane(ix, 63))) return false;
        const uint32_t r = 63u - uint32_t(__builtin_clzll(__ballot(x > 0u && ix - x <= index)));
        within = index - uint32_t(__builtin_amdgcn_readlane(ix - x, r));
        parts = __builtin_amdgcn_readlane(s, r);
        n_tiles = __builtin_amdgcn_readlane(n, r);
        slot0 = __builtin_amdgcn_readlane(iy - y, r);
        tile0 = __builtin_amdgcn_readlane(in - n, r);
        w.req = r;
        w.q_start = __builtin_amdgcn_readlane(q.q_start, r);
        w.q_len = __builtin_amdgcn_readlane(q.q_len, r);
        w.kv_len = __builtin_amdgcn_readlane(q.kv_len, r);
    } else {
        // more requests than lanes: L from the sum of their key tiles
        const uint32_t wave = tid / kWave;
        uint64_t *sums = reinterpret_cast<uint64_t *>(scratch);
        uint64_t all = 0, tiles = 0;
        for (uint32_t r = tid; r < a.n_requests; r += kThreads) {
            uint32_t n, c;
            tiles_of(a, request(a, r, bad), n, c);
            all += uint64_t(n) * c;
            tiles += n;
        }
#pragma unroll
        for (int d = 32; d; d /= 2) {
            all += __shfl_xor(all, d);
            tiles += __shfl_xor(tiles, d);
        }
        if (lane == 0) sums[wave] = all, sums[kWaves + wave] = tiles;
        __syncthreads();
        all = (sums[0] + sums[1] + sums[2] + sums[3]) * a.kv_heads;
        const bool fits = sums[4] + sums[5] + sums[6] + sums[7] <= a.tile_cap;
        if (!fits) bad |= kStatusCorrupt;
        const uint64_t target = uint64_t(a.extra) * a.kv_heads;
        piece = a.extra ? uint32_t(min(uint64_t(1) << 30, max(uint64_t(a.min_piece), (all + target - 1u) / target)))
                        : 1u << 30;
        uint32_t px = 0, py = 0, pn = 0;  // before this chunk of requests
        uint32_t *found = scratch + 16, *part = scratch + 32;
        if (tid == 0) found[0] = 0;
        for (uint32_t r0 = 0; r0 < a.n_requests; r0 += kThreads) {
            Req q{0, 0, 0};
            uint32_t unused = 0, n, c;
            if (r0 + tid < a.n_requests) q = request(a, r0 + tid, unused);
            tiles_of(a, q, n, c);
            const uint32_t s = max(1u, ceil_of(c, piece)), x = n * s, y = s > 1u ? x : 0u;
            uint32_t ix = wave_inclusive_scan(x), iy = wave_inclusive_scan(y), in = wave_inclusive_scan(n);
            __syncthreads();  // part has been read
            if (lane == 63u) part[3u * wave] = ix, part[3u * wave + 1u] = iy, part[3u * wave + 2u] = in;
            __syncthreads();
            ix += px, iy += py, in += pn;
            for (uint32_t k = 0; k < kWaves; ++k) {
                const uint32_t tx = part[3u * k], ty = part[3u * k + 1u], tn = part[3u * k + 2u];
                if (k < wave) ix += tx, iy += ty, in += tn;
                px += tx, py += ty, pn += tn;
            }
            if (ix - x <= index && index < ix) {
                found[0] = 1;
                found[1] = r0 + tid, found[2] = uint32_t(q.q_start), found[3] = uint32_t(q.q_len);
                found[4] = uint32_t(q.kv_len), found[5] = index - (ix - x), found[6] = s, found[7] = n;
                found[8] = iy - y, found[9] = in - n;
            }
            if (!first && px > index) break;  // this chunk had it
        }
        __syncthreads();
        if (first && tid == 0) *a.tile_count = fits ? pn : 0u;
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
    int32_t lo, hi;
    tile_keys(a, Req{w.q_start, w.q_len, w.kv_len}, w.row0, lo, hi);
    const uint32_t c = key_tiles(a, lo, hi);
    w.splits = min(parts, max(1u, ceil_of(c, piece)));
    w.slot = slot0 + tile * parts;
    w.tile = tile0 + tile;
    // even shares of the key tiles
    w.lo = lo + int32_t(uint32_t(uint64_t(c) * w.split / w.splits) * a.key_tile);
    w.hi = min(hi, lo + int32_t(uint32_t(uint64_t(c) * (w.split + 1u) / w.splits) * a.key_tile));
    return w.split < w.splits;
}

// ------------------------------------------------------------- attention

template <typename E>
struct Type;
template <>
struct Type<__bf16> {
    using V8 = __attribute__((ext_vector_type(8))) __bf16;
    // probabilities up to 2^kSlack: bf16 has the range of fp32
    static constexpr float kSlack = 8.0f, kBias = 0.0f;
    static constexpr uint32_t kExp = 0x7f80u, kOne = 0x0080u;
    static __device__ __forceinline__ f32x16 mfma(V8 a, V8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Type<_Float16> {
    using V8 = __attribute__((ext_vector_type(8))) _Float16;
    // fp16 ends at 65504 and loses bits below 2^-14: probabilities are held
    // 2^8 above their value, so that the largest are in [2^8, 2^14] and a
    // weight keeps its bits down to 2^-22 of the largest
    static constexpr float kSlack = 6.0f, kBias = 8.0f;
    static constexpr uint32_t kExp = 0x7c00u, kOne = 0x0400u;
    static __device__ __forceinline__ f32x16 mfma(V8 a, V8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// 16-byte pieces of K and V rows in LDS are permuted within the row so that
// the reads below spread over the banks.  K: a read takes the same piece of
// 32 rows.  V: a transposing read takes 64 bytes of each of 4 rows.
template <int DP>
__device__ __forceinline__ uint32_t k_place(uint32_t row, uint32_t c) {
    return row * (DP / 8) + (c ^ (row & (DP >= 128 ? 15u : 7u)));
}
template <int DP>
__device__ __forceinline__ uint32_t v_place(uint32_t row, uint32_t c) {
    const uint32_t turn = DP >= 128 ? (row & 3u) : ((row ^ (row >> 1)) & 1u);
    return row * (DP / 8) + (c ^ (turn << 2));
}

__device__ __forceinline__ float other_half(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 32u) ? r[0] : r[1]);
}

template <typename E, int DP, int RW, int KT>
struct Shape {
    static constexpr int KW = kWaves / RW;             // groups along the keys
    static constexpr int kBuffers = RW == 1 ? 1 : 2;   // a wavefront alone needs no second one
    static constexpr uint32_t kTileBytes = KT * DP * 2;          // of K or of V
    static constexpr uint32_t kGroupBytes = 2 * kTileBytes * kBuffers;
    static constexpr uint32_t kOutBytes = 32 * DP * 4;           // a wavefront's rows in fp32
    static constexpr uint32_t kLoop = KW * kGroupBytes;
    static constexpr uint32_t kEnd = kWaves * kOutBytes;
    static constexpr uint32_t kMl = kLoop > kEnd ? kLoop : kEnd;  // offset of the joined maxima and sums
    static constexpr uint32_t kLds = kMl + kWaves * 32 * 8;
};

// The same sums for 32 rows of a wavefront, a row at a time and without
// matrix instructions, so that a key that a row does not see takes no part at
// all: for tiles in which such a key's value is not finite.  Lanes take keys
// for the scores and columns for the sums.  The wavefront's keys are the
// tiles of `kt` keys every `stride` from w.lo + first.
template <typename E, int DP>
__device__ __forceinline__ void rows_one_by_one(const AttnArgs &a, const Piece &w, uint32_t kvh, uint32_t row_base,
                                                uint32_t first, uint32_t stride, int kt, float *own, float *ml) {
    using V8 = __attribute__((ext_vector_type(8))) E;
    const uint32_t lane = threadIdx.x % kWave;
    const int32_t *table = a.table + int64_t(w.req) * a.table_stride;
    const E *kbase = static_cast<const E *>(a.k) + int64_t(kvh) * a.k_stride[2];
    const E *vbase = static_cast<const E *>(a.v) + int64_t(kvh) * a.v_stride[2];
    const int32_t page_mask = (1 << a.page_shift) - 1;
    constexpr int NO = DP / 64;
#pragma unroll 1
    for (uint32_t r = 0; r < 32u; ++r) {
        const int32_t row = int32_t(w.row0 + row_base + r);
        if (row >= w.q_len * int32_t(a.group)) break;
        const int32_t tok = row / int32_t(a.group), g = row - tok * int32_t(a.group);
        const int32_t pos = w.kv_len - w.q_len + tok;
        const int32_t see_hi = a.causal ? min(pos + 1, w.hi) : w.hi;
        const int32_t see_lo = a.window ? int32_t(max(int64_t(0), int64_t(pos) + 1 - int64_t(a.window))) : 0;
        const E *qp = static_cast<const E *>(a.q) + int64_t(w.q_start + tok) * a.q_stride[0] +
                      int64_t(kvh * a.group + uint32_t(g)) * a.q_stride[1];
        float m = -INFINITY, l = 0.0f, o[NO] = {};
#pragma unroll 1
        for (int32_t start = w.lo + int32_t(first); start < w.hi; start += int32_t(stride)) {
            const int32_t key = start + int32_t(lane);
            int32_t page = -1;
            if (int32_t(lane) < kt && key >= see_lo && key < see_hi) page = table[key >> a.page_shift];
            const bool seen = int32_t(lane) < kt && key >= see_lo && key < see_hi;
            if (uint32_t(page) >= a.n_pages) page = -1;  // counts as zeros
            const int64_t in_page = key & page_mask;
            float z = 0.0f;
            if (page >= 0) {
                const E *kp = kbase + page * a.k_stride[0] + in_page * a.k_stride[1];
                for (uint32_t d = 0; d < a.dim; d += 8u) {
                    const V8 x = *reinterpret_cast<const V8 *>(kp + d), y = *reinterpret_cast<const V8 *>(qp + d);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z = __builtin_fmaf(float(x[j]), float(y[j]), z);
                }
            }
            if (!seen) z = -INFINITY;
            float top = z;
#pragma unroll
            for (int d = 32; d; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
            const float m2 = fmaxf(m, top);
            const float f = m2 == m ? 1.0f : __builtin_amdgcn_exp2f((m - m2) * a.scale_log2);
            m = m2;
            const float off = Type<E>::kBias - (m == -INFINITY ? 0.0f : m * a.scale_log2);
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, a.scale_log2, off));
            float sum = e;
#pragma unroll
            for (int d = 32; d; d /= 2) sum += __shfl_xor(sum, d);
            l = l * f + sum;
#pragma unroll
            for (int j = 0; j < NO; ++j) o[j] *= f;
            const uint64_t seen_mask = __ballot(seen), page_in = __ballot(page >= 0);
#pragma unroll 1
            for (int k = 0; k < kt; ++k) {
                if (!((seen_mask & page_in) >> k & 1u)) continue;
                const float p = __shfl(e, k);
                const int32_t pg = __shfl(page, k);
                const E *vp = vbase + pg * a.v_stride[0] + int64_t((start + k) & page_mask) * a.v_stride[1];
#pragma unroll
                for (int j = 0; j < NO; ++j)
                    if (lane + 64u * uint32_t(j) < a.dim) o[j] += p * float(vp[lane + 64u * uint32_t(j)]);
            }
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const uint32_t d = lane + 64u * uint32_t(j);
            own[4u * (r * (DP / 4) + ((d / 4u) ^ (r & 7u))) + d % 4u] = o[j];
        }
        if (lane == 0) *reinterpret_cast<float2 *>(ml + 2u * r) = float2{m, l};
    }
}

template <typename E, int DP, int RW, int KT>
__global__ __launch_bounds__(kThreads, DP > 128 ? 1 : 2) void attention_kernel(AttnArgs a) {
    using T = Type<E>;
    using V8 = typename T::V8;
    using Sh = Shape<E, DP, RW, KT>;
    constexpr int KW = Sh::KW;
    constexpr int CPR = DP / 8;                       // 16-byte pieces per row
    constexpr int GT = 64 * RW;                       // threads that load a tile together
    constexpr int NL = KT * CPR / GT;                 // pieces of K (and of V) per thread
    constexpr int NB = KT / 32, NS = KT / 16, ND = DP / 32, NQ = DP / 16;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const uint32_t kvh = blockIdx.x % a.kv_heads, index = blockIdx.x / a.kv_heads;
    Piece w;
    if (!find_piece(a, index, blockIdx.x == 0, reinterpret_cast<uint32_t *>(lds), w)) return;
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t rw = wave % RW, kw = wave / RW;
    const uint32_t c = lane & 31u, h = lane >> 5;
    const int32_t n_rows = w.q_len * int32_t(a.group);
    const int32_t lo = w.lo, hi = w.hi;

    // this lane's row
    const int32_t row = int32_t(w.row0 + 32u * rw + c);
    const bool row_in = row < n_rows;
    const int32_t row_c = min(row, n_rows - 1);
    const int32_t tok = row_c / int32_t(a.group), g = row_c - tok * int32_t(a.group);
    const int32_t pos = w.kv_len - w.q_len + tok;
    const int32_t see_hi = a.causal ? min(pos + 1, hi) : hi;
    const int32_t see_lo = a.window ? int32_t(max(int64_t(0), int64_t(pos) + 1 - int64_t(a.window))) : 0;
    // over the wavefront's rows (positions ascend with the row)
    const int32_t hi_min = __builtin_amdgcn_readfirstlane(see_hi), lo_min = __builtin_amdgcn_readfirstlane(see_lo);
    const int32_t hi_max = __builtin_amdgcn_readlane(see_hi, 31), lo_max = __builtin_amdgcn_readlane(see_lo, 31);
    const bool idle = int32_t(w.row0 + 32u * rw) >= n_rows;

    V8 qf[NQ];
    {
        const E *qp = static_cast<const E *>(a.q) + int64_t(w.q_start + tok) * a.q_stride[0] +
                      int64_t(kvh * a.group + uint32_t(g)) * a.q_stride[1];
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
            V8 x = {};
            const uint32_t d = 16u * uint32_t(s) + 8u * h;
            if (row_in && d < a.dim) x = *reinterpret_cast<const V8 *>(qp + d);
            qf[s] = x;
        }
    }

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d] = f32x16{};
    float m = -INFINITY, l = 0.0f;  // reference (raw scores); this lane's share of the sum
    const float slack = fminf(T::kSlack / a.scale_log2, 1e30f);

    uint8_t *group = lds + kw * Sh::kGroupBytes;
    const uint32_t gtid = rw * 64u + lane;  // thread among those of the key group
    const int32_t *table = a.table + int64_t(w.req) * a.table_stride;
    const E *kbase = static_cast<const E *>(a.k) + int64_t(kvh) * a.k_stride[2];
    const E *vbase = static_cast<const E *>(a.v) + int64_t(kvh) * a.v_stride[2];
    const int32_t page_mask = (1 << a.page_shift) - 1;
    const int32_t n_tiles = (hi - lo + KT - 1) / KT;
    const int32_t n_steps = (n_tiles + KW - 1) / KW;  // the same for every group: they meet at barriers
    bool missing = false;
    uint32_t odd = 0;  // a tile with masked keys held a value that is not finite

    // The entry of the block table for key start + lane of a tile (-1 past the
    // piece), as it was read: it is looked at a step later.
    auto pages_of = [&](int32_t start) -> int32_t {
        const int32_t key = start + int32_t(lane % KT);
        return key < hi ? table[key >> a.page_shift] : -1;
    };
    // A load instruction of a wavefront covers kRpi rows, whole ones.  Where a
    // tile lies wholly inside the piece and such rows inside a page, their
    // address is one scalar and a constant per lane; other tiles find every
    // lane's row by itself and leave zeros where there is none.
    constexpr int kRpi = 64 / CPR;
    const bool in_dim = lane % CPR * 8u < a.dim;
    const uint32_t lane_off = uint32_t((int64_t(lane / CPR) * a.k_stride[1] + (in_dim ? lane % CPR * 8u : 0u)) * 2);
    uint4 kr[NL], vr[NL];
    auto load = [&](int32_t start, int32_t pages) {
        const bool none = uint32_t(pages) >= a.n_pages;
        if (a.simple_rows && start + KT <= hi && !__any(none)) {
#pragma unroll
            for (int n = 0; n < NL; ++n) {
                const uint32_t r0 = (rw + uint32_t(n) * RW) * kRpi;
                const uint32_t page = __builtin_amdgcn_readlane(pages, r0);
                const uint32_t in_page = (uint32_t(start) + r0) & uint32_t(page_mask);
                const uint64_t off = (uint64_t(page) * a.page_units + uint64_t(in_page) * a.slot_units) * 16u;
                kr[n] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(kbase) + off + lane_off);
                vr[n] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(vbase) + off + lane_off);
            }
            if (a.dim != DP) {
                // lanes past the head have read its first piece
                const uint32_t keep = in_dim ? ~0u : 0u;
#pragma unroll
                for (int n = 0; n < NL; ++n) {
                    kr[n].x &= keep, kr[n].y &= keep, kr[n].z &= keep, kr[n].w &= keep;
                    vr[n].x &= keep, vr[n].y &= keep, vr[n].z &= keep, vr[n].w &= keep;
                }
            }
            return;
        }
        if (none && start + int32_t(lane % KT) < hi) missing = true;
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const uint32_t i = gtid + uint32_t(n) * GT;
            const uint32_t r = i / CPR, ch = i % CPR;
            const int32_t page = __shfl(none ? -1 : pages, int(r));
            kr[n] = vr[n] = uint4{0, 0, 0, 0};
            if (page >= 0 && ch * 8u < a.dim) {
                const int64_t in_page = (start + int32_t(r)) & page_mask;
                kr[n] = *reinterpret_cast<const uint4 *>(kbase + page * a.k_stride[0] + in_page * a.k_stride[1] + ch * 8u);
                vr[n] = *reinterpret_cast<const uint4 *>(vbase + page * a.v_stride[0] + in_page * a.v_stride[1] + ch * 8u);
            }
        }
    };
    auto tile_start = [&](int32_t step) { return lo + (step * KW + int32_t(kw)) * KT; };

    int32_t pages = pages_of(tile_start(0));
    load(tile_start(0), pages);
    pages = pages_of(tile_start(1));

    // Where this lane reads its operands in a tile's K and V.  A later piece of
    // a K row is an exclusive or away, later rows an immediate offset.
    const uint32_t k_at = k_place<DP>(c, h) * 16u;
    uint32_t v_at[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const uint32_t i16 = lane % 16u;
        v_at[d] = Sh::kTileBytes + 8u * (i16 & 1u) +
                  16u * v_place<DP>(4u * h + i16 / 4u, 4u * uint32_t(d) + 2u * ((lane >> 4) & 1u) + (i16 % 4u) / 2u);
    }

    for (int32_t step = 0; step < n_steps; ++step) {
        const int32_t start = tile_start(step);
        uint8_t *buf = group + (Sh::kBuffers == 2 ? uint32_t(step & 1) : 0u) * 2u * Sh::kTileBytes;
        uint4 *kl = reinterpret_cast<uint4 *>(buf);
        uint4 *vl = reinterpret_cast<uint4 *>(buf + Sh::kTileBytes);
        if constexpr (RW == 1) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const uint32_t i = gtid + uint32_t(n) * GT;
            kl[k_place<DP>(i / CPR, i % CPR)] = kr[n];
            vl[v_place<DP>(i / CPR, i % CPR)] = vr[n];
        }
        // one barrier a step: a buffer is written again two steps later, when
        // every wavefront has passed the next step's barrier
        if constexpr (RW == 1)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        else
            __syncthreads();
        if (step + 1 < n_steps) {
            load(tile_start(step + 1), pages);
            pages = pages_of(tile_start(step + 2));
        }
        if (idle || start >= hi_max || start + KT <= lo_min) continue;

        // S^T = K Q^T.  Operands are read a group of four ahead of the
        // products that use them; left to itself the compiler reads each one
        // just before its product and waits for it.
        f32x16 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) s[b] = f32x16{};
        {
            constexpr int KG = 4 / NB;       // 16-column steps per group
            constexpr int NG = NQ / KG;
            V8 kf[2][KG][NB];
            auto read = [&](int g) {
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        kf[g & 1][k][b] = *reinterpret_cast<const V8 *>(
                            buf + (k_at ^ (uint32_t(g * KG + k) << 5)) + b * 32 * DP * 2);
            };
            read(0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g + 1 < NG) read(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int b = 0; b < NB; ++b) s[b] = T::mfma(kf[g & 1][k][b], qf[g * KG + k], s[b]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        const bool masked = start + KT > hi_min || start < lo_max;
        if (masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int32_t key = start + 32 * b + 8 * (r / 4) + 4 * int32_t(h) + r % 4;
                    if (key >= see_hi || key < see_lo) s[b][r] = -INFINITY;
                }
        }
        // the running reference
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
        top = fmaxf(top, other_half(top));
        if (__any(top > m + slack)) {
            const float m2 = fmaxf(m, top);
            const float f = m2 == m ? 1.0f : __builtin_amdgcn_exp2f((m - m2) * a.scale_log2);
            m = m2;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[d] *= f;
        }
        const float off = T::kBias - (m == -INFINITY ? 0.0f : m * a.scale_log2);
        V8 p[NS];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r], a.scale_log2, off));
                l += e;
                p[2 * b + r / 8][r % 8] = E(e);
            }

        // O^T += V^T P^T
        auto v_frag = [&](int st, int d) -> V8 {
            using L4 = __attribute__((address_space(3))) s16x4;
            struct Two {
                s16x4 a, b;
            } t;
            const uint8_t *at = buf + v_at[d] + st * 16 * DP * 2;
            t.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)at);
            t.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)(at + 8 * DP * 2));
            return __builtin_bit_cast(V8, t);
        };
        if (masked) {
            // a masked key adds nothing, whatever its value holds, but 0 x inf
            // in the product below is not nothing: note it, and see the end
            constexpr uint32_t kE = T::kExp * 0x10001u, kO = T::kOne * 0x10001u;
            uint32_t bits = 0;
#pragma unroll 2
            for (uint32_t i = lane; i < uint32_t(KT * CPR); i += 64u) {
                const uint4 x = vl[i];
                bits |= ((x.x & kE) + kO) | ((x.y & kE) + kO) | ((x.z & kE) + kO) | ((x.w & kE) + kO);
            }
            odd |= bits & 0x80008000u;
        }
        {
            // groups of up to four operands, as above
            constexpr int VG = ND < 4 ? ND : 4;
            constexpr int NG = NS * ND / VG;
            V8 vf[2][VG];
            auto read = [&](int g) {
#pragma unroll
                for (int j = 0; j < VG; ++j) vf[g & 1][j] = v_frag((g * VG + j) / ND, (g * VG + j) % ND);
            };
            read(0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g + 1 < NG) read(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < VG; ++j) {
                    const int d = (g * VG + j) % ND;
                    acc[d] = T::mfma(vf[g & 1][j], p[(g * VG + j) / ND], acc[d]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (missing && a.status) atomicOr(a.status, kStatusCorrupt);

    // Join the key groups and write.  A wavefront's rows go to LDS; the
    // wavefronts of a row group then each take a share of its rows, so that
    // stores run along the rows.
    l += other_half(l);
    float *ml = reinterpret_cast<float *>(lds + Sh::kMl) + 64u * wave;
    auto place = [&](uint32_t r, uint32_t q4) { return r * (DP / 4) + (q4 ^ (r & 7u)); };
    float4 *own = reinterpret_cast<float4 *>(lds + wave * Sh::kOutBytes);
    __syncthreads();
    if (!__any(odd != 0)) {
        if (h == 0) *reinterpret_cast<float2 *>(ml + 2u * c) = float2{m, l};
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
                own[place(c, 8u * uint32_t(d) + 2u * uint32_t(q4) + h)] =
                    float4{acc[d][4 * q4], acc[d][4 * q4 + 1], acc[d][4 * q4 + 2], acc[d][4 * q4 + 3]};
    } else {
        rows_one_by_one<E, DP>(a, w, kvh, 32u * rw, kw * KT, uint32_t(KW * KT), KT, reinterpret_cast<float *>(own), ml);
    }
    __syncthreads();
    auto weight = [&](float mk, float top) {
        return mk == top ? 1.0f : __builtin_amdgcn_exp2f((mk - top) * a.scale_log2);
    };
    ml = reinterpret_cast<float *>(lds + Sh::kMl);
    const bool whole = w.splits == 1;
    const uint64_t slot = (uint64_t(w.slot + w.split) * a.kv_heads + kvh) * a.rows_per_tile;
    if (a.tiles && kvh == 0 && w.split == 0 && threadIdx.x == 0) {
        Tile t;
        t.splits = w.splits;
        t.slot = w.slot;
        t.token0 = w.q_start;
        t.row0 = w.row0;
        t.rows = uint32_t(min(int32_t(a.rows_per_tile), n_rows - int32_t(w.row0)));
        a.tiles[w.tile] = t;
    }
#pragma unroll 2
    for (uint32_t i = lane; i < 32u / KW * CPR; i += 64u) {
        const uint32_t r = kw * (32u / KW) + i / CPR, ch = i % CPR;
        const int32_t at = int32_t(w.row0 + 32u * rw + r);
        if (at >= n_rows || ch * 8u >= a.dim) continue;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KW; ++k) top = fmaxf(top, ml[2u * (32u * (uint32_t(k) * RW + rw) + r)]);
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const uint32_t src = uint32_t(k) * RW + rw;
            const float2 v = *reinterpret_cast<const float2 *>(ml + 2u * (32u * src + r));
            const float f = KW == 1 ? 1.0f : weight(v.x, top);
            sum += v.y * f;
            const float4 *o = reinterpret_cast<const float4 *>(lds + src * Sh::kOutBytes);
            const float4 x0 = o[place(r, 2u * ch)], x1 = o[place(r, 2u * ch + 1u)];
            x[0] += x0.x * f, x[1] += x0.y * f, x[2] += x0.z * f, x[3] += x0.w * f;
            x[4] += x1.x * f, x[5] += x1.y * f, x[6] += x1.z * f, x[7] += x1.w * f;
        }
        if (whole) {
            const int32_t t = at / int32_t(a.group), hg = at - t * int32_t(a.group);
            const uint32_t head = kvh * a.group + uint32_t(hg);
            const int64_t token = w.q_start + t;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key gives 0
            V8 y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = E(x[j] * inv);
            *reinterpret_cast<V8 *>(static_cast<E *>(a.out) + token * a.out_stride[0] + int64_t(head) * a.out_stride[1] +
                                    ch * 8u) = y;
            if (a.lse && ch == 0)
                a.lse[token * a.heads + head] =
                    sum == 0.0f ? -INFINITY : top * a.scale + (__builtin_amdgcn_logf(sum) - T::kBias) * 0.69314718f;
        } else {
            const uint64_t pr = slot + (uint32_t(at) - w.row0);
            float4 *o = reinterpret_cast<float4 *>(a.part_o + pr * DP + ch * 8u);
            o[0] = float4{x[0], x[1], x[2], x[3]};
            o[1] = float4{x[4], x[5], x[6], x[7]};
            if (ch == 0) *reinterpret_cast<float2 *>(a.part_ml + 2u * pr) = float2{top, sum};
        }
    }
}

// The pieces of a split tile joined.  A wavefront takes a row (WPR = 1, for
// tiles of many rows and few pieces) or a quarter of its pieces (WPR = 4);
// lanes run along the row in 16-byte steps and, where the row is shorter,
// over several pieces.  Each lane keeps its own running maximum.
template <typename E, int DP, int WPR>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a) {
    using T = Type<E>;
    constexpr uint32_t CPR = DP / 4;                     // float4 pieces per row
    constexpr uint32_t SL = 64 / CPR;                    // lanes side by side on one column
    constexpr uint32_t kRows = kWaves / WPR;             // rows at a time
    __shared__ float4 part_x[WPR == 4 ? 4 : 1][CPR];
    __shared__ float2 part_ml[4];
    const uint32_t kvh = blockIdx.x % a.kv_heads, index = blockIdx.x / a.kv_heads;
    if (index >= *a.tile_count) return;
    const Tile w = a.tiles[index];
    const uint32_t splits = __builtin_amdgcn_readfirstlane(w.splits), slot = __builtin_amdgcn_readfirstlane(w.slot);
    const uint32_t row0 = __builtin_amdgcn_readfirstlane(w.row0), rows = __builtin_amdgcn_readfirstlane(w.rows);
    const int32_t token0 = __builtin_amdgcn_readfirstlane(w.token0);
    if (splits == 1u) return;
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t ch = lane % CPR, sl = lane / CPR;
    auto weight = [&](float m, float top) { return m == top ? 1.0f : __builtin_amdgcn_exp2f((m - top) * a.scale_log2); };
    for (uint32_t r = blockIdx.y * kRows + (WPR == 4 ? 0u : wave); r < rows; r += gridDim.y * kRows) {
        float top = -INFINITY, sum = 0.0f;
        float4 x{0, 0, 0, 0};
        auto add = [&](float m, float l, const float4 &o) {
            const float t2 = fmaxf(top, m), f = weight(top, t2), g = weight(m, t2);
            top = t2;
            sum = sum * f + l * g;
            x.x = x.x * f + o.x * g, x.y = x.y * f + o.y * g, x.z = x.z * f + o.z * g, x.w = x.w * f + o.w * g;
        };
#pragma unroll 4
        for (uint32_t s = (WPR == 4 ? wave * SL : 0u) + sl; s < splits; s += SL * WPR) {
            const uint64_t pr = (uint64_t(slot + s) * a.kv_heads + kvh) * a.rows_per_tile + r;
            const float2 v = *reinterpret_cast<const float2 *>(a.part_ml + 2u * pr);
            add(v.x, v.y, *reinterpret_cast<const float4 *>(a.part_o + pr * DP + 4u * ch));
        }
#pragma unroll
        for (uint32_t d = CPR; d < 64u; d *= 2) {
            const float m = __shfl_xor(top, int(d)), l = __shfl_xor(sum, int(d));
            add(m, l, float4{__shfl_xor(x.x, int(d)), __shfl_xor(x.y, int(d)), __shfl_xor(x.z, int(d)),
                             __shfl_xor(x.w, int(d))});
        }
        if constexpr (WPR == 4) {
            __syncthreads();  // the row before has been read
            if (sl == 0) part_x[wave][ch] = x;
            if (lane == 0) part_ml[wave] = float2{top, sum};
            __syncthreads();
            if (wave == 0 && sl == 0) {
#pragma unroll
                for (int k = 1; k < 4; ++k) add(part_ml[k].x, part_ml[k].y, part_x[k][ch]);
            }
            if (wave != 0) continue;
        }
        if (sl != 0 || ch * 4u >= a.dim) continue;
        const uint32_t gr = row0 + r;
        const uint32_t t = gr / a.group, head = kvh * a.group + gr % a.group;
        const int64_t token = int64_t(token0) + t;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        using E4 = __attribute__((ext_vector_type(4))) E;
        const E4 y = {E(x.x * inv), E(x.y * inv), E(x.z * inv), E(x.w * inv)};
        *reinterpret_cast<E4 *>(static_cast<E *>(a.out) + token * a.out_stride[0] + int64_t(head) * a.out_stride[1] +
                                4u * ch) = y;
        if (a.lse && ch == 0)
            a.lse[token * a.heads + head] =
                sum == 0.0f ? -INFINITY : top * a.scale + (__builtin_amdgcn_logf(sum) - T::kBias) * 0.69314718f;
    }
}

// ------------------------------------------------------------------ launch

// The launch's shape, from what the host knows: sizes only.
struct LaunchPlan {
    int rw, kt, dp;
    uint32_t rows_per_tile, min_piece, resident, extra, tile_cap, slot_cap, most_rows;
    float piece_cost, join_cost;
    uint64_t off_tiles, off_ml, off_o, bytes;
};

LaunchPlan launch_plan(const dfc_attention_args &a) {
    LaunchPlan p;
    const uint32_t group = a.heads / a.cache.kv_heads;
    p.dp = a.cache.head_dim <= 64 ? 64 : a.cache.head_dim <= 128 ? 128 : 256;
    // most rows a request has per cache head
    const uint64_t most = std::min<uint64_t>(a.max_q_len ? a.max_q_len : a.tokens, a.tokens) * group;
    // one wavefront holds a whole key tile of K and V on its way to LDS: too
    // many registers at 256 columns
    p.rw = most <= 32 && p.dp <= 128 ? 1 : most <= 64 ? 2 : 4;
    p.kt = p.rw == 4 && p.dp <= 128 ? 64 : 32;
    p.rows_per_tile = 32u * uint32_t(p.rw);
    p.resident = p.dp > 128 ? 256u : 512u;
    p.min_piece = p.rw == 4 ? 2u : kWaves / uint32_t(p.rw);
    p.piece_cost = p.rw == 4 ? 1.0f : 4.0f;
    p.join_cost = p.rw == 4 ? 2.0f : 8.0f;
    const uint64_t tiles = std::min<uint64_t>(dfc::ceil_div(a.tokens * group, uint64_t(p.rows_per_tile)) + a.n_requests,
                                              uint64_t(a.tokens) * group);
    // a tile of c key tiles has at most ceil(c / min_piece) pieces; there are
    // up to four rounds of pieces beyond one a tile
    const uint64_t longest = dfc::ceil_div(uint64_t(a.max_pages) * a.cache.page_size, uint64_t(p.kt)) + 1u;
    const uint64_t each = longest > p.min_piece ? dfc::ceil_div(longest, uint64_t(p.min_piece)) - 1u : 0u;
    const uint64_t extra = std::min<uint64_t>(4u * p.resident / a.cache.kv_heads + 1u, tiles * each);
    p.extra = uint32_t(extra);
    p.tile_cap = uint32_t(tiles);
    // a tile's pieces are at most twice those beyond its first
    p.slot_cap = uint32_t(std::min<uint64_t>(2u * extra, tiles + extra));
    p.most_rows = uint32_t(std::min<uint64_t>(most, p.rows_per_tile));
    p.off_tiles = 256;
    p.off_ml = p.off_tiles + uint64_t(p.tile_cap) * sizeof(Tile);
    const uint64_t rows = uint64_t(p.slot_cap) * a.cache.kv_heads * p.rows_per_tile;
    p.off_o = (p.off_ml + rows * 8u + 255u) & ~uint64_t(255);
    p.bytes = p.off_o + rows * uint64_t(p.dp) * 4u;
    return p;
}

dfc_status check_attention(const dfc_attention_args &a) {
    const dfc_status cs = dfc::check_cache(a.cache);
    if (cs != DFC_OK) return cs;
    if (!a.heads || a.heads % a.cache.kv_heads || a.heads > 65536u) return DFC_EINVAL;
    if (a.tokens > 0x7fffffffull || a.n_requests > 0x7fffffffu) return DFC_EINVAL;
    // rows (tokens x heads of a group), and the tiles of 64 requests, are
    // counted in 32 bits
    if (a.tokens * (a.heads / a.cache.kv_heads) > 0x3fffffffull) return DFC_EUNSUPPORTED;
    if (!(a.scale > 0.0f) || !std::isfinite(a.scale)) return DFC_EINVAL;
    if (a.window > 0x7fffffffu) return DFC_EINVAL;
    return DFC_OK;
}

template <typename E, int DP, int RW, int KT>
dfc_status launch(const AttnArgs &a, const LaunchPlan &p, hipStream_t st) {
    using Sh = Shape<E, DP, RW, KT>;
    const void *fn = reinterpret_cast<const void *>(&attention_kernel<E, DP, RW, KT>);
    if (!allow_full_lds(fn)) return DFC_EHIP;
    const uint64_t grid = (uint64_t(p.tile_cap) + p.extra) * a.kv_heads;
    if (grid > 0x7fffffffull) return DFC_EUNSUPPORTED;
    hipLaunchKernelGGL((attention_kernel<E, DP, RW, KT>), dim3(uint32_t(grid)), dim3(kThreads), Sh::kLds, st, a);
    if (a.tiles) {
        constexpr int WPR = RW == 4 ? 1 : 4;
        hipLaunchKernelGGL((join_kernel<E, DP, WPR>),
                           dim3(p.tile_cap * a.kv_heads, WPR == 4 ? p.most_rows : (p.most_rows + 7u) / 8u),
                           dim3(kThreads), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP;
}

template <typename E>
dfc_status launch_type(const AttnArgs &a, const LaunchPlan &p, hipStream_t st) {
    switch (p.dp * 8 + p.rw) {
        case 64 * 8 + 1: return launch<E, 64, 1, 32>(a, p, st);
        case 64 * 8 + 2: return launch<E, 64, 2, 32>(a, p, st);
        case 64 * 8 + 4: return launch<E, 64, 4, 64>(a, p, st);
        case 128 * 8 + 1: return launch<E, 128, 1, 32>(a, p, st);
        case 128 * 8 + 2: return launch<E, 128, 2, 32>(a, p, st);
        case 128 * 8 + 4: return launch<E, 128, 4, 64>(a, p, st);
        case 256 * 8 + 2: return launch<E, 256, 2, 32>(a, p, st);
        default: return launch<E, 256, 4, 32>(a, p, st);
    }
}

}  // namespace

extern "C" {

dfc_status dfc_paged_attention_workspace(const dfc_attention_args *args, uint64_t *bytes) {
    if (!args || !bytes) return DFC_EINVAL;
    const dfc_status s = check_attention(*args);
    if (s != DFC_OK) return s;
    *bytes = args->tokens && args->n_requests ? launch_plan(*args).bytes : 0;
    return DFC_OK;
}

dfc_status dfc_paged_attention(const dfc_attention_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_attention_args &in = *args;
    const dfc_status s = check_attention(in);
    if (s != DFC_OK) return s;
    if (!in.tokens || !in.n_requests) return DFC_OK;
    if (!in.q_dev || !in.out_dev || !in.cu_q || !in.seq_lens || !in.workspace_dev) return DFC_EINVAL;
    if (in.max_pages && !in.block_table) return DFC_EINVAL;
    if (in.table_stride < int64_t(in.max_pages)) return DFC_EINVAL;
    if ((reinterpret_cast<uintptr_t>(in.q_dev) | reinterpret_cast<uintptr_t>(in.out_dev)) & 15u) return DFC_EINVAL;
    if (reinterpret_cast<uintptr_t>(in.workspace_dev) & 255u) return DFC_EINVAL;
    for (int i = 0; i < 2; ++i)
        if (in.q_stride[i] % 8 || in.out_stride[i] % 8) return DFC_EINVAL;
    const LaunchPlan p = launch_plan(in);
    if (in.workspace_bytes < p.bytes) return DFC_ESIZE;
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = in.q_dev;
    a.k = in.cache.k_dev;
    a.v = in.cache.v_dev;
    a.out = in.out_dev;
    a.lse = in.lse_dev;
    a.table = in.block_table;
    a.cu_q = in.cu_q;
    a.seq_lens = in.seq_lens;
    for (int i = 0; i < 2; ++i) {
        a.q_stride[i] = in.q_stride[i];
        a.out_stride[i] = in.out_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        a.k_stride[i] = in.cache.k_stride[i];
        a.v_stride[i] = in.cache.v_stride[i];
    }
    bool simple = in.cache.page_size >= 512u / uint32_t(p.dp);
    for (int i = 0; i < 3; ++i) simple = simple && a.k_stride[i] == a.v_stride[i] && a.k_stride[i] / 8 < (int64_t(1) << 31);
    // a lane's offset within its instruction's rows is 32 bits
    simple = simple && a.k_stride[1] < (int64_t(1) << 27);
    a.simple_rows = simple ? 1 : 0;
    a.page_units = simple ? uint32_t(a.k_stride[0] / 8) : 0u;
    a.slot_units = simple ? uint32_t(a.k_stride[1] / 8) : 0u;
    a.table_stride = in.table_stride;
    a.n_pages = in.cache.n_pages;
    a.page_shift = dfc::log2_of(in.cache.page_size);
    a.kv_heads = in.cache.kv_heads;
    a.heads = in.heads;
    a.group = in.heads / in.cache.kv_heads;
    a.dim = in.cache.head_dim;
    a.n_requests = in.n_requests;
    a.tokens = uint32_t(in.tokens);
    a.max_pages = in.max_pages;
    a.window = in.window;
    a.causal = in.causal ? 1 : 0;
    a.scale = in.scale;
    a.scale_log2 = in.scale * 1.44269504088896340736f;
    a.rows_per_tile = p.rows_per_tile;
    a.key_tile = uint32_t(p.kt);
    a.min_piece = p.min_piece;
    a.resident = p.resident;
    a.piece_cost = p.piece_cost;
    a.join_cost = p.join_cost;
    a.extra = p.extra;
    a.tile_cap = p.tile_cap;
    uint8_t *ws = static_cast<uint8_t *>(in.workspace_dev);
    a.tile_count = reinterpret_cast<uint32_t *>(ws);
    a.tiles = p.extra ? reinterpret_cast<Tile *>(ws + p.off_tiles) : nullptr;
    a.part_ml = reinterpret_cast<float *>(ws + p.off_ml);
    a.part_o = reinterpret_cast<float *>(ws + p.off_o);
    a.status = in.status_dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return in.cache.dtype == DFC_BF16 ? launch_type<__bf16>(a, p, st) : launch_type<_Float16>(a, p, st);
}

}  // extern "C"
