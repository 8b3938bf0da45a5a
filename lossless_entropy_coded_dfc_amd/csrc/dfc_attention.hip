// dfc_attention.hip - attention of a step's new tokens over the paged cache.
//
// Token i of request r (n_r new tokens, s_r tokens in all) stands at position
// p = s_r - n_r + i and sees the keys j < s_r with j <= p (causal) and
// j > p - window or j < sinks.  For each of its heads, which share the keys and values of
// one cache head in groups of G = heads / kv_heads,
//     o = sum_j exp(z_j - m) v_j / sum_j exp(z_j - m),  z_j = scale q . k_j,
// in one pass over the keys: m is a running reference no smaller than the
// running maximum less a slack, and the sums are rescaled when it moves.
//
// Rows.  The n_r G (token, head of the group) pairs of a request and cache
// head are its rows; a tile is 32 RW of them, 32 per wavefront.  A workgroup
// takes one tile and one piece of its keys.  Of four wavefronts (RW = 1, 2,
// 4), RW lie along the rows times 4 / RW groups along the keys, whose results
// the workgroup joins at the end; of eight (RW = 8) all lie along the rows.
// Pieces of one tile are joined by a second kernel.
//
// Layout.  Scores are computed transposed, S^T = K Q^T, with 32x32x16
// MFMA: lane l then holds, for the row l mod 32, the keys 8 (r / 4) +
// 4 (l / 32) + r mod 4 of each block of 32 (r = 0..15), so a row's maximum
// and sum are in-lane sums and one exchange with lane l ^ 32, and the
// rounded probabilities are, as they stand, the B operand of O^T = V^T P^T
// (the order of the keys within a step of 16 is free as long as V^T follows
// it: the transposing LDS read gives each lane those four keys at its
// column).  LDS reads of both products are free of bank conflicts.
//
// Bounds (one MI355X, 32 heads over 8 cache heads of 128, bfloat16, time a call
// among others; a device copy reaches 5.1 TB/s and a product of 16384-square
// matrices 1.35 PFLOP/s).  One token a request: the bytes of K and V (64
// requests of 1 to 8191: 212-217 us, 5.0-5.2 TB/s; 131072 keys in float16 106
// us, 5.0 TB/s), for a short one latencies: launches, lengths, page, keys (700
// keys 11.4 us).  Prompts: the two products (8192 tokens 550-600 us from card to
// card, 0.92-1.0 PFLOP/s; 512 tokens, a workgroup or two on each compute unit,
// 15-17 us).  With a window and sinks the keys of the sinks' last tile and of the
// window's first count whole: 64 requests of up to 8191 tokens under 1000 + 4
// 57 us (4.4 TB/s of what they see), 513 tokens over 32000 under 4096 + 64 in
// float16 70; with heads of 64, 80 and 256 33, 49 and 142 us (floors 25, 31 and 99)
// and 48, 70 and 188 (13, 17 and 54).  Tiles wholly inside long sinks take the masked
// path: 4096 + 1024 and 4096 + 4096 over 32000 98 and 152 us (33 and 53).  Other
// heads have only been looked at: 64 ragged requests with
// heads of 64, 80 and 256 take 130, 180 and 602 us (floors 107, 134 and 428),
// prompts of 8192 349, 529 and 1864 (204, 255 and 815).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "dfc.h"
#include "dfc_attention_schedule.h"
#include "dfc_decode_core.h"
#include "dfc_format.h"
#include "dfc_paged.h"

namespace {

using f32x16 = __attribute__((ext_vector_type(16))) float;
using s16x4 = __attribute__((ext_vector_type(4))) short;

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

// The same sums for 32 rows of a wavefront, a row at a time and without
// matrix instructions, so that a key that a row does not see takes no part at
// all: for tiles in which such a key's value is not finite.  Lanes take keys
// for the scores and columns for the sums.  The wavefront's keys are the
// tiles of `kt` keys every `stride` from w.lo + first.  One after the other
// these take long: one infinite value at token 1000 of a prompt of 2048 makes
// 10 ms of 0.08, at token 4000 of 8192 42 ms of 0.6 (bfloat16, heads of 128),
// before a window of 100,000 keys of a single token 0.75 ms of 0.11.
template <typename E, int DP, bool Sinks>
__device__ __forceinline__ void rows_one_by_one(const AttnArgs &a, const Piece &w, uint32_t kvh, uint32_t row_base,
                                                uint32_t first, uint32_t stride, int kt, float *own, float *ml) {
    using V8 = __attribute__((ext_vector_type(8))) E;
    const uint32_t lane = threadIdx.x % kWave;
    const int32_t *table = a.table + int64_t(w.req) * a.table_stride;
    const E *kbase = static_cast<const E *>(a.k) + uint64_t(kvh) * a.k_units[2] * 8u;
    const E *vbase = static_cast<const E *>(a.v) + uint64_t(kvh) * a.v_units[2] * 8u;
    const int32_t page_mask = (1 << a.page_shift) - 1;
    constexpr int NO = DP / 64;
#pragma unroll 1
    for (uint32_t r = 0; r < 32u; ++r) {
        const int32_t row = int32_t(w.row0 + row_base + r);
        if (row >= w.q_len * int32_t(a.group)) break;
        const int32_t tok = row / int32_t(a.group), g = row - tok * int32_t(a.group);
        const int32_t pos = w.kv_len - w.q_len + tok;
        const int32_t end = end_of<Sinks>(a, w), see_hi = a.causal ? min(pos + 1, end) : end;
        const int32_t see_lo = a.window ? int32_t(max(int64_t(0), int64_t(pos) + 1 - int64_t(a.window))) : 0;
        const E *qp = static_cast<const E *>(a.q) + int64_t(w.q_start + tok) * a.q_stride[0] +
                      int64_t(kvh * a.group + uint32_t(g)) * a.q_stride[1];
        float m = -INFINITY, l = 0.0f, o[NO] = {};
#pragma unroll 1
        for (int32_t at = w.lo + int32_t(first); at < w.hi; at += int32_t(stride)) {
            const int32_t start = key_at<Sinks>(a, w, at), key = start + int32_t(lane);
            const bool behind = key < see_lo && !(Sinks && key < a.sinks);
            int32_t page = -1;
            if (int32_t(lane) < kt && !behind && key < see_hi) page = table[key >> a.page_shift];
            const bool seen = int32_t(lane) < kt && !behind && key < see_hi;
            if (uint32_t(page) >= a.n_pages) page = -1;  // counts as zeros
            const uint32_t in_page = uint32_t(key & page_mask);
            float z = 0.0f;
            if (page >= 0) {
                const E *kp = kbase + (uint64_t(uint32_t(page)) * a.k_units[0] + uint64_t(in_page) * a.k_units[1]) * 8u;
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
                const E *vp = vbase + (uint64_t(uint32_t(pg)) * a.v_units[0] +
                                       uint64_t(uint32_t((start + k) & page_mask)) * a.v_units[1]) * 8u;
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

// The kernel's arguments, read again from here on: what only the end needs
// would otherwise sit in scalar registers through the loop, which has none to
// spare.
__device__ __forceinline__ const AttnArgs &again(const AttnArgs &a) {
#ifdef __HIP_DEVICE_COMPILE__
    uint64_t p = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    return *reinterpret_cast<const __attribute__((address_space(4))) AttnArgs *>(p);
#else
    return a;
#endif
}

constexpr auto nothing = [](int) {};  // no work beside the products

// A wavefront's 32 rows: their queries, limits and running sums.  Lane l has
// row l mod 32 (half l / 32 of its keys and columns).
template <typename E, int DP, int KT, bool Sinks>
struct Rows {
    using T = Type<E>;
    using V8 = typename T::V8;
    static constexpr int NB = KT / 32, NS = KT / 16, ND = DP / 32, NQ = DP / 16;

    V8 qf[NQ];
    f32x16 acc[ND];
    float m, l, slack;              // reference (raw scores); this lane's share of the sum
    int32_t see_lo, see_hi;         // the keys of the row,
    int32_t see_sinks;              // and the first so many
    int32_t hi_min, hi_max, lo_min, lo_max;  // over the wavefront's rows
    bool idle;                      // no rows
    uint32_t odd;                   // a tile with masked keys held a value that is not finite
    uint32_t k_at, v_at[ND];        // where the lane reads its operands in a tile of K and of V

    __device__ __forceinline__ void init(const AttnArgs &a, const Piece &w, uint32_t kvh, uint32_t row_base) {
        const uint32_t lane = threadIdx.x % kWave, c = lane & 31u, h = lane >> 5;
        const int32_t n_rows = w.q_len * int32_t(a.group);
        const int32_t row = int32_t(w.row0 + row_base + c);
        const int32_t row_c = min(row, n_rows - 1);
        const int32_t tok = row_c / int32_t(a.group), g = row_c - tok * int32_t(a.group);
        const int32_t pos = w.kv_len - w.q_len + tok;
        // (as the piece counts its keys: no row sees one of the gap)
        const int32_t gap = Sinks ? w.gap : 0;
        see_hi = a.causal ? min(pos + 1 - gap, w.hi) : w.hi;
        if constexpr (Sinks) see_sinks = max(min(a.sinks, see_hi), 0);
        see_lo = (a.window ? int32_t(max(int64_t(0), int64_t(pos) + 1 - int64_t(a.window))) : 0) - gap;
        // positions ascend with the row
        hi_min = __builtin_amdgcn_readfirstlane(see_hi), lo_min = __builtin_amdgcn_readfirstlane(see_lo);
        hi_max = __builtin_amdgcn_readlane(see_hi, 31), lo_max = __builtin_amdgcn_readlane(see_lo, 31);
        idle = int32_t(w.row0 + row_base) >= n_rows;
        const E *qp = static_cast<const E *>(a.q) + int64_t(w.q_start + tok) * a.q_stride[0] +
                      int64_t(kvh * a.group + uint32_t(g)) * a.q_stride[1];
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
            V8 x = {};
            const uint32_t d = 16u * uint32_t(s) + 8u * h;
            if (row < n_rows && d < a.dim) x = *reinterpret_cast<const V8 *>(qp + d);
            qf[s] = x;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = f32x16{};
        m = -INFINITY;
        l = 0.0f;
        slack = fminf(T::kSlack / a.scale_log2, 1e30f);
        odd = 0;
        // a later piece of a K row is an exclusive or away, later rows of K
        // and of V an immediate offset
        const uint32_t i16 = lane % 16u;
        k_at = k_place<DP>(c, h) * 16u;
#pragma unroll
        for (int d = 0; d < ND; ++d)
            v_at[d] = 8u * (i16 & 1u) + 16u * v_place<DP>(4u * h + i16 / 4u, 4u * uint32_t(d) + 2u * ((lane >> 4) & 1u) +
                                                                                 (i16 % 4u) / 2u);
    }

    // The queries are there from here on: a wait for them inside the loop would
    // wait for the tiles under way.
    __device__ __forceinline__ void settle() const {
#pragma unroll
        for (int s = 0; s < NQ; ++s) asm volatile("" ::"v"(qf[s]));
    }

    // No row sees a key of the tile; some row does not see all of them.  With
    // sinks, a tile before the wavefront's windows counts as one that some row
    // sees in part: those are the sinks' own and what the tile's other rows see.
    __device__ __forceinline__ bool skips(int32_t start) const {
        return idle || start >= hi_max || (!Sinks && start + KT <= lo_min);
    }
    __device__ __forceinline__ bool masks(int32_t start) const { return start + KT > hi_min || start < lo_max; }

    // O^T += V^T P^T (PV), S^T = K Q^T (QK), in groups of four products whose
    // operands are read kAhead groups before they are used: four wavefronts
    // that read at once wait longer for LDS than one group of products takes.
    // Left to itself the compiler reads each operand just before its product.
    // `beside`(g) is other work that may go among the products of group g.
    template <bool PV, bool QK, int kAhead, typename F>
    __device__ __forceinline__ void products(const uint8_t *vt, const V8 (&p)[NS], const uint8_t *kt, f32x16 (&s)[NB],
                                             F &&beside) {
        constexpr int VG = ND < 4 ? ND : 4;                   // products of V in a group
        constexpr int NV = PV ? NS * ND / VG : 0;
        constexpr int KG = 4 / NB;                            // 16-column steps of K in a group
        constexpr int N = NV + (QK ? NQ / KG : 0);
        V8 f[kAhead + 1][4];
        auto read = [&](int g) {
            V8(&to)[4] = f[g % (kAhead + 1)];
            if (g < NV) {
#pragma unroll
                for (int j = 0; j < VG; ++j) {
                    using L4 = __attribute__((address_space(3))) s16x4;
                    struct Two {
                        s16x4 a, b;
                    } t;
                    const uint8_t *at = vt + v_at[(g * VG + j) % ND] + (g * VG + j) / ND * 16 * DP * 2;
                    t.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)at);
                    t.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)(at + 8 * DP * 2));
                    to[j] = __builtin_bit_cast(V8, t);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        to[k * NB + b] = *reinterpret_cast<const V8 *>(
                            kt + (k_at ^ (uint32_t((g - NV) * KG + k) << 5)) + b * 32 * DP * 2);
            }
        };
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
            if (g < N) read(g);
#pragma unroll
        for (int g = 0; g < N; ++g) {
            if (g + kAhead < N) read(g + kAhead);
            __builtin_amdgcn_sched_barrier(0);
            beside(g);
            const V8(&from)[4] = f[g % (kAhead + 1)];
            if (g < NV) {
#pragma unroll
                for (int j = 0; j < VG; ++j) {
                    const int d = (g * VG + j) % ND;
                    acc[d] = T::mfma(from[j], p[(g * VG + j) / ND], acc[d]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int step = (g - NV) * KG + k;
                        s[b] = T::mfma(from[k * NB + b], qf[step], step == 0 ? f32x16{} : s[b]);
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Weights of a tile's scores; the sums move to a new reference where a
    // row's maximum has left the slack.  The sum takes the weights in 32 bits.
    // The second product takes them rounded to the cache's type, since matrix
    // instructions multiply 16 bits by 16: in two halves, 32 bits would cost it
    // twice.  Against 64 bits the outputs are off by 0.0018-0.0022 in bfloat16
    // and 0.0003 in float16 (root mean square, relative), where weights
    // in 32 bits and one rounding of the output leave 0.0016-0.0017 and 0.0002.
    __device__ __forceinline__ void weights(const AttnArgs &a, int32_t start, bool masked, f32x16 (&s)[NB], V8 (&p)[NS]) {
        if (masked) {
            // seen: the keys see_lo .. see_lo + width - 1, in one comparison
            const uint32_t first = uint32_t(start - see_lo) + 4u * ((threadIdx.x >> 5) & 1u);
            const uint32_t width = uint32_t(max(see_hi - see_lo, 0));
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const uint32_t at = uint32_t(32 * b + 8 * (r / 4) + r % 4);
                    bool hidden = first + at >= width;
                    if constexpr (Sinks) hidden = hidden && first + uint32_t(see_lo) + at >= uint32_t(see_sinks);
                    if (hidden) s[b][r] = -INFINITY;
                    // (each comparison's lanes are 2 of the loop's scalar registers)
                    if constexpr (Sinks) __builtin_amdgcn_sched_barrier(0);
                }
        }
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
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r], a.scale_log2, off));
                l += e;
                p[2 * b + r / 8][r % 8] = E(e);
            }
    }

    // A masked key adds nothing, whatever its value holds, but 0 x inf in the
    // product is not nothing: note it, and see store().
    __device__ __forceinline__ void check(const uint8_t *vt) {
        constexpr uint32_t kE = T::kExp * 0x10001u, kO = T::kOne * 0x10001u;
        uint32_t bits = 0;
#pragma unroll 2
        for (uint32_t i = threadIdx.x % kWave; i < uint32_t(KT * DP / 8); i += 64u) {
            const uint4 x = reinterpret_cast<const uint4 *>(vt)[i];
            bits |= ((x.x & kE) + kO) | ((x.y & kE) + kO) | ((x.z & kE) + kO) | ((x.w & kE) + kO);
        }
        odd |= bits & 0x80008000u;
    }
};

// Tiles of K and V on their way from the cache to LDS through the registers of
// NT threads, thread gtid of them: NL pieces of 16 bytes of each.
template <typename E, int DP, int KT, int NT, bool Same, bool Sinks>
struct Loader {
    static constexpr int CPR = DP / 8;             // pieces per row
    static constexpr int NL = KT * CPR / NT;       // pieces per thread
    static constexpr int kStep = NT / CPR;         // rows from one piece of a thread to its next

    const uint8_t *kbase, *vbase;                  // of the cache head
    const int32_t *table;
    int32_t hi;
    uint32_t gtid, row, chunk;                     // of the thread's first piece
    uint32_t n_pages, page_shift;
    uint32_t k_page, k_slot, v_page, v_slot;       // strides in pieces
    bool whole_dim, same;
    int32_t sink_end, gap;                         // see key_at
    int32_t pages[NL];
    bool absent, missing;                          // a page that is none of the cache's: under way, ever (wavefront)
    uint4 kr[NL], vr[NL];

    __device__ __forceinline__ void init(const AttnArgs &a, const Piece &w, uint32_t kvh, uint32_t rw) {
        gtid = rw * 64u + threadIdx.x % kWave;
        row = gtid / CPR;
        chunk = gtid % CPR * 8u < a.dim ? gtid % CPR : 0u;
        table = a.table + int64_t(w.req) * a.table_stride;
        whole_dim = a.dim == DP;
        kbase = static_cast<const uint8_t *>(a.k) + uint64_t(kvh) * a.k_units[2] * 16u;
        vbase = static_cast<const uint8_t *>(a.v) + uint64_t(kvh) * a.v_units[2] * 16u;
        k_page = a.k_units[0], k_slot = a.k_units[1], v_page = a.v_units[0], v_slot = a.v_units[1];
        same = k_page == v_page && k_slot == v_slot;
        hi = end_of<Sinks>(a, w);
        if constexpr (Sinks) sink_end = a.sink_end, gap = w.gap;
        n_pages = a.n_pages;
        page_shift = a.page_shift;
        absent = missing = false;
    }

    // The token that a tile begins with.
    __device__ __forceinline__ int32_t token(int32_t start) const {
        return Sinks && start >= sink_end ? start + gap : start;
    }

    // The block table's entries for the thread's rows of the tile at `start`
    // (the piece's last row stands for those past it): read a tile ahead of
    // the load that uses them.
    __device__ __forceinline__ int32_t page_of(int32_t start, int n) const {
        return table[min(start + int32_t(row) + n * kStep, hi - 1) >> page_shift];
    }
    __device__ __forceinline__ void fetch_pages(int32_t start) {
#pragma unroll
        for (int n = 0; n < NL; ++n) pages[n] = page_of(token(start), n);
    }

    // A page that is none of the cache's is noted and the last one read in
    // its place, for an address that exists; rows past the piece are read, from
    // a page of the request.  put() leaves both out.
    __device__ __forceinline__ void load(int32_t start) {
        const uint32_t page_mask = (1u << page_shift) - 1u;
        uint32_t most = 0;
        start = token(start);
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const uint32_t in_page = (uint32_t(start) + row + uint32_t(n * kStep)) & page_mask;
            most = max(most, uint32_t(pages[n]));
            const uint32_t page = min(uint32_t(pages[n]), n_pages - 1u);
            const uint64_t at = uint64_t(page) * k_page + (uint64_t(in_page) * k_slot + chunk);
            kr[n] = *reinterpret_cast<const uint4 *>(kbase + at * 16u);
            if (Same || same)
                vr[n] = *reinterpret_cast<const uint4 *>(vbase + at * 16u);
            else
                vr[n] = *reinterpret_cast<const uint4 *>(
                    vbase + (uint64_t(page) * v_page + (uint64_t(in_page) * v_slot + chunk)) * 16u);
        }
        absent = __any(most >= n_pages);
        missing |= absent;
    }

    // Into LDS; rows past the piece, columns past the head and pages that are
    // none of the cache's become zeros.
    __device__ __forceinline__ void put(uint8_t *kt, uint8_t *vt, int32_t start) {
        start = token(start);
        if (!whole_dim || start + KT > hi || absent) {
            const bool in_dim = whole_dim || gtid % CPR == chunk;
#pragma unroll
            for (int n = 0; n < NL; ++n) {
                bool there = in_dim && start + int32_t(row) + n * kStep < hi;
                if (absent) there = there && uint32_t(page_of(start, n)) < n_pages;  // (which ones: seldom asked)
                const uint32_t keep = there ? ~0u : 0u;
                kr[n].x &= keep, kr[n].y &= keep, kr[n].z &= keep, kr[n].w &= keep;
                vr[n].x &= keep, vr[n].y &= keep, vr[n].z &= keep, vr[n].w &= keep;
            }
        }
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const uint32_t i = gtid + uint32_t(n) * NT;
            reinterpret_cast<uint4 *>(kt)[k_place<DP>(i / CPR, i % CPR)] = kr[n];
            reinterpret_cast<uint4 *>(vt)[v_place<DP>(i / CPR, i % CPR)] = vr[n];
        }
    }
};

// A page that is none of the cache's was read: told if a row sees a key of it.
// The piece's first tile of keys may begin before every row's window, where a
// request need not hold its pages any more.
template <bool Sinks>
__device__ __forceinline__ void tell_missing(const AttnArgs &a, const Piece &w) {
    int32_t lo, hi, first, gap;
    tile_keys<Sinks>(a, Req{w.q_start, w.q_len, w.kv_len}, w.row0, lo, hi, first, gap);
    const int32_t *table = a.table + int64_t(w.req) * a.table_stride;
    bool bad = false;
    auto look = [&](int32_t from, int32_t to) {  // the keys from .. to - 1
        if (from >= to) return;
        for (int32_t i = (from >> a.page_shift) + int32_t(threadIdx.x % kWave); i <= (to - 1) >> a.page_shift;
             i += int32_t(kWave))
            bad |= uint32_t(table[i]) >= a.n_pages;
    };
    look(max(first, key_at<Sinks>(a, w, w.lo)), end_of<Sinks>(a, w));
    if constexpr (Sinks) look(w.lo, min(w.hi, a.sinks));
    if (bad && a.status) atomicOr(a.status, kStatusCorrupt);
}

// The end of a workgroup of RW x KW wavefronts (along the rows, along the
// keys): every wavefront's rows go to LDS, and the wavefronts of a row group
// each write a share of its rows, joined over the key groups, so that stores
// run along the rows.  All of LDS but the maxima and sums at `ml_at` is free.
template <int DP>
constexpr uint32_t out_bytes() { return 32u * DP * 4u; }

template <typename E, int DP, int KT, int RW, int KW, bool Sinks>
__device__ __forceinline__ void store(const AttnArgs &a, const Piece &w, uint32_t kvh, uint8_t *lds, uint32_t ml_at,
                                      Rows<E, DP, KT, Sinks> &x, uint32_t wave) {
    using T = Type<E>;
    using V8 = typename T::V8;
    constexpr int CPR = DP / 8, ND = DP / 32;
    const uint32_t lane = threadIdx.x % kWave, c = lane & 31u, h = lane >> 5;
    const uint32_t rw = wave % RW, kw = wave / RW;
    const int32_t n_rows = w.q_len * int32_t(a.group);
    const float l = x.l + other_half(x.l);
    float *ml = reinterpret_cast<float *>(lds + ml_at) + 64u * wave;
    auto place = [&](uint32_t r, uint32_t q4) { return r * (DP / 4) + (q4 ^ (r & 7u)); };
    float4 *own = reinterpret_cast<float4 *>(lds + wave * out_bytes<DP>());
    __syncthreads();
    if (!__any(x.odd != 0)) {
        if (h == 0) *reinterpret_cast<float2 *>(ml + 2u * c) = float2{x.m, l};
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
                own[place(c, 8u * uint32_t(d) + 2u * uint32_t(q4) + h)] = float4{
                    x.acc[d][4 * q4], x.acc[d][4 * q4 + 1], x.acc[d][4 * q4 + 2], x.acc[d][4 * q4 + 3]};
    } else {
        rows_one_by_one<E, DP, Sinks>(a, w, kvh, 32u * rw, kw * KT, uint32_t(KW * KT), KT, reinterpret_cast<float *>(own), ml);
    }
    __syncthreads();
    auto weight = [&](float mk, float top) {
        return mk == top ? 1.0f : __builtin_amdgcn_exp2f((mk - top) * a.scale_log2);
    };
    ml = reinterpret_cast<float *>(lds + ml_at);
    const bool whole = w.splits == 1;
    const uint64_t slot = (uint64_t(w.slot + w.split) * a.kv_heads + kvh) * a.rows_per_tile;
#pragma unroll 2
    for (uint32_t i = lane; i < 32u / KW * CPR; i += 64u) {
        const uint32_t r = kw * (32u / KW) + i / CPR, ch = i % CPR;
        const int32_t at = int32_t(w.row0 + 32u * rw + r);
        if (at >= n_rows || ch * 8u >= a.dim) continue;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KW; ++k) top = fmaxf(top, ml[2u * (32u * (uint32_t(k) * RW + rw) + r)]);
        float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const uint32_t src = uint32_t(k) * RW + rw;
            const float2 v = *reinterpret_cast<const float2 *>(ml + 2u * (32u * src + r));
            const float f = KW == 1 ? 1.0f : weight(v.x, top);
            sum += v.y * f;
            const float4 *from = reinterpret_cast<const float4 *>(lds + src * out_bytes<DP>());
            const float4 x0 = from[place(r, 2u * ch)], x1 = from[place(r, 2u * ch + 1u)];
            o[0] += x0.x * f, o[1] += x0.y * f, o[2] += x0.z * f, o[3] += x0.w * f;
            o[4] += x1.x * f, o[5] += x1.y * f, o[6] += x1.z * f, o[7] += x1.w * f;
        }
        if (whole) {
            const int32_t t = at / int32_t(a.group), hg = at - t * int32_t(a.group);
            const uint32_t head = kvh * a.group + uint32_t(hg);
            const int64_t token = w.q_start + t;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key gives 0
            V8 y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = E(o[j] * inv);
            *reinterpret_cast<V8 *>(static_cast<E *>(a.out) + token * a.out_stride[0] + int64_t(head) * a.out_stride[1] +
                                    ch * 8u) = y;
            if (a.lse && ch == 0)
                a.lse[token * a.heads + head] =
                    sum == 0.0f ? -INFINITY : top * a.scale + (__builtin_amdgcn_logf(sum) - T::kBias) * 0.69314718f;
        } else {
            const uint64_t pr = slot + (uint32_t(at) - w.row0);
            float4 *to = reinterpret_cast<float4 *>(a.part_o + pr * DP + ch * 8u);
            to[0] = float4{o[0], o[1], o[2], o[3]};
            to[1] = float4{o[4], o[5], o[6], o[7]};
            if (ch == 0) *reinterpret_cast<float2 *>(a.part_ml + 2u * pr) = float2{top, sum};
        }
    }
}

// Four wavefronts, for decoding and small steps.  K and V go from the cache to
// registers and on to LDS: the load of the next tile is under way while this
// one is multiplied.  With RW = 1 every wavefront reads keys of its own, into
// one buffer and without barriers: what a step of few rows needs, since the
// keys pass through each compute unit once and two workgroups a compute unit
// keep 5 TB/s in flight (a second buffer would leave room for one).  With more
// along the rows, which share a tile's keys, one barrier a step suffices with
// two buffers.
// RW wavefronts along the rows and 4 / RW groups along the keys, tiles of KT
// keys dealt out to the groups in turn.
template <int DP, int RW, int KT>
struct Shape {
    static constexpr int KW = kWaves / RW;
    static constexpr int kBuffers = RW == 1 ? 1 : 2;             // a wavefront alone needs no second one
    static constexpr uint32_t kTileBytes = KT * DP * 2;          // of K or of V
    static constexpr uint32_t kGroupBytes = 2 * kTileBytes * kBuffers;
    static constexpr uint32_t kLoop = KW * kGroupBytes;
    static constexpr uint32_t kEnd = kWaves * out_bytes<DP>();
    static constexpr uint32_t kMl = kLoop > kEnd ? kLoop : kEnd;
    static constexpr uint32_t kLds = kMl + kWaves * 32 * 8;
};

template <typename E, int DP, int RW, int KT, bool Sinks>
__global__ __launch_bounds__(kThreads, DP > 128 ? 1 : 2) void attention_kernel(AttnArgs a) {
    using Sh = Shape<DP, RW, KT>;
    using R = Rows<E, DP, KT, Sinks>;
    constexpr int KW = Sh::KW;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t kvh = blockIdx.x % a.kv_heads, index = blockIdx.x / a.kv_heads;
    Piece w;
    if (!find_piece<kThreads, Sinks>(again(a), index, blockIdx.x == 0, reinterpret_cast<uint32_t *>(lds), w)) return;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t rw = wave % RW, kw = wave / RW;
    Loader<E, DP, KT, 64 * RW, false, Sinks> ld;
    ld.init(a, w, kvh, rw);
    const int32_t n_tiles = (w.hi - w.lo + KT - 1) / KT;
    const int32_t n_steps = (n_tiles + KW - 1) / KW;  // the same for every group: they meet at barriers
    auto tile_start = [&](int32_t step) { return w.lo + (step * KW + int32_t(kw)) * KT; };
    R x;
    if (n_steps) ld.fetch_pages(tile_start(0));
    x.init(a, w, kvh, 32u * rw);
    if (tile_start(0) < w.hi) {
        ld.load(tile_start(0));
        ld.fetch_pages(tile_start(1));
    }
    x.settle();

    for (int32_t step = 0; step < n_steps; ++step) {
        const int32_t start = tile_start(step);
        uint8_t *kt = lds + kw * Sh::kGroupBytes + (Sh::kBuffers == 2 ? uint32_t(step & 1) : 0u) * 2u * Sh::kTileBytes;
        uint8_t *vt = kt + Sh::kTileBytes;
        if constexpr (RW == 1) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        ld.put(kt, vt, start);
        // one barrier a step: a buffer is written again two steps later, when
        // every wavefront has passed the next step's barrier
        if constexpr (RW == 1)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        else
            __syncthreads();
        if (tile_start(step + 1) < w.hi) {
            ld.load(tile_start(step + 1));
            ld.fetch_pages(tile_start(step + 2));
        }
        if (x.skips(start)) continue;
        f32x16 s[R::NB];
        typename R::V8 p[R::NS];
        x.template products<false, true, 1>(vt, p, kt, s, nothing);
        const bool masked = x.masks(start);
        x.weights(a, start, masked, s, p);
        if (masked) x.check(vt);
        x.template products<true, false, 1>(vt, p, kt, s, nothing);
    }
    const AttnArgs &b = again(a);
    if (ld.missing) tell_missing<Sinks>(b, w);
    store<E, DP, KT, RW, KW, Sinks>(b, w, kvh, lds, Sh::kMl, x, wave);
}

// Eight wavefronts of 32 rows each, for steps with tiles of 256 rows for
// every compute unit.  Two wavefronts share a SIMD.  Left alone they fall into
// step, both at their products and then both at their exponentials, and the
// matrix unit idles half the time; here the second half of the workgroup runs
// one phase behind the first, held there by a barrier after every phase: while
// one half multiplies (V of the tile before, K of this one), the other takes
// its exponentials and moves the next tiles.
//
//   phase    2i              2i + 1          2i + 2
//   half 0   products i      weights i       products i + 1
//   half 1   weights i - 1   products i      weights i
//
// A half's loads of a tile leave the cache during its products and go to LDS
// as its weights begin.
//
// Against the four-wavefront kernel's 128-row tiles, on one card and in a graph:
// a prompt of 8192 tokens 549 and not 608 us, of 4100 193 and not 213.  The
// matrix units work 47% of the time: a phase of products takes some 1,900
// cycles where its 32 products take 1,024, since the reads of K and V (LDS gives
// 128 bytes a cycle to eight wavefronts) and the loads issue beside them.  No
// part alone decides: with its LDS reads left out the kernel takes 93% of the
// time, without its loads 92%, without its exponentials 95%.
//
// Products i read K tile i and V tile i - 1 in phases 2i and 2i + 1, so both
// halves put tile i + 1 into LDS by the end of phase 2i + 1: K into the place
// of K tile i - 1 and V, of three places, into that of V tile i - 2, which
// were last read in phase 2i - 1.
template <int DP>
struct Shape8 {
    static constexpr int KT = 64;
    static constexpr uint32_t kWaves8 = 8;
    static constexpr uint32_t kTileBytes = KT * DP * 2;
    static constexpr uint32_t kLoop = 5 * kTileBytes;            // two of K, three of V
    static constexpr uint32_t kEnd = kWaves8 * out_bytes<DP>();
    static constexpr uint32_t kMl = kLoop > kEnd ? kLoop : kEnd;
    static constexpr uint32_t kLds = kMl + kWaves8 * 32 * 8;
};

template <typename E, int DP, bool Sinks>
__global__ __launch_bounds__(512, 2) void attention8_kernel(AttnArgs a) {
    using Sh = Shape8<DP>;
    constexpr int KT = Sh::KT;
    using R = Rows<E, DP, KT, Sinks>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t kvh = blockIdx.x % a.kv_heads, index = blockIdx.x / a.kv_heads;
    Piece w;
    if (!find_piece<512, Sinks>(again(a), index, blockIdx.x == 0, reinterpret_cast<uint32_t *>(lds), w)) return;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool second = wave >= 4u;
    Loader<E, DP, KT, 512, true, Sinks> ld;  // (the launcher sees to it)
    ld.init(a, w, kvh, wave);
    const int32_t n = (w.hi - w.lo + KT - 1) / KT;
    auto tile_start = [&](int32_t t) { return w.lo + t * KT; };
    auto k_tile = [&](int32_t t) { return lds + uint32_t(t & 1) * Sh::kTileBytes; };
    R x;
    if (n) ld.fetch_pages(tile_start(0));
    x.init(a, w, kvh, 32u * wave);
    // half 0 moves tile t + 1 in its turn t, half 1 tile t + 2
    const int32_t lead = second ? 2 : 1;
    auto v_tile = [&](int32_t t) { return lds + uint32_t(2 + t % 3) * Sh::kTileBytes; };
    auto put = [&](int32_t t) {
        if (t < n) ld.put(k_tile(t), v_tile(t), tile_start(t));
    };
    // (past the end, the last tile again: nothing waits for it)
    auto load = [&](int32_t t) { ld.load(tile_start(min(t, n - 1))); };
    auto fetch = [&](int32_t t) { ld.fetch_pages(tile_start(min(t, n - 1))); };
    if (n) {
        load(0);
        fetch(1);
        put(0);
        if (second) {
            load(1);
            fetch(2);
        }
    }
    x.settle();
    __syncthreads();
    if (second) {
        put(1);
        __syncthreads();
    }
    // the wavefront's own tiles: t0 .. t1 - 1
    int32_t t = 0, t0 = 0, t1 = 0;
    if (!x.idle) {
        const int32_t first = Sinks && w.lo < a.sink_end ? w.lo : x.lo_min;  // every row sees the sinks
        t0 = min(max((first - w.lo) / KT, 0), n);
        t1 = min(max((x.hi_max - w.lo + KT - 1) / KT, t0), n);
    }
    auto turn_without_rows = [&]() {
        load(t + lead);
        fetch(t + lead + 1);
        __syncthreads();
        put(t + lead);
        __syncthreads();
        ++t;
    };
    while (t < t0) turn_without_rows();
    if (t0 < t1) {
        f32x16 s[R::NB];
        typename R::V8 p[R::NS];
        load(t + lead);
        fetch(t + lead + 1);
        x.template products<false, true, 1>(lds, p, k_tile(t), s, nothing);
        __syncthreads();
        put(t + lead);
        bool masked = x.masks(tile_start(t));
        x.weights(a, tile_start(t), masked, s, p);
        __syncthreads();
        for (++t; t < t1; ++t) {
            uint8_t *vt = v_tile(t - 1);
            if (masked) x.check(vt);
            x.template products<true, true, 2>(vt, p, k_tile(t), s, [&](int g) {
                if (g == 1) load(t + lead);
                if (g == 3) fetch(t + lead + 1);
            });
            __syncthreads();
            put(t + lead);
            masked = x.masks(tile_start(t));
            x.weights(a, tile_start(t), masked, s, p);
            __syncthreads();
        }
        uint8_t *vt = v_tile(t - 1);
        if (masked) x.check(vt);
        x.template products<true, false, 1>(vt, p, lds, s, nothing);
        if (t < n) turn_without_rows();
    }
    while (t < n) turn_without_rows();
    if (!second) __syncthreads();
    const AttnArgs &b = again(a);
    if (ld.missing) tell_missing<Sinks>(b, w);
    store<E, DP, KT, 8, 1, Sinks>(b, w, kvh, lds, Sh::kMl, x, wave);
}

// The pieces of a split tile joined.  A wavefront takes a row (WPR = 1, for
// tiles of many rows and few pieces) or a quarter of its pieces (WPR = 4);
// lanes run along the row in 16-byte steps and, where the row is shorter,
// over several pieces.  Each lane keeps its own running maximum.  The order
// of the pieces is fixed, so results repeat bit for bit.  Bound by the latency
// of its chain (count, tile, sums): 2.6 us for one tile of 4 rows, 9 us for the
// 28 MB of a step of 513 tokens over 32000.  A step in which nothing is split
// costs the launch alone.
template <typename E, int DP, int WPR>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a) {
    using T = Type<E>;
    constexpr uint32_t CPR = DP / 4;                     // float4 pieces per row
    constexpr uint32_t SL = 64 / CPR;                    // lanes side by side on one column
    constexpr uint32_t kRows = kWaves / WPR;             // rows at a time
    __shared__ float4 part_x[WPR == 4 ? 4 : 1][CPR];
    __shared__ float2 part_ml[4];
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t ch = lane % CPR, sl = lane / CPR;
    auto weight = [&](float m, float top) { return m == top ? 1.0f : __builtin_amdgcn_exp2f((m - top) * a.scale_log2); };
    // units: a share of the rows of one cache head of one tile
    const uint32_t units = *a.tile_count * a.kv_heads * a.join_shares;
    for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const uint32_t kvh = unit % a.kv_heads, rest = unit / a.kv_heads;
        const uint32_t share = rest % a.join_shares;
        const Tile w = a.tiles[rest / a.join_shares];
        const uint32_t splits = __builtin_amdgcn_readfirstlane(w.splits), slot = __builtin_amdgcn_readfirstlane(w.slot);
        const uint32_t row0 = __builtin_amdgcn_readfirstlane(w.row0), rows = __builtin_amdgcn_readfirstlane(w.rows);
        const int32_t token0 = __builtin_amdgcn_readfirstlane(w.token0);
        if (splits == 1u) continue;  // a shorter tile than its request's longest
        for (uint32_t r = share * kRows + (WPR == 4 ? 0u : wave); r < rows; r += a.join_shares * kRows) {
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
}

// ------------------------------------------------------------------ launch

// The launch's shape, from what the host knows: sizes only.
struct LaunchPlan {
    int rw, kt, dp;
    uint32_t rows_per_tile, min_piece, resident, extra, tile_cap, slot_cap, most_rows;
    float piece_cost, split_cost, join_cost;
    uint64_t off_tiles, off_ml, off_o, bytes;
};

// most rows a request has per cache head: no tile needs more
uint64_t most_rows(const dfc_attention_args &a) {
    return std::min<uint64_t>(a.max_q_len ? a.max_q_len : a.tokens, a.tokens) * (a.heads / a.cache.kv_heads);
}

int padded_dim(const dfc_attention_args &a) { return a.cache.head_dim <= 64 ? 64 : a.cache.head_dim <= 128 ? 128 : 256; }

// 32-row units of a tile of `most` rows, in the heights there are
int tallest(uint64_t most) { return most <= 32 ? 1 : most <= 64 ? 2 : most <= 128 ? 4 : 8; }

uint64_t most_tiles(const dfc_attention_args &a, int rw) {
    const uint64_t rows = a.tokens * (a.heads / a.cache.kv_heads);
    return std::min<uint64_t>(dfc::ceil_div(rows, uint64_t(32 * rw)) + (a.n_requests == 1 ? 0u : a.n_requests), rows);
}

uint32_t workgroups_at_once(int dp, int rw) { return dp > 128 || rw == 8 ? 256u : 512u; }

// Tile height, in units of 32 rows: the least whose tiles all run at once, but
// large tiles where keys are long, since they read K and V less often.  (us,
// Llama-3-8B heads, tiles of 32 / 64 / 128 / 256 rows; prompts of 200, 512,
// 1024, 2000, 4100: 11.1 / 12.8 / 16.5 / 19.7, 17.4 / 18.8 / 23.2 / 27.7, 40.0 /
// 33.3 / 39.2 / 45.0, 98 / 79 / 72 / 76, 327 / 254 / 213 / 193; 256 tokens over
// 2000: 43 / 42 / 63 / 70, 512 over 4000: 86 / 89 / 74 / 132, 256 over 32000: 274
// / 224 / 183 / 166.)  The limits were measured with these heads and are used for
// all.  The keys are those the table has room for, since the lengths are on the
// device: under a table for 8192 tokens or more a prompt of 512 takes 28.4 and
// not 16.1 us, of 200 16.7-19.5 and not 10.6, 64 single tokens over 700 49 and
// not 40 (launch_plan leaves them to be split then).
int tile_height(const dfc_attention_args &a, uint32_t sinks) {
    const uint32_t group = a.heads / a.cache.kv_heads;
    const uint64_t most = most_rows(a);
    const int dp = padded_dim(a), fit = tallest(most);
    uint64_t keys = uint64_t(a.max_pages) * a.cache.page_size;
    if (a.window) keys = std::min<uint64_t>(keys, uint64_t(a.window) + most / group + sinks);
    // pairs of 32 rows and 64 keys there may be
    const double pairs = double(a.tokens * group) / 32.0 * a.cache.kv_heads * double(keys) / 64.0;
    int rw = 1;
    for (double limit = 6000.0; rw < fit; rw *= 2, limit *= 3.3)
        if (pairs < limit && most_tiles(a, rw) * a.cache.kv_heads <= workgroups_at_once(dp, rw)) break;
    bool same = true;  // K and V have one layout
    for (int i = 0; i < 2; ++i) same = same && a.cache.k_stride[i] == a.cache.v_stride[i];
    return rw == 8 && !same ? 4 : rw;
}

// `cut`: a split counts for as little as it costs under a window, see below.
LaunchPlan launch_plan(const dfc_attention_args &a, uint32_t sinks, int rw, bool cut = false) {
    LaunchPlan p;
    const uint32_t group = a.heads / a.cache.kv_heads;
    p.dp = padded_dim(a);
    // at 256 columns eight wavefronts have no room for two key tiles, and one
    // that holds a whole key tile of K and V on its way to LDS no registers
    p.rw = p.dp > 128 ? std::min(std::max(rw, 2), 4) : rw;
    p.kt = p.rw >= 4 && p.dp <= 128 ? 64 : 32;
    p.rows_per_tile = 32u * uint32_t(p.rw);
    p.most_rows = uint32_t(std::min<uint64_t>(most_rows(a), p.rows_per_tile));
    p.resident = workgroups_at_once(p.dp, p.rw);
    p.min_piece = p.rw >= 4 ? 2u : kWaves / uint32_t(p.rw);
    // measured by their sweep: without split_cost 256 tokens over 256 took
    // 29.5 us and not 20.5, eight times 64 over 500 47.2 and not 23.9; at half
    // of it 300 over 700 took 33.6 and not 29.8
    p.piece_cost = 4.0f;
    p.split_cost = float(p.most_rows) / 4.0f;
    // Tall tiles under a window are longer than those: with sinks a split counts
    // for less (us with a quarter and a tenth of the rows, 32 heads over 8 of 128:
    // 1000 tokens over 32000 under 4096 + 64 138 and 102, 768 under 8192 + 64 250
    // and 142, 513 over 8192 under 2048 + 16 63 and 48, eight times 128 over 8000
    // 140 and 105; prompts the same).  The same would hold under a window without
    // sinks; those calls keep the old price, and with it the bits of their results.
    if (cut && p.rw >= 4) p.split_cost = float(p.most_rows) / 10.0f;
    p.join_cost = p.rw >= 4 ? 2.0f : 8.0f;
    const uint64_t tiles = most_tiles(a, p.rw);
    // a tile of c key tiles has at most ceil(c / min_piece) pieces
    uint64_t longest = dfc::ceil_div(uint64_t(a.max_pages) * a.cache.page_size, uint64_t(p.kt)) + 1u;
    const uint64_t each = longest > p.min_piece ? dfc::ceil_div(longest, uint64_t(p.min_piece)) - 1u : 0u;
    // Up to two rounds of pieces beyond one a tile.  With one, 64 requests of
    // 1 to 8191 tokens take 248 us and not 216 (four: 213); with four, 64 of
    // 700 take 55 and not 49: workgroups that find no piece come last, 2 us a
    // round.
    uint64_t extra = std::min<uint64_t>(2u * p.resident / a.cache.kv_heads + 1u, tiles * each);
    // The joining's launch alone costs 2.5 us, some five key tiles.  Where the
    // device could not win that back by splitting tiles as long as they may
    // be, none is split (one token over 250 keys: 9.4 and not 11.6 us, over 450
    // 12.0 / 11.4; prompt of 512 18.7 / 21.5, 128 tokens over 600 17.4 / 23.7, 64
    // single ones over 700 40 / 49).  The lengths of several requests may
    // differ, so that splitting pays however many tiles there are (64 of 1 to
    // 8191: 245 without, 216 with it): they are left to the device from 40 key
    // tiles on.
    if (a.window && a.causal)
        longest = std::min<uint64_t>(longest, (uint64_t(a.window) + p.rows_per_tile / group) / p.kt + 3u +
                                                  dfc::ceil_div(uint64_t(sinks), uint64_t(p.kt)));
    const double load = double(tiles) * a.cache.kv_heads / p.resident;
    const double rounds = a.n_requests == 1 ? std::ceil(load) : std::max(1.0, load);
    const double unsplit = rounds * (double(longest) + p.piece_cost);
    const double split = load * double(longest) + p.piece_cost + p.split_cost + p.join_cost + 5.0;
    if (unsplit <= split && (a.n_requests == 1 || longest <= 40u)) extra = 0;
    p.extra = uint32_t(extra);
    p.tile_cap = uint32_t(tiles);
    // a tile's pieces are at most twice those beyond its first
    p.slot_cap = uint32_t(std::min<uint64_t>(2u * extra, tiles + extra));
    p.off_tiles = 256;
    p.off_ml = (p.off_tiles + uint64_t(p.extra) * sizeof(Tile) + 255u) & ~uint64_t(255);
    const uint64_t rows = uint64_t(p.slot_cap) * a.cache.kv_heads * p.rows_per_tile;
    p.off_o = (p.off_ml + rows * 8u + 255u) & ~uint64_t(255);
    p.bytes = p.off_o + rows * uint64_t(p.dp) * 4u;
    return p;
}

// What a call needs depends on the window, and by the tile height on the
// layouts; one size has to serve every call of the same sizes.  A window, with
// sinks or without, never needs more.
uint64_t workspace_bytes(dfc_attention_args a) {
    uint64_t bytes = 0;
    a.window = 0;
    for (int rw = 1; rw <= tallest(most_rows(a)); rw *= 2) bytes = std::max(bytes, launch_plan(a, 0, rw).bytes);
    return bytes;
}

dfc_status check_attention(const dfc_attention_args &a) {
    const dfc_status cs = dfc::check_cache(a.cache);
    if (cs != DFC_OK) return cs;
    if (!a.heads || a.heads % a.cache.kv_heads || a.heads > 65536u) return DFC_EINVAL;
    if (a.tokens > 0x7fffffffull || a.n_requests > 0x7fffffffu) return DFC_EINVAL;
    // rows (tokens x heads of a group), and the tiles of 64 requests, are
    // counted in 32 bits
    if (a.tokens * (a.heads / a.cache.kv_heads) > 0x3fffffffull) return DFC_EUNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (a.cache.k_stride[i] >> 34 || a.cache.v_stride[i] >> 34) return DFC_EUNSUPPORTED;
    if (!(a.scale > 0.0f) || !std::isfinite(a.scale)) return DFC_EINVAL;
    if (a.window > 0x7fffffffu) return DFC_EINVAL;
    return DFC_OK;
}

template <typename E, int DP, int RW, int KT, bool Sinks>
dfc_status launch(const AttnArgs &a, const LaunchPlan &p, hipStream_t st) {
    constexpr uint32_t kLds = RW == 8 ? Shape8<DP>::kLds : Shape<DP, RW == 8 ? 4 : RW, KT>::kLds;
    void (*kernel)(AttnArgs);
    if constexpr (RW == 8)
        kernel = &attention8_kernel<E, DP, Sinks>;
    else
        kernel = &attention_kernel<E, DP, RW, KT, Sinks>;
    if (!allow_full_lds(reinterpret_cast<const void *>(kernel))) return DFC_EHIP;
    const uint64_t grid = (uint64_t(p.tile_cap) + p.extra) * a.kv_heads;
    if (grid > 0x7fffffffull) return DFC_EUNSUPPORTED;
    hipLaunchKernelGGL(kernel, dim3(uint32_t(grid)), dim3(RW == 8 ? 512 : kThreads), kLds, st, a);
    if (a.tiles) {
        constexpr int WPR = RW >= 4 ? 1 : 4;
        // as many workgroups as may have work, up to a few per compute unit
        const uint64_t units = uint64_t(p.extra) * a.kv_heads * a.join_shares;
        if (units > 0xffffffffull) return DFC_EUNSUPPORTED;
        hipLaunchKernelGGL((join_kernel<E, DP, WPR>), dim3(uint32_t(std::min<uint64_t>(units, 2048u))), dim3(kThreads), 0,
                           st, a);
    }
    return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP;
}

template <typename E, bool Sinks>
dfc_status launch_type(const AttnArgs &a, const LaunchPlan &p, hipStream_t st) {
    switch (p.dp * 16 + p.rw) {
        case 64 * 16 + 1: return launch<E, 64, 1, 32, Sinks>(a, p, st);
        case 64 * 16 + 2: return launch<E, 64, 2, 32, Sinks>(a, p, st);
        case 64 * 16 + 4: return launch<E, 64, 4, 64, Sinks>(a, p, st);
        case 64 * 16 + 8: return launch<E, 64, 8, 64, Sinks>(a, p, st);
        case 128 * 16 + 1: return launch<E, 128, 1, 32, Sinks>(a, p, st);
        case 128 * 16 + 2: return launch<E, 128, 2, 32, Sinks>(a, p, st);
        case 128 * 16 + 4: return launch<E, 128, 4, 64, Sinks>(a, p, st);
        case 128 * 16 + 8: return launch<E, 128, 8, 64, Sinks>(a, p, st);
        case 256 * 16 + 2: return launch<E, 256, 2, 32, Sinks>(a, p, st);
        default: return launch<E, 256, 4, 32, Sinks>(a, p, st);
    }
}

}  // namespace

extern "C" {

dfc_status dfc_paged_attention_workspace(const dfc_attention_args *args, uint64_t *bytes) {
    if (!args || !bytes) return DFC_EINVAL;
    const dfc_status s = check_attention(*args);
    if (s != DFC_OK) return s;
    *bytes = args->tokens && args->n_requests ? workspace_bytes(*args) : 0;
    return DFC_OK;
}

dfc_status dfc_paged_attention(const dfc_attention_args *args, void *stream) {
    return dfc_paged_attention_sinks(args, 0, stream);
}

dfc_status dfc_paged_attention_sinks(const dfc_attention_args *args, uint32_t sinks, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_attention_args &in = *args;
    const dfc_status s = check_attention(in);
    if (s != DFC_OK) return s;
    if (sinks > 0x7fffffffu) return DFC_EINVAL;
    // without a window every token is visible; there are no more tokens than
    // the table has room for
    if (!in.window) sinks = 0;
    sinks = uint32_t(std::min<uint64_t>({sinks, uint64_t(in.max_pages) * in.cache.page_size, 0x7ffffe00u}));
    if (!in.tokens || !in.n_requests) return DFC_OK;
    if (!in.q_dev || !in.out_dev || !in.cu_q || !in.seq_lens || !in.workspace_dev) return DFC_EINVAL;
    if (in.max_pages && !in.block_table) return DFC_EINVAL;
    if (in.table_stride < int64_t(in.max_pages)) return DFC_EINVAL;
    if ((reinterpret_cast<uintptr_t>(in.q_dev) | reinterpret_cast<uintptr_t>(in.out_dev)) & 15u) return DFC_EINVAL;
    if (reinterpret_cast<uintptr_t>(in.workspace_dev) & 255u) return DFC_EINVAL;
    for (int i = 0; i < 2; ++i)
        if (in.q_stride[i] % 8 || in.out_stride[i] % 8) return DFC_EINVAL;
    const uint64_t bytes = workspace_bytes(in);
    if (in.workspace_bytes < bytes) return DFC_ESIZE;
    const int rw = tile_height(in, sinks);
    LaunchPlan p = launch_plan(in, sinks, rw, sinks > 0);
    // where no call without a window splits its tiles there is no room for it
    if (p.bytes > bytes) p = launch_plan(in, sinks, rw);
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
        a.k_units[i] = uint32_t(in.cache.k_stride[i] / 8);
        a.v_units[i] = uint32_t(in.cache.v_stride[i] / 8);
    }
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
    a.rows_shift = dfc::log2_of(p.rows_per_tile);
    a.key_shift = dfc::log2_of(uint32_t(p.kt));
    a.min_piece = p.min_piece;
    a.resident = p.resident;
    a.piece_cost = p.piece_cost;
    a.split_cost = p.split_cost;
    a.join_cost = p.join_cost;
    a.extra = p.extra;
    a.tile_cap = p.tile_cap;
    a.join_shares = p.rw >= 4 ? (p.most_rows + 7u) / 8u : p.most_rows;
    uint8_t *ws = static_cast<uint8_t *>(in.workspace_dev);
    a.tile_count = reinterpret_cast<uint32_t *>(ws);
    a.tiles = p.extra ? reinterpret_cast<Tile *>(ws + p.off_tiles) : nullptr;
    a.part_ml = reinterpret_cast<float *>(ws + p.off_ml);
    a.part_o = reinterpret_cast<float *>(ws + p.off_o);
    a.status = in.status_dev;
    a.sinks = int32_t(sinks);
    a.sink_end = int32_t((sinks + uint32_t(p.kt) - 1u) / uint32_t(p.kt) * uint32_t(p.kt));
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool bf = in.cache.dtype == DFC_BF16;
    if (sinks) return bf ? launch_type<__bf16, true>(a, p, st) : launch_type<_Float16, true>(a, p, st);
    return bf ? launch_type<__bf16, false>(a, p, st) : launch_type<_Float16, false>(a, p, st);
}

}  // extern "C"
