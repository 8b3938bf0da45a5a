// dfc_verify.hip - drafted tokens against the model's probabilities, and the
// token that follows them, from given random numbers.
//
// With p = softmax(z / T) of a row of the model's logits and q the drafter's,
// draft x holds if u q(x) < p(x), and the token that follows the drafts that
// hold is found by inverting the sums of w = max(p - q, 0), or of p where no
// draft was refused.
//
// Which token that is changes where the sums cross u sum(w).  Of V tokens whose
// sums are off by a factor of 1 + e, a random number lands next to a border with
// a probability of up to 2 e V: one call in 40 for e = 1e-7 and a vocabulary of
// 128256.  Exponentials and sums are therefore in 64 bits, to their last bits, where
// it is one in 10^8 at most.  (Differences of rows that nearly agree are off by more
// of themselves: by 5e-14 over the sum of max(p - q, 0), which is also about how
// often such a draft is refused.)
//
// A row is cut into pieces of 1,024 values, one a wavefront and 16 a lane, which
// are read once: their largest, its first index, and the sum of
// exp((z - largest) / T), all without a word to other wavefronts.  Everything
// after that works on a row's few pieces, and on one piece of values for the
// token itself; only where a draft is refused against a drafter's logits are the
// two rows read again, since max(p - q, 0) needs both of their sums first.
//
// Bounds (one MI355X, 128256 values a row in fp32, medians).  64 requests of five
// drafts, 328 MB of logits that count: the pass over them 71-74 us, 4.4-4.6 TB/s, nearly
// the rate of a copy and nearly as long as its 24 instructions a value take (with
// sums of the values in place of their exponentials it took 50), then 7 us to
// decide, 15 for the refused rows (66 MB, 4.4 TB/s), 6 for the tokens.  One row:
// 3.8 and 6.4 us, latency.  The whole call (98 us, floor 65): without a drafter's
// logits 50 (39).  In 16 bits the bytes halve and the instructions stay: 91 (33),
// without a drafter's logits 47 (20).  Rows that are not 16-byte aligned come a value
// at a time: a vocabulary of 128257 114 and, in 16 bits, 153.  Every wavefront looks
// through all of cu_rows: 512 single rows 78 (52), 1,024 of 32000 57 (26), 4,096 of
// them 335 (104).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "dfc.h"
#include "dfc_decode_core.h"
#include "dfc_format.h"

namespace {

constexpr uint32_t kVThreads = 256;
constexpr uint32_t kVWaves = kVThreads / kWave;
constexpr uint32_t kPerLane = 16;                    // values
constexpr uint32_t kPiece = kPerLane * kWave;
constexpr uint32_t kMostRequests = 65536;
constexpr uint32_t kMostGroups = 0xffffffffu / kVThreads;  // a launch counts its threads in 32 bits

// What a row's piece holds; top is NaN where a value is NaN or +inf.
struct alignas(16) Part {
    float top;
    uint32_t at;  // lowest index of the largest value
    double sum;   // of exp((z - top) / T); 0 for T = 0 and where nothing is above -inf
};

// What was found for a request.
struct alignas(16) Found {
    double p_scale, q_scale;  // p = p_scale exp((z - p_top) / T)
    float p_top, q_top;
    uint32_t row, accepted;   // the row that the token is drawn from
    int32_t drafted;          // a refused draft without a drafter's logits, which has no weight; -1: none
    uint32_t mode;
    uint32_t bad;             // what the status is told of the row
    uint32_t pad;
};
enum : uint32_t { kNone = 0, kGreedy = 1, kPlain = 2, kRest = 3 };  // no token; the largest; of p; of max(p - q, 0)

struct VerifyArgs {
    dfc_verify_args a;
    uint32_t pieces;       // of a row
    uint32_t groups;       // workgroups a row
    Part *target, *draft;  // rows x pieces
    double *rest;          // n_requests x pieces: sums of max(p - q, 0)
    Found *found;
};

// Inclusive prefix of an operation over the wavefront (DPP row shifts, then row
// broadcasts 15 and 31), and its last value, for every lane.
struct Sum {
    static constexpr double kNone = 0.0;
    static __device__ __forceinline__ double of(double a, double b) { return a + b; }
};
struct Largest {
    static constexpr float kNone = -INFINITY;
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};
struct Least {
    static constexpr uint32_t kNone = ~0u;
    static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return min(a, b); }
};

template <int Ctrl, int Rows, typename T>
__device__ __forceinline__ T shifted(T x, T none) {
    if constexpr (sizeof(T) == 8) {
        using Two = __attribute__((ext_vector_type(2))) int;
        const Two v = __builtin_bit_cast(Two, x), o = __builtin_bit_cast(Two, none);
        return __builtin_bit_cast(T, Two{__builtin_amdgcn_update_dpp(o.x, v.x, Ctrl, Rows, 0xf, false),
                                         __builtin_amdgcn_update_dpp(o.y, v.y, Ctrl, Rows, 0xf, false)});
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x),
                                                                 Ctrl, Rows, 0xf, false));
    }
}
template <typename F, typename T>
__device__ __forceinline__ T scan_of(T x) {
    x = F::of(x, shifted<0x111, 0xf>(x, F::kNone));
    x = F::of(x, shifted<0x112, 0xf>(x, F::kNone));
    x = F::of(x, shifted<0x114, 0xf>(x, F::kNone));
    x = F::of(x, shifted<0x118, 0xf>(x, F::kNone));
    x = F::of(x, shifted<0x142, 0xa>(x, F::kNone));
    return F::of(x, shifted<0x143, 0xc>(x, F::kNone));
}
template <typename T>
__device__ __forceinline__ T of_lane(T x, uint32_t lane) {
    if constexpr (sizeof(T) == 8) {
        using Two = __attribute__((ext_vector_type(2))) int;
        const Two v = __builtin_bit_cast(Two, x);
        return __builtin_bit_cast(T, Two{__builtin_amdgcn_readlane(v.x, lane), __builtin_amdgcn_readlane(v.y, lane)});
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
    }
}
template <typename F, typename T>
__device__ __forceinline__ T over_wave(T x) {
    return of_lane(scan_of<F>(x), kWave - 1);
}

// 2^t for t <= 0, within 6.3e-16 of it and 1 for 0: t = n + f with |f| <= 1/2 by
// adding and taking off a number whose last bit is 1, and 2^f as 1 + f q(f), q the
// polynomial of degree 9 through (2^f - 1) / f at the Chebyshev nodes of
// [-1/2, 1/2].  A degree less is off by 4e-14, as much as some 300 roundings of 64
// bits: it answered for drafts next to the border what the definition does not.  Its
// instructions decide, 3 a degree: 64 requests of five drafts 98.6 us in a graph with
// this, 96.0 with the degree less; some 30 more with a library's exponential, which
// has twice as many.  (With a table of 64 roots and degree 4, a quarter fewer, it
// took the same.)
__device__ __forceinline__ double exp2_of(double t) {
    t = fmax(t, -1100.0);  // (2^-1100 is 0)
    const double whole = t + 0x1.8p52, f = t - (whole - 0x1.8p52);
    double y = 0x1.e5e9f548e5725p-28;
    y = fma(y, f, 0x1.b6571de2f2351p-24);
    y = fma(y, f, 0x1.62bfe46117445p-20);
    y = fma(y, f, 0x1.ffcb76789860fp-17);
    y = fma(y, f, 0x1.4309130378460p-13);
    y = fma(y, f, 0x1.5d87fe908f88ap-10);
    y = fma(y, f, 0x1.3b2ab6fba385fp-7);
    y = fma(y, f, 0x1.c6b08d7044119p-5);
    y = fma(y, f, 0x1.ebfbdff82c590p-3);
    y = fma(y, f, 0x1.62e42fefa39f7p-1);
    y = fma(y, f, 1.0);
    return __builtin_ldexp(y, int(uint32_t(__builtin_bit_cast(uint64_t, whole))));
}

// exp((z - top) / T) for z <= top, `rate` = log2(e) / T.
__device__ __forceinline__ double weight_of(float z, float top, double rate) {
    return exp2_of((double(z) - double(top)) * rate);
}
__device__ __forceinline__ double rate_of(float t) { return t > 0.0f ? 1.4426950408889634 / double(t) : 0.0; }

// The value in [0, 1) nearest to a random number that is none; NaN stays.
__device__ __forceinline__ float within(float u) {
    return u != u ? u : fminf(fmaxf(u, 0.0f), 0x1.fffffep-1f);
}

// The request of a row: the number of requests that end at or before it.
__device__ __forceinline__ uint32_t request_of(const dfc_verify_args &a, uint32_t row) {
    uint32_t n = 0;
    for (uint32_t r = threadIdx.x % kWave; r - threadIdx.x % kWave < a.n_requests; r += kWave)
        n += uint32_t(__popcll(__ballot(r < a.n_requests && int64_t(a.cu_rows[r + 1u]) <= int64_t(row))));
    return __builtin_amdgcn_readfirstlane(n);
}

// A request's rows, held inside the buffers.
struct Rows {
    uint32_t first, count;
};
__device__ __forceinline__ Rows rows_of(const dfc_verify_args &a, uint32_t r, uint32_t &bad) {
    const int64_t c0 = a.cu_rows[r], c1 = a.cu_rows[r + 1u], rows = int64_t(a.rows);
    const int64_t first = min(max(c0, int64_t(0)), rows), end = min(max(c1, first), rows);
    if (c0 != first || c1 != end) bad |= kStatusCorrupt;
    return Rows{uint32_t(first), uint32_t(end - first)};
}

__device__ __forceinline__ float temperature_of(const dfc_verify_args &a, uint32_t r) {
    return a.temperature ? a.temperature[r] : 1.0f;
}

// Index in the row of the lane's value i of a piece: lanes take runs of W
// values side by side.
template <uint32_t W>
__device__ __forceinline__ uint32_t index_of(uint32_t piece, uint32_t i) {
    return piece * kPiece + (i / W * kWave + threadIdx.x % kWave) * W + i % W;
}

// A lane's 16 values of a piece of a row; -inf past the row.  Loads pass the
// caches by: most logits are read once (64 requests of five drafts 3% faster, one
// row the same).
template <typename E>
__device__ __forceinline__ void load_piece(const E *row, uint32_t vocab, uint32_t piece, float (&x)[kPerLane]) {
    constexpr uint32_t W = 16u / sizeof(E);
    using V = __attribute__((ext_vector_type(W))) E;
    const bool whole = (uint64_t(piece) + 1u) * kPiece <= vocab;
    if (whole && (reinterpret_cast<uintptr_t>(row) & 15u) == 0) {
#pragma unroll
        for (uint32_t k = 0; k < kPerLane / W; ++k) {
            const V v = __builtin_nontemporal_load(reinterpret_cast<const V *>(row + index_of<W>(piece, k * W)));
#pragma unroll
            for (uint32_t j = 0; j < W; ++j) x[k * W + j] = float(v[j]);
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i) {
            const uint32_t at = index_of<W>(piece, i);
            x[i] = at < vocab ? float(row[at]) : -INFINITY;
        }
    }
}

template <typename E>
__device__ __forceinline__ Part part_of(const float (&x)[kPerLane], uint32_t piece, float t) {
    constexpr uint32_t W = 16u / sizeof(E);
    float top = x[0];  // NaN if one is: an instruction for two values, where fmaxf took four
#pragma unroll
    for (uint32_t i = 1; i < kPerLane; ++i) top = __builtin_elementwise_maximum(top, x[i]);
    const bool odd = top != top;
    top = over_wave<Largest>(top);
    Part p{top, 0u, 0.0};
    if (__any(odd) || top == INFINITY) {
        p.top = __builtin_nanf("");
    } else if (t == 0.0f) {
        uint32_t at = ~0u;
#pragma unroll
        for (uint32_t i = kPerLane; i-- > 0;)
            if (x[i] == top) at = index_of<W>(piece, i);
        p.at = over_wave<Least>(at);
    } else if (top > -INFINITY) {
        const double rate = rate_of(t);
        double s = 0.0;
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i) s += weight_of(x[i], top, rate);
        p.sum = over_wave<Sum>(s);
    }
    return p;
}

// The pieces of the model's rows, and behind them of the drafter's.  (Several
// pieces a wavefront, the next one loaded before this one's sums: 111 us for the
// call with two and with four, 112 with one, 117 with sixteen.)
template <typename E>
__global__ __launch_bounds__(kVThreads) void parts_kernel(VerifyArgs p) {
    const dfc_verify_args &a = p.a;
    const uint32_t lane = threadIdx.x % kWave;
    uint32_t row = blockIdx.x / p.groups;
    const uint32_t piece = blockIdx.x % p.groups * kVWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (piece >= p.pieces) return;
    float x[kPerLane];
    if (row < a.rows) {
        load_piece(static_cast<const E *>(a.logits_dev) + int64_t(row) * a.logits_stride, a.vocab, piece, x);
        const uint32_t r = request_of(a, row);
        if (r >= a.n_requests) return;
        const Part y = part_of<E>(x, piece, temperature_of(a, r));
        if (lane == 0) p.target[uint64_t(row) * p.pieces + piece] = y;
    } else {
        row -= uint32_t(a.rows);
        const uint32_t r = request_of(a, row);
        // nothing was drafted from a request's last row, and greedy answers need no q
        if (r >= a.n_requests || a.cu_rows[r + 1u] == int32_t(row) + 1) return;
        const float t = temperature_of(a, r);
        if (t == 0.0f) return;
        load_piece(static_cast<const E *>(a.draft_logits_dev) + int64_t(row) * a.draft_stride, a.vocab, piece, x);
        const Part y = part_of<E>(x, piece, t);
        if (lane == 0) p.draft[uint64_t(row) * p.pieces + piece] = y;
    }
}

// A row's pieces joined by a wavefront.
struct Whole {
    double sum;  // of exp((z - top) / T)
    float top;
    uint32_t at;
    uint32_t ok;  // the row has probabilities
    uint32_t pad;
};
__device__ __forceinline__ Whole whole_of(const Part *parts, uint32_t pieces, float t) {
    const uint32_t lane = threadIdx.x % kWave;
    const double rate = rate_of(t);
    float top = -INFINITY;
    uint32_t at = ~0u;
    double sum = 0.0;
    bool odd = false;
    for (uint32_t k = lane; k < pieces; k += kWave) {
        const Part x = parts[k];
        odd |= !(x.top < INFINITY);
        // pieces come in the order of their indexes: a later one has to be larger
        if (x.top > top) {
            sum = sum > 0.0 ? sum * weight_of(top, x.top, rate) : 0.0;
            top = x.top;
            at = x.at;
        }
        if (x.sum > 0.0) sum += x.sum * weight_of(x.top, top, rate);
    }
    Whole w;
    w.top = over_wave<Largest>(top);
    w.at = over_wave<Least>(top == w.top ? at : ~0u);
    w.sum = over_wave<Sum>(sum > 0.0 ? sum * weight_of(top, w.top, rate) : 0.0);
    w.ok = !__any(odd) && w.top > -INFINITY;
    w.pad = 0;
    return w;
}

// The drafts of a request that hold, and where its next token comes from.
// Called by all wavefronts of a workgroup: each joins the pieces of a row at a
// time, and then the lanes of all of them look at a draft each.
constexpr uint32_t kDecideThreads = 1024, kDecideWaves = kDecideThreads / kWave;
struct Decision {
    Whole target[kDecideWaves], draft[kDecideWaves];
    Found f;
};
template <typename E>
__device__ __forceinline__ Found decide(const VerifyArgs &p, uint32_t r, Decision &lds) {
    const dfc_verify_args &a = p.a;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    Found none{};
    const Rows rows = rows_of(a, r, none.bad);
    const float t = temperature_of(a, r);
    none.drafted = -1;
    none.row = rows.first;
    if (!rows.count) return none;
    if (!(t >= 0.0f) || !(t < INFINITY)) {
        none.bad = kStatusCorrupt;
        return none;
    }
    const double rate = rate_of(t);
    const bool against = a.draft_logits_dev && t > 0.0f;
    for (uint32_t i0 = 0; i0 < rows.count; i0 += kDecideWaves) {
        const uint32_t here = min(rows.count - i0, kDecideWaves);
        // the model's rows, then the drafter's but for the last
        for (uint32_t j = wave; j < (against ? 2u * here : here); j += kDecideWaves) {
            const bool model = j < here;
            const uint32_t i = model ? j : j - here;
            if (!model && i0 + i + 1u == rows.count) continue;
            const Whole w = whole_of((model ? p.target : p.draft) + uint64_t(rows.first + i0 + i) * p.pieces, p.pieces, t);
            if (lane == 0) (model ? lds.target : lds.draft)[i] = w;
        }
        __syncthreads();
        bool stops = false;
        Found f = none;
        if (lane < here) {
            const uint32_t i = i0 + lane, row = rows.first + i;
            const bool last = i + 1u == rows.count;
            const int64_t x = last ? 0 : a.drafts[row];
            const bool there = x >= 0 && x < int64_t(a.vocab);
            const Whole w = lds.target[lane];
            f.row = row;
            f.accepted = i;
            stops = last || !w.ok;
            if (w.ok && t == 0.0f) {
                f.mode = kGreedy;
                f.drafted = int32_t(w.at);
                stops = last || x != int64_t(w.at);
            } else if (w.ok) {
                f.mode = kPlain;
                f.p_top = w.top;
                f.p_scale = 1.0 / w.sum;
                if (!last) {
                    auto share = [&](const void *logits, int64_t stride, const Whole &of) {
                        const E z = static_cast<const E *>(logits)[int64_t(row) * stride + (there ? x : 0)];
                        return weight_of(float(z), of.top, rate) / of.sum;
                    };
                    const double px = there ? share(a.logits_dev, a.logits_stride, w) : 0.0;
                    double qx = 1.0;
                    if (against) {
                        const Whole v = lds.draft[lane];
                        f.q_top = v.top;
                        f.q_scale = 1.0 / v.sum;
                        if (!v.ok) f.mode = kNone;  // nothing can be drawn against what is not known
                        if (there) qx = share(a.draft_logits_dev, a.draft_stride, v);
                    }
                    stops = f.mode == kNone || !(double(within(a.uniforms[row])) * qx < px);
                    if (stops && f.mode == kPlain) {
                        if (against)
                            f.mode = kRest;
                        else if (there)
                            f.drafted = int32_t(x);
                    }
                }
            }
            if (f.mode == kNone || !(last || there)) f.bad |= kStatusCorrupt;
        }
        const uint64_t who = __ballot(stops);  // the same for every wavefront
        if (who && wave == 0 && lane == uint32_t(__builtin_ctzll(who))) lds.f = f;
        __syncthreads();
        if (who) return lds.f;
    }
    return none;
}

// The weights that a token is drawn with: a lane's 16 of a piece.
template <typename E>
__device__ __forceinline__ void weights_of(const VerifyArgs &p, const Found &f, float t, uint32_t piece,
                                           double (&w)[kPerLane]) {
    constexpr uint32_t W = 16u / sizeof(E);
    const dfc_verify_args &a = p.a;
    const double rate = rate_of(t);
    float x[kPerLane];
    load_piece(static_cast<const E *>(a.logits_dev) + int64_t(f.row) * a.logits_stride, a.vocab, piece, x);
    if (f.mode == kRest) {
        float y[kPerLane];
        load_piece(static_cast<const E *>(a.draft_logits_dev) + int64_t(f.row) * a.draft_stride, a.vocab, piece, y);
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i) {
            const double px = f.p_scale * weight_of(x[i], f.p_top, rate), qx = f.q_scale * weight_of(y[i], f.q_top, rate);
            w[i] = px > qx ? px - qx : 0.0;
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i)
            w[i] = int32_t(index_of<W>(piece, i)) == f.drafted ? 0.0 : weight_of(x[i], f.p_top, rate);
    }
}

template <typename E>
__global__ __launch_bounds__(kDecideThreads) void decide_kernel(VerifyArgs p) {
    __shared__ Decision lds;
    const Found f = decide<E>(p, blockIdx.x, lds);
    if (threadIdx.x == 0) p.found[blockIdx.x] = f;
}

// What is left of p where a draft was refused against a drafter's q, summed
// over each piece.
template <typename E>
__global__ __launch_bounds__(kVThreads) void rest_kernel(VerifyArgs p) {
    const uint32_t r = blockIdx.x / p.groups;
    const uint32_t piece = blockIdx.x % p.groups * kVWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Found f = p.found[r];
    if (f.mode != kRest || piece >= p.pieces) return;
    double w[kPerLane];
    weights_of<E>(p, f, temperature_of(p.a, r), piece, w);
    double s = 0.0;
#pragma unroll
    for (uint32_t i = 0; i < kPerLane; ++i) s += w[i];
    s = over_wave<Sum>(s);
    if (threadIdx.x % kWave == 0) p.rest[uint64_t(r) * p.pieces + piece] = s;
}

// The token: first the piece in which the sums pass the random number's share
// of them all, then the value.  The sum of all pieces is the last of the prefix
// sums that are searched, so some piece passes; within it the sums are added in
// another order, and where none passes by a rounding the last value with any
// weight is it.  A wavefront's work: the prefix sums of the first kAhead pieces a
// lane are kept, those of larger vocabularies are added up twice.
template <typename E>
__device__ __forceinline__ int64_t draw(const VerifyArgs &p, Found f, uint32_t r, float u) {
    constexpr uint32_t W = 16u / sizeof(E), kAhead = 4;
    const uint32_t lane = threadIdx.x % kWave;
    const float t = temperature_of(p.a, r);
    const double rate = rate_of(t);
    const Part *parts = p.target + uint64_t(f.row) * p.pieces;
    const double *rest = p.rest + uint64_t(r) * p.pieces;
    double all = 0.0, without = 0.0;  // without: the drafted token's piece without it
    double w[kPerLane], ahead[kAhead];
    bool some[kAhead];
    auto weight = [&](uint32_t k) -> double {
        if (k >= p.pieces) return 0.0;
        if (f.mode == kRest) return rest[k];
        const Part x = parts[k];
        if (f.drafted >= 0 && uint32_t(f.drafted) / kPiece == k) return without;
        return x.sum > 0.0 ? x.sum * weight_of(x.top, f.p_top, rate) : 0.0;
    };
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        if (f.mode == kPlain && f.drafted >= 0) {
            weights_of<E>(p, f, t, uint32_t(f.drafted) / kPiece, w);
#pragma unroll
            for (uint32_t i = 0; i < kPerLane; ++i) without += w[i];
            without = over_wave<Sum>(without);
        }
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            ahead[i] = weight(i * kWave + lane);
            some[i] = ahead[i] > 0.0;
        }
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            ahead[i] = scan_of<Sum>(ahead[i]);
            all += of_lane(ahead[i], kWave - 1);
        }
#pragma unroll 1
        for (uint32_t k0 = kAhead * kWave; k0 < p.pieces; k0 += kWave) all += over_wave<Sum>(weight(k0 + lane));
        if (all > 0.0) break;
        f.mode = kPlain;  // nothing is left: of p
        f.drafted = -1;
    }
    const double share = u == u ? double(within(u)) * all : 0.0;
    double before = 0.0;
    uint32_t piece = 0;
    bool found = false;
    // (prefix sums round apart: one may pass where nothing was added)
    auto look = [&](uint32_t k0, double sum, bool has) {
        const uint64_t past = __ballot(has && before + sum > share);
        if (past) {
            const uint32_t who = uint32_t(__builtin_ctzll(past));
            piece = k0 + who;
            if (who) before += of_lane(sum, who - 1u);
            found = true;
        } else {
            before += of_lane(sum, kWave - 1);
        }
    };
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i)
        if (!found) look(i * kWave, ahead[i], some[i]);
#pragma unroll 1
    for (uint32_t k0 = kAhead * kWave; k0 < p.pieces && !found; k0 += kWave) {
        const double own = weight(k0 + lane);
        look(k0, scan_of<Sum>(own), own > 0.0);
    }
    weights_of<E>(p, f, t, piece, w);
    uint32_t last = 0;
#pragma unroll
    for (uint32_t g = 0; g < kPerLane / W; ++g) {
        double own = 0.0;
#pragma unroll
        for (uint32_t j = 0; j < W; ++j) {
            own += w[g * W + j];
            if (w[g * W + j] > 0.0) last = index_of<W>(piece, g * W + j);
        }
        const double sum = scan_of<Sum>(own);
        const uint64_t past = __ballot(own > 0.0 && before + sum > share);
        if (past) {
            double at = before + shifted<0x138, 0xf>(sum, 0.0);  // of the lanes below
            uint32_t token = last;  // (of this lane: its last with any weight)
            bool here = false;
#pragma unroll
            for (uint32_t j = 0; j < W; ++j) {
                at += w[g * W + j];
                if (!here && at > share && w[g * W + j] > 0.0) token = index_of<W>(piece, g * W + j), here = true;
            }
            return int64_t(of_lane(token, uint32_t(__builtin_ctzll(past))));
        }
        before += of_lane(sum, kWave - 1);
    }
    // (0 for lanes without any)
    return int64_t(~over_wave<Least>(~last));
}

template <typename E, bool Decided>
__global__ __launch_bounds__(Decided ? kWave : kDecideThreads) void token_kernel(VerifyArgs p) {
    const dfc_verify_args &a = p.a;
    const uint32_t r = blockIdx.x;
    Found f;
    if constexpr (Decided) {
        f = p.found[r];
    } else {
        __shared__ Decision lds;
        f = decide<E>(p, r, lds);
        if (threadIdx.x >= kWave) return;
    }
    int64_t token = -1;
    if (f.mode == kGreedy) {
        token = f.drafted;
    } else if (f.mode != kNone) {
        uint32_t unused = 0;
        const Rows rows = rows_of(a, r, unused);
        token = draw<E>(p, f, r, a.uniforms[rows.first + rows.count - 1u]);
    }
    if (threadIdx.x == 0) {
        a.accepted[r] = int32_t(f.accepted);
        a.tokens[r] = token;
        if (f.bad && a.status_dev) atomicOr(a.status_dev, f.bad);
    }
}

uint32_t pieces_of(const dfc_verify_args &a) { return uint32_t(dfc::ceil_div(uint64_t(a.vocab), uint64_t(kPiece))); }
uint32_t groups_of(const dfc_verify_args &a) { return uint32_t(dfc::ceil_div(uint64_t(pieces_of(a)), uint64_t(kVWaves))); }

uint64_t workspace_of(const dfc_verify_args &a) {
    const uint64_t pieces = pieces_of(a), parts = a.rows * pieces * sizeof(Part);
    uint64_t bytes = parts;
    if (a.draft_logits_dev)
        bytes += parts + uint64_t(a.n_requests) * (sizeof(Found) + ((pieces * sizeof(double) + 15u) & ~uint64_t(15)));
    return bytes;
}

dfc_status check_verify(const dfc_verify_args &a) {
    if (a.dtype != DFC_F32 && a.dtype != DFC_BF16 && a.dtype != DFC_F16) return DFC_EUNSUPPORTED;
    if (!a.vocab || a.vocab > (1u << 30) || a.n_requests > kMostRequests || a.rows > kMostGroups) return DFC_EUNSUPPORTED;
    const uint64_t rows = std::max<uint64_t>(a.draft_logits_dev ? 2u * a.rows : a.rows, a.n_requests);
    return rows * groups_of(a) > kMostGroups ? DFC_EUNSUPPORTED : DFC_OK;
}

template <typename E>
dfc_status launch_verify(const VerifyArgs &p, hipStream_t st) {
    const dfc_verify_args &a = p.a;
    const uint64_t rows = a.rows * (a.draft_logits_dev ? 2u : 1u);
    const uint64_t parts = rows * p.groups, rests = uint64_t(a.n_requests) * p.groups;
    if (parts) hipLaunchKernelGGL((parts_kernel<E>), dim3(uint32_t(parts)), dim3(kVThreads), 0, st, p);
    if (a.draft_logits_dev) {
        hipLaunchKernelGGL((decide_kernel<E>), dim3(a.n_requests), dim3(kDecideThreads), 0, st, p);
        hipLaunchKernelGGL((rest_kernel<E>), dim3(uint32_t(rests)), dim3(kVThreads), 0, st, p);
        hipLaunchKernelGGL((token_kernel<E, true>), dim3(a.n_requests), dim3(kWave), 0, st, p);
    } else {
        hipLaunchKernelGGL((token_kernel<E, false>), dim3(a.n_requests), dim3(kDecideThreads), 0, st, p);
    }
    return hipGetLastError() == hipSuccess ? DFC_OK : DFC_EHIP;
}

}  // namespace

extern "C" {

dfc_status dfc_verify_workspace(const dfc_verify_args *args, uint64_t *bytes) {
    if (!args || !bytes) return DFC_EINVAL;
    const dfc_status s = check_verify(*args);
    if (s != DFC_OK) return s;
    *bytes = workspace_of(*args);
    return DFC_OK;
}

dfc_status dfc_verify_drafts(const dfc_verify_args *args, void *stream) {
    if (!args) return DFC_EINVAL;
    const dfc_verify_args &a = *args;
    const dfc_status s = check_verify(a);
    if (s != DFC_OK) return s;
    if (!a.n_requests) return DFC_OK;
    if (!a.cu_rows || !a.accepted || !a.tokens) return DFC_EINVAL;
    if (a.rows && (!a.logits_dev || !a.drafts || !a.uniforms)) return DFC_EINVAL;
    if (!a.workspace_dev && workspace_of(a)) return DFC_EINVAL;
    if (a.logits_stride < int64_t(a.vocab) || (a.draft_logits_dev && a.draft_stride < int64_t(a.vocab))) return DFC_EINVAL;
    if (reinterpret_cast<uintptr_t>(a.workspace_dev) & 255u) return DFC_EINVAL;
    if (a.workspace_bytes < workspace_of(a)) return DFC_ESIZE;
    VerifyArgs p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    p.pieces = pieces_of(a);
    p.groups = groups_of(a);
    uint8_t *work = static_cast<uint8_t *>(a.workspace_dev);
    const uint64_t parts = a.rows * p.pieces * sizeof(Part);
    p.target = reinterpret_cast<Part *>(work);
    if (a.draft_logits_dev) {
        p.draft = reinterpret_cast<Part *>(work + parts);
        p.found = reinterpret_cast<Found *>(work + 2 * parts);
        p.rest = reinterpret_cast<double *>(work + 2 * parts + uint64_t(a.n_requests) * sizeof(Found));
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    switch (a.dtype) {
        case DFC_F32: return launch_verify<float>(p, st);
        case DFC_BF16: return launch_verify<__bf16>(p, st);
        default: return launch_verify<_Float16>(p, st);
    }
}

}  // extern "C"
