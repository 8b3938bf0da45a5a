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
// 128256.  Exponentials and sums are therefore in 64 bits, where it is one in
// 10^8.
//
// A row is cut into pieces of 1,024 values, one a wavefront and 16 a lane, which
// are read once: their largest, its first index, and the sum of
// exp((z - largest) / T), all without a word to other wavefronts.  Everything
// after that works on a row's few pieces, and on one piece of values for the
// token itself.
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

template <typename F>
__device__ __forceinline__ auto over_wave(decltype(F::id()) x) {
#pragma unroll
    for (int d = 32; d; d /= 2) x = F::of(x, __shfl_xor(x, d));
    return x;
}
struct Largest {
    static __device__ float id() { return 0.0f; }
    static __device__ float of(float a, float b) { return fmaxf(a, b); }
};
struct Least {
    static __device__ uint32_t id() { return 0u; }
    static __device__ uint32_t of(uint32_t a, uint32_t b) { return min(a, b); }
};
struct Sum {
    static __device__ double id() { return 0.0; }
    static __device__ double of(double a, double b) { return a + b; }
};

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

// A lane's 16 values of a piece of a row; -inf past the row.
template <typename E>
__device__ __forceinline__ void load_piece(const E *row, uint32_t vocab, uint32_t piece, float (&x)[kPerLane]) {
    constexpr uint32_t W = 16u / sizeof(E);
    using V = __attribute__((ext_vector_type(W))) E;
    const bool whole = (uint64_t(piece) + 1u) * kPiece <= vocab;
    if (whole && (reinterpret_cast<uintptr_t>(row) & 15u) == 0) {
#pragma unroll
        for (uint32_t k = 0; k < kPerLane / W; ++k) {
            const V v = *reinterpret_cast<const V *>(row + index_of<W>(piece, k * W));
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
    float top = -INFINITY;
    bool odd = false;
#pragma unroll
    for (uint32_t i = 0; i < kPerLane; ++i) {
        top = fmaxf(top, x[i]);
        odd |= !(x[i] < INFINITY);
    }
    top = over_wave<Largest>(top);
    Part p{top, 0u, 0.0};
    if (__any(odd)) {
        p.top = __builtin_nanf("");
    } else if (t == 0.0f) {
        uint32_t at = ~0u;
#pragma unroll
        for (uint32_t i = kPerLane; i-- > 0;)
            if (x[i] == top) at = index_of<W>(piece, i);
        p.at = over_wave<Least>(at);
    } else if (top > -INFINITY) {
        const double inv = 1.0 / double(t);
        double s = 0.0;
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i) s += exp((double(x[i]) - double(top)) * inv);
        p.sum = over_wave<Sum>(s);
    }
    return p;
}

// The pieces of the model's rows, and behind them of the drafter's.
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
    float top;
    uint32_t at;
    double sum;  // of exp((z - top) / T)
    bool ok;     // the row has probabilities
};
__device__ __forceinline__ Whole whole_of(const Part *parts, uint32_t pieces, float t) {
    const uint32_t lane = threadIdx.x % kWave;
    const double inv = t > 0.0f ? 1.0 / double(t) : 0.0;
    float top = -INFINITY;
    uint32_t at = ~0u;
    double sum = 0.0;
    bool odd = false;
    for (uint32_t k = lane; k < pieces; k += kWave) {
        const Part x = parts[k];
        odd |= !(x.top < INFINITY);
        // pieces come in the order of their indexes: a later one has to be larger
        if (x.top > top) {
            sum = sum > 0.0 ? sum * exp((double(top) - double(x.top)) * inv) : 0.0;
            top = x.top;
            at = x.at;
        }
        if (x.sum > 0.0) sum += x.sum * exp((double(x.top) - double(top)) * inv);
    }
    Whole w;
    w.top = over_wave<Largest>(top);
    w.at = over_wave<Least>(top == w.top ? at : ~0u);
    w.sum = over_wave<Sum>(sum > 0.0 ? sum * exp((double(top) - double(w.top)) * inv) : 0.0);
    w.ok = !__any(odd) && w.top > -INFINITY;
    return w;
}

// The drafts of a request that hold, and where its next token comes from.
// Called by all wavefronts of a workgroup, which take a row each; `lds` is one
// Found and a word a wavefront.
struct Decision {
    Found f;
    uint32_t refused[kVWaves];
};
template <typename E>
__device__ __forceinline__ Found decide(const VerifyArgs &p, uint32_t r, Decision &lds) {
    const dfc_verify_args &a = p.a;
    const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
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
    const double inv = t > 0.0f ? 1.0 / double(t) : 0.0;
    for (uint32_t i0 = 0; i0 < rows.count; i0 += kVWaves) {
        const uint32_t i = i0 + wave, row = rows.first + i;
        bool stops = false;
        Found f = none;
        if (i < rows.count) {
            f.row = row;
            f.accepted = i;
            const Whole w = whole_of(p.target + uint64_t(row) * p.pieces, p.pieces, t);
            const bool last = i + 1u == rows.count;
            const int64_t x = last ? 0 : a.drafts[row];
            const bool there = x >= 0 && x < int64_t(a.vocab);
            stops = last;
            if (!w.ok) {
                stops = true;
            } else if (t == 0.0f) {
                f.mode = kGreedy;
                f.drafted = int32_t(w.at);
                if (!last) stops = x != int64_t(w.at);
            } else {
                f.mode = kPlain;
                f.p_top = w.top;
                f.p_scale = 1.0 / w.sum;
                if (!last) {
                    auto value = [&](const void *logits, int64_t stride) {
                        return double(float(static_cast<const E *>(logits)[int64_t(row) * stride + (there ? x : 0)]));
                    };
                    const double px = there ? exp((value(a.logits_dev, a.logits_stride) - double(w.top)) * inv) / w.sum : 0.0;
                    double qx = 1.0;
                    if (a.draft_logits_dev) {
                        const Whole v = whole_of(p.draft + uint64_t(row) * p.pieces, p.pieces, t);
                        f.q_top = v.top;
                        f.q_scale = 1.0 / v.sum;
                        if (!v.ok) f.mode = kNone;  // nothing can be drawn against what is not known
                        if (there) qx = exp((value(a.draft_logits_dev, a.draft_stride) - double(v.top)) * inv) / v.sum;
                    }
                    stops = f.mode == kNone || !(double(a.uniforms[row]) * qx < px);
                    if (stops && f.mode == kPlain) {
                        if (a.draft_logits_dev)
                            f.mode = kRest;
                        else if (there)
                            f.drafted = int32_t(x);
                    }
                }
            }
            if (f.mode == kNone || !(last || there)) f.bad |= kStatusCorrupt;
        }
        __syncthreads();  // the ones before have been read
        if (lane == 0) lds.refused[wave] = stops;
        __syncthreads();
        uint32_t who = kVWaves;
#pragma unroll
        for (uint32_t k = kVWaves; k-- > 0;)
            if (lds.refused[k]) who = k;
        if (who == kVWaves) continue;
        if (wave == who && lane == 0) lds.f = f;
        __syncthreads();
        return lds.f;
    }
    return none;
}

// The weights that a token is drawn with: a lane's 16 of a piece.
template <typename E>
__device__ __forceinline__ void weights_of(const VerifyArgs &p, const Found &f, float t, uint32_t piece,
                                           double (&w)[kPerLane]) {
    constexpr uint32_t W = 16u / sizeof(E);
    const dfc_verify_args &a = p.a;
    const double inv = 1.0 / double(t);
    float x[kPerLane];
    load_piece(static_cast<const E *>(a.logits_dev) + int64_t(f.row) * a.logits_stride, a.vocab, piece, x);
    if (f.mode == kRest) {
        float y[kPerLane];
        load_piece(static_cast<const E *>(a.draft_logits_dev) + int64_t(f.row) * a.draft_stride, a.vocab, piece, y);
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i) {
            const double px = f.p_scale * exp((double(x[i]) - double(f.p_top)) * inv);
            const double qx = f.q_scale * exp((double(y[i]) - double(f.q_top)) * inv);
            w[i] = px > qx ? px - qx : 0.0;
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < kPerLane; ++i)
            w[i] = int32_t(index_of<W>(piece, i)) == f.drafted ? 0.0 : exp((double(x[i]) - double(f.p_top)) * inv);
    }
}

// What is left of p where a draft was refused against a drafter's q, summed
// over each piece.  Every workgroup finds out for itself which drafts hold.
template <typename E>
__global__ __launch_bounds__(kVThreads) void rest_kernel(VerifyArgs p) {
    __shared__ Decision lds;
    const dfc_verify_args &a = p.a;
    const uint32_t r = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
    const Found f = decide<E>(p, r, lds);
    if (group == 0 && threadIdx.x == 0) p.found[r] = f;
    const uint32_t piece = group * kVWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (f.mode != kRest || piece >= p.pieces) return;
    double w[kPerLane];
    weights_of<E>(p, f, temperature_of(a, r), piece, w);
    double s = 0.0;
#pragma unroll
    for (uint32_t i = 0; i < kPerLane; ++i) s += w[i];
    s = over_wave<Sum>(s);
    if (threadIdx.x % kWave == 0) p.rest[uint64_t(r) * p.pieces + piece] = s;
}

// Inclusive prefix sum over the wavefront.
__device__ __forceinline__ double scan_of(double x) {
#pragma unroll
    for (uint32_t d = 1; d < kWave; d *= 2) {
        const double y = __shfl_up(x, d);
        if (threadIdx.x % kWave >= d) x += y;
    }
    return x;
}

// The token: first the piece in which the sums pass the random number's share
// of them all, then the value.  The sum of all pieces is the last of the prefix
// sums that are searched, so some piece passes; within it the sums are added in
// another order, and where none passes by a rounding the last value with any
// weight is it.
template <typename E>
__device__ __forceinline__ int64_t draw(const VerifyArgs &p, Found f, uint32_t r, float u) {
    constexpr uint32_t W = 16u / sizeof(E);
    const dfc_verify_args &a = p.a;
    const uint32_t lane = threadIdx.x % kWave;
    const float t = temperature_of(a, r);
    const double inv = 1.0 / double(t);
    const Part *parts = p.target + uint64_t(f.row) * p.pieces;
    double all = 0.0, w[kPerLane];
    double without = 0.0;  // the drafted token's piece without it
    auto weight = [&](uint32_t k) -> double {
        if (k >= p.pieces) return 0.0;
        if (f.mode == kRest) return p.rest[uint64_t(r) * p.pieces + k];
        if (f.drafted >= 0 && uint32_t(f.drafted) / kPiece == k) return without;
        const Part x = parts[k];
        return x.sum > 0.0 ? x.sum * exp((double(x.top) - double(f.p_top)) * inv) : 0.0;
    };
    for (int turn = 0; turn < 2; ++turn) {
        if (f.mode == kPlain && f.drafted >= 0) {
            weights_of<E>(p, f, t, uint32_t(f.drafted) / kPiece, w);
#pragma unroll
            for (uint32_t i = 0; i < kPerLane; ++i) without += w[i];
            without = over_wave<Sum>(without);
        }
        for (uint32_t k0 = 0; k0 < p.pieces; k0 += kWave) all += __shfl(scan_of(weight(k0 + lane)), kWave - 1);
        if (all > 0.0) break;
        f.mode = kPlain;  // nothing is left: of p
        f.drafted = -1;
    }
    u = !(u >= 0.0f) ? 0.0f : fminf(u, 0x1.fffffep-1f);
    const double share = double(u) * all;
    double before = 0.0;
    uint32_t piece = 0;
    for (uint32_t k0 = 0; k0 < p.pieces; k0 += kWave) {
        const double sum = scan_of(weight(k0 + lane));
        const uint64_t past = __ballot(before + sum > share);
        if (past) {
            const uint32_t who = uint32_t(__builtin_ctzll(past));
            piece = k0 + who;
            if (who) before += __shfl(sum, int(who) - 1);
            break;
        }
        before += __shfl(sum, kWave - 1);
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
        const double sum = scan_of(own);
        const uint64_t past = __ballot(before + sum > share);
        if (past) {
            const uint32_t who = uint32_t(__builtin_ctzll(past));
            double at = before + __shfl_up(sum, 1);
            if (lane == 0) at = before;
            uint32_t token = last;  // (of this lane: its last with any weight)
            bool found = false;
#pragma unroll
            for (uint32_t j = 0; j < W; ++j) {
                at += w[g * W + j];
                if (!found && at > share && w[g * W + j] > 0.0) token = index_of<W>(piece, g * W + j), found = true;
            }
            return int64_t(__shfl(token, int(who)));
        }
        before += __shfl(sum, kWave - 1);
    }
#pragma unroll
    for (int d = 32; d; d /= 2) last = max(last, uint32_t(__shfl_xor(int(last), d)));
    return int64_t(last);
}

template <typename E>
__global__ __launch_bounds__(kVThreads) void token_kernel(VerifyArgs p) {
    __shared__ Decision lds;
    const dfc_verify_args &a = p.a;
    const uint32_t r = blockIdx.x;
    const Found f = a.draft_logits_dev ? p.found[r] : decide<E>(p, r, lds);
    if (threadIdx.x >= kWave) return;
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

uint64_t workspace_of(const dfc_verify_args &a) {
    const uint64_t pieces = pieces_of(a), parts = a.rows * pieces * sizeof(Part);
    uint64_t bytes = parts;
    if (a.draft_logits_dev)
        bytes += parts + uint64_t(a.n_requests) * (sizeof(Found) + ((pieces * sizeof(double) + 15u) & ~uint64_t(15)));
    return bytes;
}

dfc_status check_verify(const dfc_verify_args &a) {
    if (a.dtype != DFC_F32 && a.dtype != DFC_BF16 && a.dtype != DFC_F16) return DFC_EUNSUPPORTED;
    if (!a.vocab || a.vocab > (1u << 30) || a.n_requests > kMostRequests || a.rows > 0x3fffffffull) return DFC_EUNSUPPORTED;
    return DFC_OK;
}

template <typename E>
dfc_status launch_verify(const VerifyArgs &p, hipStream_t st) {
    const dfc_verify_args &a = p.a;
    const uint64_t rows = a.rows * (a.draft_logits_dev ? 2u : 1u);
    const uint64_t parts = rows * p.groups, rests = uint64_t(a.n_requests) * p.groups;
    if (parts > 0x7fffffffull || rests > 0x7fffffffull) return DFC_EUNSUPPORTED;
    if (parts) hipLaunchKernelGGL((parts_kernel<E>), dim3(uint32_t(parts)), dim3(kVThreads), 0, st, p);
    if (a.draft_logits_dev) hipLaunchKernelGGL((rest_kernel<E>), dim3(uint32_t(rests)), dim3(kVThreads), 0, st, p);
    hipLaunchKernelGGL((token_kernel<E>), dim3(a.n_requests), dim3(kVThreads), 0, st, p);
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
    if (a.rows && (!a.logits_dev || !a.drafts || !a.uniforms || !a.workspace_dev)) return DFC_EINVAL;
    if (a.logits_stride < int64_t(a.vocab) || (a.draft_logits_dev && a.draft_stride < int64_t(a.vocab))) return DFC_EINVAL;
    if (reinterpret_cast<uintptr_t>(a.workspace_dev) & 255u) return DFC_EINVAL;
    if (a.workspace_bytes < workspace_of(a)) return DFC_ESIZE;
    VerifyArgs p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    p.pieces = pieces_of(a);
    p.groups = uint32_t(dfc::ceil_div(uint64_t(p.pieces), uint64_t(kVWaves)));
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
