// route_scores.cu -- from a token's router scores to its k experts, and back.
//
//   s    softmax of the token's logits over all experts, or their sigmoids
//   key  s + bias[e]; without a bias the experts keep the order of the logits
//   choice  the groups of experts with the best scores stay (a group's score is
//        its largest key or the sum of its two largest), and of their experts
//        the k with the largest keys, ties to the lower index
//   w_j  scale * s_j, divided by the sum over the chosen if renormalised
//   losses  balance = E / (k T) sum_e count_e mean_t p[t, e] with p the scores
//        divided by their sum, and z = mean_t (log sum_e exp(logit))^2
//
// One warp takes a token; lane l holds the V = 1, 2, 4 or 8 experts from l V on,
// so that a token is read with vector loads and the lower lane has the lower
// index.  The largest key of a warp is one redux.sync on keys mapped to unsigned
// integers of the same order.
//
// The choice is that of exact keys.  Those of fp32 are off by a few units of the
// last place, so where two that matter (neighbours among the k + 1 largest, the k-th
// and any behind it, the last kept group and the first dropped) are closer than their
// error allows, keys of fp64 decide, of the experts whose fp32 keys leave it open.
// Experts of the same logit and the same bias have the same key in either and need no
// second look; what lies behind such a pair at the last place does.  exp of fp64
// takes a warp 2000 cycles and a division 1600: 20 to 30 tokens of 32768 have such
// neighbours, and with the keys of all 256 experts in fp64 each of them held its block for
// 37 thousand, 15 to 28 us at the end of a batch.
//
// What bounds it: instructions, where there are many tokens.  32768 x 256 fp32 logits, 8
// chosen of 4 of 8 groups by sigmoids with a bias: 50 us (5 us of bytes), with the losses
// 63, without bias and groups 35, tokens of one value 62 (with groups 640: the groups are
// too close in fp32 and all take fp64).  The gradient: 33 us with losses, 21 without (10 us
// of bytes).  These are events around a single call, whose launch and end count; calls back
// to back overlap, 60 us with the losses and 30 for their gradient.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxChoices = 8;
constexpr int kWarps = 8;          // per block
constexpr int kPerSm = 3;          // blocks; a warp's set-up is shared by a dozen tokens (4 spill: 72 us where 3 take 63)
constexpr int kPerSmBwd = 4;       // of the gradient, which waits more than it computes (3: 25 us where 4 take 21)
constexpr int kLossBlocks = 512;   // at most, where loads and losses are summed
constexpr int kLossColumns = 8;    // experts per block of the second kernel
constexpr int kLossThreads = 1024; // of it (256 take 1 us more)

struct ScoreArgs {
    const void* logits;
    int64_t ld, T;
    int32_t E, k, n_groups, topk_groups, group_top;
    int32_t sigmoid, renormalize;
    float scale;
    int32_t wide;         // rows of logits may be read V elements at a time
    const float* bias;    // [E] or null
    int32_t* idx;         // [T, k]
    float* w;             // [T, k]
    // loads and losses
    float* share;         // [blocks, E] sums of p
    int32_t* load;        // [blocks, E]
    float* z;             // [blocks]
    uint32_t* ticket;     // [1], cleared by the first kernel
    float* part;          // [E / 8] balance sums of the second kernel's blocks
    int32_t* counts;      // [E]
    float* losses;        // [2]
    int32_t blocks;
    // gradient
    const float* dw;      // [T, k] or null
    const float* dlosses; // [2] or null
    float per_count;      // E / (k T^2)
    void* dlogits;
    int64_t ldd;
    int32_t wide_out;
};


// ------------------------------------------------------------------- keys --
// Unsigned integers in the order of the keys, which are numbers or -infinity; 0 for
// what may not be chosen.  -infinity, chosen only when nothing else is left, comes
// just below the numbers.
constexpr uint32_t kDead = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float f) {
    const int b = __float_as_int(f + 0.0f);  // -0 and 0 are one key
    return static_cast<uint32_t>(b ^ (b >> 31 | static_cast<int>(0x80000000u)));
}
__device__ __forceinline__ uint64_t key_of(double f) {
    const long long b = __double_as_longlong(f + 0.0);
    return static_cast<uint64_t>(b ^ (b >> 63 | static_cast<long long>(0x8000000000000000ull)));
}
__device__ __forceinline__ float number_of(uint32_t u) {
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ float warp_maxf(float v) {  // -infinity for a warp without numbers
    return number_of(warp_max(key_of(v)));
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float sum8(float v) {  // of lanes 0 .. 7, in them
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// ---------------------------------------------------------------- logits --
template <typename T>
__device__ __forceinline__ float as_float(T v) { return to_float<T>(v); }
template <>
__device__ __forceinline__ float as_float(float v) { return v; }

template <int BYTES>
__device__ __forceinline__ void load_bytes(const void* p, uint32_t (&r)[(BYTES + 3) / 4]) {
    if constexpr (BYTES == 32) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    } else if constexpr (BYTES == 16) {
        const uint4 v = ld_dep(static_cast<const uint4*>(p));
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = ld_dep(static_cast<const uint2*>(p));
        r[0] = v.x, r[1] = v.y;
    } else if constexpr (BYTES == 4) {
        r[0] = ld_dep(static_cast<const uint32_t*>(p));
    } else {
        r[0] = ld_dep(static_cast<const uint16_t*>(p));
    }
}
template <int BYTES>
__device__ __forceinline__ void store_bytes(void* p, const uint32_t (&r)[(BYTES + 3) / 4]) {
    if constexpr (BYTES == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else if constexpr (BYTES == 16) {
        *static_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    } else if constexpr (BYTES == 8) {
        *static_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    } else if constexpr (BYTES == 4) {
        *static_cast<uint32_t*>(p) = r[0];
    } else {
        *static_cast<uint16_t*>(p) = static_cast<uint16_t>(r[0]);
    }
}

// The lane's V logits of token t as they lie in memory, and as they are taken:
// -infinity for NaN, for -infinity and past E, +infinity as the largest finite number.
template <typename T, int V>
struct Raw {
    uint32_t r[(V * sizeof(T) + 3) / 4];
    __device__ __forceinline__ void load(const ScoreArgs& a, int64_t t, int lane, bool wide) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld + lane * V;
        if (wide) {
            if (lane * V < a.E) load_bytes<V * sizeof(T)>(row, r);
        } else {
            T v[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < a.E) v[i] = ld_dep(row + i);
            memcpy(r, v, sizeof v);
        }
    }
    __device__ __forceinline__ void take(const ScoreArgs& a, int lane, float (&l)[V]) const {
        T v[V];
        memcpy(v, r, sizeof v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float f = lane * V + i < a.E ? as_float<T>(v[i]) : -INFINITY;
            l[i] = f > -INFINITY ? fminf(f, FLT_MAX) : -INFINITY;
        }
    }
};
// Biases as keys take them: NaN as -infinity, +infinity as the largest number.
__device__ __forceinline__ float tame(float b) { return b > -INFINITY ? fminf(b, FLT_MAX) : -INFINITY; }

// Value i of the lane that has expert e = lane * V + i, in a lane that asks for e.
template <int V>
__device__ __forceinline__ float value_of(const float (&l)[V], int e) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = __shfl_sync(kAll, l[i], e / V);
        r = e % V == i ? v : r;
    }
    return r;
}

// ---------------------------------------------------------------- choice --
// Which groups stay, as a bit mask, from the experts' keys; *close: the last kept
// score and the first dropped are within tol of one another.  buf holds a warp's
// 32 V keys.
template <int V, typename F>
__device__ __forceinline__ uint32_t kept_groups(const ScoreArgs& a, int gsz, int lane, const F (&key)[V], F* buf, F tol,
                                                bool* close) {
    F b1 = -INFINITY, b2 = -INFINITY;  // of group `lane`
    const int q = gsz / V;
    if (q > 0 && q * V == gsz && (q & (q - 1)) == 0) {  // a group is q whole lanes
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
        }
        for (int o = 1; o < q; o <<= 1) {
            const F o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            b2 = max(min(b1, o1), max(b2, o2));
            b1 = max(b1, o1);
        }
        b1 = __shfl_sync(kAll, b1, lane * q);  // past the last group: unused
        b2 = __shfl_sync(kAll, b2, lane * q);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) buf[lane * V + i] = key[i];
        __syncwarp();
        if (lane < a.n_groups)
            for (int e = lane * gsz; e < (lane + 1) * gsz; ++e) {
                b2 = max(b2, min(b1, buf[e]));
                b1 = max(b1, buf[e]);
            }
        __syncwarp();
    }
    // of fp32 keys half the sum, which stays a number
    const F part = a.group_top == 2 && sizeof(F) == 4 ? 0.5 : 1.0;
    const F score = a.group_top == 2 && b2 > -INFINITY ? part * b1 + part * b2 : part * b1;
    const auto u = lane < a.n_groups ? key_of(score) : 0;
    int rank = 0;  // groups before this one
#pragma unroll 4
    for (int g = 0; g < a.n_groups; ++g) rank += __shfl_sync(kAll, u, g) + (g < lane) > u;  // ties to the lower group
    const uint32_t kept = __ballot_sync(kAll, lane < a.n_groups && rank < a.topk_groups);
    *close = false;
    if (a.topk_groups < a.n_groups) {
        const int last = __ffs(__ballot_sync(kAll, lane < a.n_groups && rank == a.topk_groups - 1)) - 1;
        const int first = __ffs(__ballot_sync(kAll, lane < a.n_groups && rank == a.topk_groups)) - 1;
        const F lo = __shfl_sync(kAll, score, first), hi = __shfl_sync(kAll, score, last);
        *close = lo > -INFINITY && hi - lo <= part * tol;
    }
    return kept;
}

// The k + 1 largest keys of the experts that may be chosen: lane r gets the r-th
// and its expert (key 0 where there is none).
template <int V, typename U>
__device__ __forceinline__ void largest(int k, int lane, U (&u)[V], U& my_key, int& my_expert) {
    my_key = 0;
    my_expert = 0;
    for (int r = 0; r <= k; ++r) {
        U best = 0;
        int slot = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (u[i] >= best) {
                best = u[i];
                slot = i;
            }
        const U m = warp_max(best);
        const int owner = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = __shfl_sync(kAll, slot, owner) + owner * V;
        if (lane == r) {
            my_key = m;
            my_expert = e;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane == owner && slot == i) u[i] = 0;
    }
}

// V words of a lane in shared memory, aligned to them all
template <int V>
__device__ __forceinline__ void put_words(uint32_t* p, const uint32_t (&v)[V]) {
    if constexpr (V == 1) {
        p[0] = v[0];
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<uint4*>(p + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
template <int V>
__device__ __forceinline__ void get_words(const uint32_t* p, uint32_t (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = p[0];
    } else if constexpr (V == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        v[0] = u.x, v[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(p + i);
            v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
        }
    }
}

// A lane's expert among a token's k + 1 largest keys, and how many come before it; no
// expert: rank above k.
struct Pick {
    int rank, expert;
    uint32_t key;
    float logit;
};

// The same choice in parallel: the (k + 1)-th largest of the lanes' own largest keys is
// no larger than the (k + 1)-th key of all, so that what is not below it, a dozen
// experts as a rule, holds all that is looked for, and all that is within `margin` of it
// where that is taken off; these are dealt to the lanes and count who comes before them.
// False where they are more than the lanes (many ties, or few lanes with experts that may
// be chosen).  buf: the warp's 32 V logits, 32 V keys and 32 experts; floor_: the bound.
template <int V>
__device__ __forceinline__ bool largest_in_parallel(int k, int lane, const uint32_t (&u)[V], const float (&l)[V],
                                                    float margin, uint32_t* buf, Pick& mine, uint32_t& floor_) {
    uint32_t best = u[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, u[i]);
    floor_ = 1;
    for (int n = 0; n <= k;) {
        const uint32_t m = warp_max(best);
        if (m == 0) {  // every expert that may be chosen is looked at
            floor_ = 1;
            break;
        }
        floor_ = m;
        n += __popc(__ballot_sync(kAll, best == m));
        best = best == m ? 0u : best;
    }
    if (margin > 0.0f && floor_ > kDead) floor_ = key_of(number_of(floor_) - margin);
    // in ascending order of the lane, and in a lane of the slot: of the expert
    int count = 0, before = 0;
    uint8_t* list = reinterpret_cast<uint8_t*>(buf + 64 * V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t at = __ballot_sync(kAll, u[i] >= floor_);
        count += __popc(at);
        before += __popc(at & ((1u << lane) - 1u));
    }
    if (count > 32) return false;
    uint32_t bits[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bits[i] = __float_as_uint(l[i]);
        if (u[i] >= floor_) list[before++] = static_cast<uint8_t>(lane * V + i);
    }
    put_words<V>(buf + lane * V, bits);
    put_words<V>(buf + 32 * V + lane * V, u);
    __syncwarp();
    mine.expert = lane < count ? list[lane] : 0;
    mine.key = lane < count ? buf[32 * V + mine.expert] : 0u;
    mine.logit = __uint_as_float(buf[mine.expert]);
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) rank += __shfl_sync(kAll, mine.key, j) + (j < lane) > mine.key;  // ties to the lower expert
    mine.rank = lane < count ? rank : 32;
    __syncwarp();
    return true;
}

// Whether the error of two fp32 keys, the first no smaller, may hide their order; off: that
// of their scores' difference.  The sums with the biases add half a unit of each.
__device__ __forceinline__ bool too_close(float f0, float f1, float off) {
    return f0 - f1 <= off + 0x1p-23f * fmaxf(fabsf(f0), fabsf(f1));
}

// Whether two experts have equal keys in any precision.
__device__ __forceinline__ bool same_key(const ScoreArgs& a, float l0, int e0, float l1, int e1) {
    return l0 == l1 && (!a.bias || tame(ld_dep(a.bias + e0)) == tame(ld_dep(a.bias + e1)));
}

// The choice of token t with keys of fp64 of all experts; lane r gets the r-th.  For
// softmaxes, whose sum needs all of them, and where more experts than lanes are too close.
template <typename T, int V>
__device__ __noinline__ int choose_exact(const ScoreArgs& a, int64_t t, double* buf) {
    const int lane = threadIdx.x & 31;
    float l[V];
    Raw<T, V> raw;
    raw.load(a, t, lane, false);
    raw.take(a, lane, l);
    double key[V], pick[V];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = warp_maxf(top);
    double sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double x = l[i];
        key[i] = !(l[i] > -INFINITY) ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top);
        sum += key[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (!a.sigmoid) key[i] /= sum;
        if (a.bias && e < a.E) key[i] += static_cast<double>(tame(ld_dep(a.bias + e)));
        if (!(l[i] > -INFINITY)) key[i] = -INFINITY;
        pick[i] = a.bias ? key[i] : static_cast<double>(l[i]);
    }
    uint32_t kept = kAll;
    const int gsz = a.n_groups ? a.E / a.n_groups : a.E;
    if (a.n_groups) {
        bool close;
        if (a.group_top == 1)
            kept = kept_groups<V, double>(a, gsz, lane, pick, buf, 0.0, &close);
        else
            kept = kept_groups<V, double>(a, gsz, lane, key, buf, 0.0, &close);
    }
    uint64_t u[V], my_key;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        u[i] = e < a.E && (kept >> (e / gsz) & 1u) ? key_of(pick[i]) : 0;
    }
    int expert;
    largest<V, uint64_t>(a.k, lane, u, my_key, expert);
    return expert;
}

// The kept groups by keys of fp64, which only the experts have that may be a group's best
// (or two best): the others' fp32 keys are further below than `margin`, their error.  buf: a
// warp's 32 slots fp32 keys, its 32 slots logits, a list of experts; top: the largest logit.
__device__ __noinline__ uint32_t exact_groups(const ScoreArgs& a, uint32_t* buf, int slots, float margin, float top) {
    const int lane = threadIdx.x & 31, gsz = a.E / a.n_groups;
    const float* key = reinterpret_cast<const float*>(buf);
    const float* logit = key + 32 * slots;
    uint8_t* list = reinterpret_cast<uint8_t*>(buf + 64 * slots);
    uint64_t* exact = reinterpret_cast<uint64_t*>(buf);  // of the list's experts, over what has been read
    float f1 = -INFINITY, f2 = -INFINITY;  // of group `lane`
    if (lane < a.n_groups)
#pragma unroll 1
        for (int e = lane * gsz; e < (lane + 1) * gsz; ++e) {
            f2 = fmaxf(f2, fminf(f1, key[e]));
            f1 = fmaxf(f1, key[e]);
        }
    const float least = (a.group_top == 2 ? f2 : f1) - margin;
    int count = 0;
#pragma unroll 1
    for (int base = 0; base < a.E; base += 32) {
        const int e = base + lane;
        const float from = __shfl_sync(kAll, least, e < a.E ? e / gsz : 0);
        const bool need = e < a.E && key[e] > -INFINITY && key[e] >= from;
        const uint32_t at = __ballot_sync(kAll, need);
        if (need) list[count + __popc(at & ((1u << lane) - 1u))] = static_cast<uint8_t>(e);
        count += __popc(at);
    }
    double sum = 0;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32)
            if (logit[e] > -INFINITY) sum += exp(static_cast<double>(logit[e]) - top);
        sum = warp_sum(sum);
    }
    __syncwarp();
    // entry c of the list has expert c or a later one, whose logit lies past where
    // its 32 keys and all before them go
#pragma unroll 1
    for (int c0 = 0; c0 < count; c0 += 32) {
        const int e = list[min(c0 + lane, count - 1)];
        const double x = logit[e];
        __syncwarp();
        const double ex = exp(a.sigmoid ? -x : x - top);
        double v = (a.sigmoid ? 1.0 : ex) / (a.sigmoid ? 1.0 + ex : sum);
        if (a.bias) v += static_cast<double>(tame(ld_dep(a.bias + e)));
        if (c0 + lane < count) exact[c0 + lane] = key_of(v);
        __syncwarp();
    }
    uint64_t b1 = 0, b2 = 0;
#pragma unroll 1
    for (int c = 0; c < count; ++c) {
        const int e = list[c];
        if (e >= lane * gsz && e < (lane + 1) * gsz) {
            const uint64_t u = exact[c];
            b2 = max(b2, min(b1, u));
            b1 = max(b1, u);
        }
    }
    auto number = [](uint64_t u) { return __longlong_as_double(u >> 63 ? u ^ 0x8000000000000000ull : ~u); };
    if (a.group_top == 2 && b2) b1 = key_of(number(b1) + number(b2));
    int rank = 0;  // groups before this one; ties to the lower group
#pragma unroll 1
    for (int g = 0; g < a.n_groups; ++g) rank += __shfl_sync(kAll, b1, g) + (g < lane) > b1;
    __syncwarp();
    return __ballot_sync(kAll, lane < a.n_groups && rank < a.topk_groups);
}

// How many of the experts that `need` be compared come before the lane's, by sigmoids of
// fp64; ties to the lower lane.  Experts without a score (logit -infinity) are among them
// where the k-th key is next to the lowest number, and come last as they do in fp32.
__device__ __noinline__ int exact_rank(float logit, float bias, bool need) {
    const int lane = threadIdx.x & 31;
    double v = 1.0 / (1.0 + exp(-static_cast<double>(logit))) + static_cast<double>(bias);
    if (!(logit > -INFINITY)) v = -INFINITY;
    const uint64_t u = need ? key_of(v) : 0;
    int rank = 0;
#pragma unroll 1
    for (uint32_t m = __ballot_sync(kAll, need); m; m &= m - 1) {
        const int j = __ffs(m) - 1;
        rank += __shfl_sync(kAll, u, j) + (j < lane) > u;
    }
    return rank;
}

// exp and 1 / x for what is compared, and for sums of all experts (of losses, of gradients
// and under plain softmax weights, which are off by 5.6e-8 of themselves in the mean; with
// expf there 5.2e-8, and 32768 x 256 take 2 us more): off by 2 and 1 units of the last
// place, and exp by its rounded argument.
__device__ __forceinline__ float exp_fast(float x) { return __expf(x); }
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x / y for the weights, y from 1/2 to 16: the approximate quotient q and what is left of x, in
// y's, so that of 2^n equal scores each has 2^-n to the bit.  (Renormalised sigmoids are off by
// 4.3e-8 in the mean; with x * rcp_fast(y) by 5.3e-8, with divisions by 4.3e-8 and 32768 x 256
// take 2 us more.)
__device__ __forceinline__ float quotient(float x, float y) {
    const float r = rcp_fast(y), q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// 1 / (1 + exp(-x)) = pos or neg by the sign, from e = exp(-|x|): the score and
// one minus the score without cancellation.
struct Sigmoid {
    float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float x) {
    const float e = expf(-fabsf(x)), d = 1.0f / (1.0f + e), ed = e * d;
    return x >= 0.0f ? Sigmoid{d, ed} : Sigmoid{ed, d};
}
__device__ __forceinline__ Sigmoid sigmoid_fast(float x) {
    const float e = exp_fast(-fabsf(x)), d = rcp_fast(1.0f + e), ed = e * d;
    return x >= 0.0f ? Sigmoid{d, ed} : Sigmoid{ed, d};
}
// Scores of one token over their sum: sigmoids times exp(-m), m = min(0, largest
// logit), so that none of a token's underflow together.
__device__ __forceinline__ float shifted_sigmoid(float x, float m) {
    if (!(x > -INFINITY)) return 0.0f;
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - m) / (1.0f + expf(x));
}
// The part of this lane's expert (logit lx; -infinity or not one of the chosen: none) in
// the scores of the chosen, k lanes of the warp.
__device__ __forceinline__ float chosen_share(const ScoreArgs& a, float lx) {
    const float top = warp_maxf(lx);
    float v = 0.0f;
    if (a.sigmoid) {
        if (top >= 0.0f) {
            const float e = expf(-fabsf(lx)), d = quotient(1.0f, 1.0f + e);
            v = lx >= 0.0f ? d : e * d;  // exp(-infinity) = 0
        } else {
            v = shifted_sigmoid(lx, top);
        }
    } else if (lx > -INFINITY) {
        v = expf(lx - top);
    }
    const float sum = warp_sum(v);
    return sum > 0.0f ? quotient(v, sum) : 0.0f;  // a sum is from 1/2 to 8, its largest part from 1/2 to 1
}

template <typename T, int V, bool LOSS>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) k_route_scores(const __grid_constant__ ScoreArgs a) {
    constexpr int W = kWarps;
    __shared__ __align__(32) double s_buf[W][32 * V + 32];  // 32 V keys of fp64 or logits and keys, and a list of experts
    __shared__ __align__(32) float s_bias[32 * V];
    __shared__ __align__(32) uint32_t s_group[32 * V];  // the bit of an expert's group
    __shared__ int s_load[LOSS ? 32 * V : 1];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gsz = a.n_groups ? a.E / a.n_groups : a.E;
    const bool grouped = a.n_groups > 0;
    const bool by_score = a.bias || (grouped && a.group_top == 2);  // keys need scores
    const bool soft = LOSS || (!a.sigmoid && (by_score || !a.renormalize));  // the softmax is needed
    float share[LOSS ? V : 1], z = 0.0f;
    for (int e = threadIdx.x; e < 32 * V; e += 32 * W) {
        s_bias[e] = a.bias && e < a.E ? tame(ld_dep(a.bias + e)) : 0.0f;
        const int group = e / gsz;
        s_group[e] = !grouped || group < a.n_groups ? 1u << (group & 31) : 0u;
    }
    if constexpr (LOSS) {
#pragma unroll
        for (int i = 0; i < V; ++i) share[i] = 0.0f;
    }
    if constexpr (LOSS) {
        for (int e = threadIdx.x; e < 32 * V; e += 32 * W) s_load[e] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    }
    __syncthreads();
    float most = 0.0f;  // of a key's magnitude
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, s_bias[lane * V + i] > -INFINITY ? fabsf(s_bias[lane * V + i]) : 0.0f);
    most = 1.0f + warp_maxf(most);
    Raw<T, V> raw;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * W + warp, stride = static_cast<int64_t>(gridDim.x) * W;
    if (first < a.T) raw.load(a, first, lane, a.wide);
    for (int64_t t = first; t < a.T; t += stride) {
        float l[V];
        raw.take(a, lane, l);
        if (t + stride < a.T) raw.load(a, t + stride, lane, a.wide);  // the next token's come meanwhile
        float s[V], top = -INFINITY, inv = 0.0f, scores_top = 1.0f;
        if (soft) {  // softmax, and the z loss of either
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
            top = warp_maxf(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = l[i] > -INFINITY ? exp_fast(l[i] - top) : 0.0f;
                sum += s[i];
            }
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            if (LOSS && sum > 0.0f) {
                const float lse = top + logf(sum);
                z = fmaf(lse, lse, z);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] *= inv;
            scores_top = inv;
            if constexpr (LOSS) {
                if (!a.sigmoid) {
#pragma unroll
                    for (int i = 0; i < V; ++i) share[i] += s[i];
                }
            }
        }
        if (a.sigmoid && (LOSS || by_score)) {
            scores_top = 1.0f;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = sigmoid_fast(l[i]).s;
                sum += s[i];
            }
            if constexpr (LOSS) {
                if (top >= 0.0f) {
                    const float f = 1.0f / warp_sum(sum);
#pragma unroll
                    for (int i = 0; i < V; ++i) share[i] = fmaf(s[i], f, share[i]);
                } else {  // small scores, on a common factor
                    float r[V];
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        r[i] = shifted_sigmoid(l[i], top);
                        sum += r[i];
                    }
                    sum = warp_sum(sum);
                    const float f = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) share[i] = fmaf(r[i], f, share[i]);
                }
            }
        }
        // keys: with a bias or a group's two best they are scores, else logits
        float key[V];
        const bool biased = a.bias != nullptr;
        uint32_t words[V];
        get_words<V>(reinterpret_cast<const uint32_t*>(s_bias) + lane * V, words);
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = by_score && l[i] > -INFINITY ? s[i] + __uint_as_float(words[i]) : l[i];
        // What the difference of two fp32 keys may be off by.  A sigmoid: its 1 + e, the
        // reciprocal and an e of at most 1 that is off by 5 units, a quarter of which
        // counts; 4 units of 2^-24 in all.  A softmax: 24 of the largest score's (exp,
        // the sum of 256, the quotient).  The sum with the bias adds half a unit of the key.
        const float off = a.sigmoid ? 0x1p-20f : 0x1p-18f * scores_top;
        bool close = false;
        uint32_t kept = kAll;
        const float margin = 2.0f * off + 0x1p-21f * most;
        if (grouped) {
            bool near_;
            kept = kept_groups<V, float>(a, gsz, lane, key, reinterpret_cast<float*>(s_buf[warp]), margin, &near_);
            if (by_score && near_) {
                uint32_t* buf = reinterpret_cast<uint32_t*>(s_buf[warp]);
#pragma unroll
                for (int i = 0; i < V; ++i) words[i] = __float_as_uint(key[i]);
                put_words<V>(buf + lane * V, words);
#pragma unroll
                for (int i = 0; i < V; ++i) words[i] = __float_as_uint(l[i]);
                put_words<V>(buf + 32 * V + lane * V, words);
                __syncwarp();
                kept = exact_groups(a, buf, V, margin, top);
                __syncwarp();
            }
        }
        // slots past the last expert have -infinity and come after all experts that do
        uint32_t u[V];
        get_words<V>(s_group + lane * V, words);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = kept & words[i] ? key_of(biased ? key[i] : l[i]) : 0u;
        Pick mine;
        uint32_t floor_;
        const bool parallel = largest_in_parallel<V>(a.k, lane, u, l, biased ? margin : 0.0f,
                                                     reinterpret_cast<uint32_t*>(s_buf[warp]), mine, floor_);
        if (!parallel) {
            largest<V, uint32_t>(a.k, lane, u, mine.key, mine.expert);
            mine.rank = lane;
            mine.logit = value_of<V>(l, mine.expert);
            if (biased) {  // the experts behind the k + 1 largest, against the k-th
                const float fk = number_of(__shfl_sync(kAll, mine.key, a.k - 1)), lk = __shfl_sync(kAll, mine.logit, a.k - 1);
                const float bk = s_bias[__shfl_sync(kAll, mine.expert, a.k - 1)];
                bool other = false;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    other |= u[i] > kDead && too_close(fk, number_of(u[i]), off) && !(l[i] == lk && s_bias[lane * V + i] == bk);
                close = __any_sync(kAll, other);
            }
        }
        uint32_t last = 0;  // the k-th largest key
        if (biased) {
            // neighbours in the order of the keys
            uint32_t* order = reinterpret_cast<uint32_t*>(s_buf[warp]);
            if (lane <= a.k) order[lane] = 0;
            __syncwarp();
            if (mine.rank <= a.k) order[mine.rank] = mine.key;
            __syncwarp();
            last = order[a.k - 1];
            const uint32_t next_key = mine.rank < a.k ? order[mine.rank + 1] : 0;
            const bool near_ = next_key > kDead && too_close(number_of(mine.key), number_of(next_key), off);
            if (__any_sync(kAll, near_)) {
                // experts of one logit and one bias have one key in any precision
                uint32_t* lane_of = order + 16;
                if (mine.rank <= a.k) lane_of[mine.rank] = lane;
                __syncwarp();
                const int after = near_ ? static_cast<int>(lane_of[mine.rank + 1]) : lane;
                const float ly = __shfl_sync(kAll, mine.logit, after);
                const int ey = __shfl_sync(kAll, mine.expert, after);
                bool other = near_ && !same_key(a, mine.logit, mine.expert, ly, ey);
                if (parallel) {  // the k-th may have its like behind it, and another expert behind those
                    const int at = static_cast<int>(lane_of[a.k - 1]);
                    const float lk = __shfl_sync(kAll, mine.logit, at);
                    const int ek = __shfl_sync(kAll, mine.expert, at);
                    other |= mine.rank > a.k && mine.rank < 32 && mine.key > kDead &&
                             too_close(number_of(last), number_of(mine.key), off) && !same_key(a, lk, ek, mine.logit, mine.expert);
                }
                close |= __any_sync(kAll, other);
            }
            __syncwarp();
        }
        if (close) {
            // what may be among the k lies no further below the k-th than the error; where the
            // lanes have it all, a key of fp64 each
            const uint32_t from = last > kDead ? key_of(number_of(last) - margin) : 0;
            if (parallel && a.sigmoid && from >= floor_) {
                const bool need = mine.rank < 32 && mine.key >= from;
                const int rank = exact_rank(mine.logit, s_bias[mine.expert], need);
                mine.rank = need ? rank : 32;
            } else {
                mine.expert = choose_exact<T, V>(a, t, s_buf[warp]);
                mine.rank = lane;
                mine.logit = value_of<V>(l, mine.expert);
            }
        }
        const bool chosen = mine.rank < a.k;
        const float lx = chosen ? mine.logit : -INFINITY;
        float w;
        if (a.renormalize) {
            w = chosen_share(a, lx);
        } else {
            w = !(lx > -INFINITY) ? 0.0f : a.sigmoid ? sigmoid(lx).s : expf(lx - top) * inv;
        }
        if (chosen) {
            a.idx[t * a.k + mine.rank] = mine.expert;
            a.w[t * a.k + mine.rank] = w * a.scale;
            if constexpr (LOSS) atomicAdd(&s_load[mine.expert], 1);
        }
    }
    if constexpr (LOSS) {
        // the block's sums, its warps' in their order
        float* part = reinterpret_cast<float*>(s_buf[warp]);
        float* zs = reinterpret_cast<float*>(s_buf[0]) + 32 * V;  // past the first warp's sums, in its own buffer
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) part[lane * V + i] = share[i];
        if (lane == 0) zs[warp] = z;
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += 32 * W) {
            float sum = 0.0f;
            for (int j = 0; j < W; ++j) sum += reinterpret_cast<const float*>(s_buf[j])[e];
            a.share[static_cast<int64_t>(blockIdx.x) * a.E + e] = sum;
            a.load[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_load[e];
        }
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int j = 0; j < W; ++j) sum += zs[j];
            a.z[blockIdx.x] = sum;
        }
    }
}

// The blocks' sums to the loads and losses.  A block takes eight experts; the one
// that ends last adds up what the others left, in their order.
__global__ void __launch_bounds__(kLossThreads) k_route_losses(const __grid_constant__ ScoreArgs a) {
    constexpr int kRows = kLossThreads / kLossColumns, W = kLossThreads / 32;
    __shared__ float s_share[W][kLossColumns];
    __shared__ int s_load[W][kLossColumns];
    __shared__ float s_sum[W];
    __shared__ bool s_last;
    pdl_trigger();
    pdl_wait();
    const int c = threadIdx.x % kLossColumns, r = threadIdx.x / kLossColumns, e = blockIdx.x * kLossColumns + c;
    float share = 0.0f;
    int load = 0;
    if (e < a.E)
#pragma unroll 4
        for (int b = r; b < a.blocks; b += kRows) {
            share += ld_dep(a.share + static_cast<int64_t>(b) * a.E + e);
            load += ld_dep(a.load + static_cast<int64_t>(b) * a.E + e);
        }
#pragma unroll
    for (int o = kLossColumns; o < 32; o <<= 1) {
        share += __shfl_xor_sync(kAll, share, o);
        load += __shfl_xor_sync(kAll, load, o);
    }
    if ((threadIdx.x & 31) < kLossColumns) {
        s_share[threadIdx.x >> 5][c] = share;
        s_load[threadIdx.x >> 5][c] = load;
    }
    __syncthreads();
    if (threadIdx.x < kLossColumns) {
        share = 0.0f;
        load = 0;
        for (int i = 0; i < W; ++i) {
            share += s_share[i][c];
            load += s_load[i][c];
        }
        if (e < a.E) a.counts[e] = load;
        // count / (k T) times the mean share
        float v = e < a.E ? static_cast<float>(load) / (static_cast<float>(a.k) * static_cast<float>(a.T)) * share : 0.0f;
#pragma unroll
        for (int o = kLossColumns / 2; o > 0; o >>= 1) v += __shfl_xor_sync((1u << kLossColumns) - 1, v, o);
        if (threadIdx.x == 0) {
            a.part[blockIdx.x] = v;
            __threadfence();
            s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float z = 0.0f;
    for (int b = threadIdx.x; b < a.blocks; b += kLossThreads) z += ld_dep(a.z + b);
    z = warp_sum(z);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = z;
    __syncthreads();
    if (threadIdx.x == 0) {
        float balance = 0.0f;
        for (int b = 0; b < static_cast<int>(gridDim.x); ++b) balance += ld_dep(a.part + b);
        z = 0.0f;
        for (int i = 0; i < W; ++i) z += s_sum[i];
        const float T = static_cast<float>(a.T);
        a.losses[0] = balance * static_cast<float>(a.E) / T;
        a.losses[1] = z / T;
    }
}

// -------------------------------------------------------------- gradient --
// With r the chosen experts' parts of the sum of their scores, d the mean of dw
// under r, p the softmax and D = scale sum_j p_j dw_j:
//   renormalised     dlogit_j  = scale r_j (dw_j - d), times 1 - s_j for sigmoids
//   softmax          dlogit_e  = p_e (scale dw_e - D)
//   sigmoid          dlogit_j  = scale dw_j s_j (1 - s_j)
//   balance          dlogit_e += p_e (c_e - sum p c), times 1 - s_e for sigmoids,
//                    c_e = dbalance E count_e / (k T^2), p the scores over their sum
//   z                dlogit_e += dz (2 / T) lse softmax_e
template <typename T, int V, bool LOSS>
__global__ void __launch_bounds__(32 * kWarps, kPerSmBwd) k_route_scores_bwd(const __grid_constant__ ScoreArgs a) {
    __shared__ __align__(32) float s_add[kWarps][32 * V];
    __shared__ __align__(32) float s_count[LOSS ? 32 * V : 1];  // E / (k T^2) dbalance count
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float c[LOSS ? V : 1], dz = 0.0f;
    if constexpr (LOSS) {
        // by way of shared memory: where every warp reads the counts itself, their few lines
        // are what all wait for (52 us of 32768 x 256 against 33)
        const float f = a.per_count * ld_dep(a.dlosses);
        dz = ld_dep(a.dlosses + 1) * 2.0f / static_cast<float>(a.T);
        for (int e = threadIdx.x; e < 32 * V; e += 32 * kWarps)
            s_count[e] = e < a.E ? f * static_cast<float>(ld_dep(a.counts + e)) : 0.0f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = s_count[lane * V + i];
    }
    const bool soft = LOSS || (!a.sigmoid && !a.renormalize);
    Raw<T, V> raw;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWarps + warp, stride = static_cast<int64_t>(gridDim.x) * kWarps;
    int next_expert = -1;
    float next_dw = 0.0f;
    auto load = [&](int64_t t) {
        raw.load(a, t, lane, a.wide);
        if (a.dw && lane < a.k) {
            next_expert = ld_dep(a.idx + t * a.k + lane);
            next_dw = ld_dep(a.dw + t * a.k + lane);
        }
    };
    if (first < a.T) load(first);
    for (int64_t t = first; t < a.T; t += stride) {
        float l[V], g[V];
        raw.take(a, lane, l);
        int expert = next_expert;
        float dw = next_dw;
        if (t + stride < a.T) load(t + stride);  // the next token's come meanwhile
        const bool known = expert >= 0 && expert < a.E;
        expert = known ? expert : 0;
        float lx = value_of<V>(l, expert);
        lx = known ? lx : -INFINITY;
        dw = lx > -INFINITY ? dw : 0.0f;  // a masked expert has no weight
        float top = -INFINITY, inv = 0.0f, lse = 0.0f, p[V];
        if (soft) {
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
            top = warp_maxf(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = l[i] > -INFINITY ? exp_fast(l[i] - top) : 0.0f;
                sum += p[i];
            }
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            lse = sum > 0.0f ? top + logf(sum) : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] *= inv;
        }
        // what goes to the chosen experts alone, and to all by their softmax
        float mine, all = 0.0f;
        if (a.renormalize) {
            const float r = chosen_share(a, lane < a.k ? lx : -INFINITY);
            const float mean = sum8(r * dw);
            mine = a.scale * r * (dw - mean);
            if (a.sigmoid) mine *= sigmoid(lx).rest;
        } else if (a.sigmoid) {
            const Sigmoid s = sigmoid(lx);
            mine = a.scale * dw * s.s * s.rest;
        } else {
            mine = lx > -INFINITY ? a.scale * dw * (expf(lx - top) * inv) : 0.0f;
            all = -__shfl_sync(kAll, sum8(mine), 0);
        }
        if constexpr (LOSS) {
            all = fmaf(dz, lse, all);
            if (!a.sigmoid) {
                float mean = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) mean = fmaf(p[i], c[i], mean);
                mean = warp_sum(mean);
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = p[i] * (c[i] - mean + all);
            } else {
                float s[V], rest[V], sum = 0.0f, mean = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const Sigmoid v = sigmoid_fast(l[i]);
                    s[i] = v.s;
                    rest[i] = v.rest;
                }
                if (top < 0.0f) {  // small scores, on a common factor
#pragma unroll
                    for (int i = 0; i < V; ++i) s[i] = shifted_sigmoid(l[i], top);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum += s[i];
                    mean = fmaf(s[i], c[i], mean);
                }
                sum = warp_sum(sum);
                mean = warp_sum(mean);
                const float f = sum > 0.0f ? 1.0f / sum : 0.0f;
                mean *= f;
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = fmaf(s[i] * f * rest[i], c[i] - mean, p[i] * all);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = soft ? p[i] * all : 0.0f;
        }
        if (a.dw) {
            const bool adds = known && mine != 0.0f;
            const uint32_t same = __match_any_sync(kAll, adds ? expert : -1 - lane);
            if (__any_sync(kAll, (same & (same - 1)) != 0)) {  // an expert that repeats: one after the other
                for (int j = 0; j < a.k; ++j) {
                    const int e = __shfl_sync(kAll, expert, j);
                    const float v = __shfl_sync(kAll, adds ? mine : 0.0f, j);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (e == lane * V + i) g[i] += v;
                }
            } else {
                float* buf = s_add[warp];
#pragma unroll
                for (int i = 0; i < V; ++i) buf[lane * V + i] = 0.0f;
                __syncwarp();
                if (adds) buf[expert] = mine;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] += buf[lane * V + i];
            }
        }
        T* row = static_cast<T*>(a.dlogits) + t * a.ldd + lane * V;
        T o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 4)
                o[i] = g[i];
            else
                o[i] = from_float<T>(g[i]);
        }
        if (a.wide_out) {
            if (lane * V < a.E) {
                uint32_t r[(V * sizeof(T) + 3) / 4];
                memcpy(r, o, sizeof o);
                store_bytes<V * sizeof(T)>(row, r);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < a.E) row[i] = o[i];
        }
    }
}

// ------------------------------------------------------------------ calls --
int elem_bytes(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
int per_lane(int E) { return E > 128 ? 8 : E > 64 ? 4 : E > 32 ? 2 : 1; }

moe_status_t check_rule(const moe_score_rule_t* r) {
    if (!r) return set_last_error(MOE_ERR_INVALID_ARG, "rule is NULL");
    if (r->E <= 0 || r->k <= 0) return set_last_error(MOE_ERR_INVALID_ARG, "E and k must be > 0");
    if (r->E > 256) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", r->E);
    if (r->k > kMaxChoices) return set_last_error(MOE_ERR_UNSUPPORTED, "k = %d > 8", r->k);
    if (r->k > r->E) return set_last_error(MOE_ERR_INVALID_ARG, "k = %d > E = %d", r->k, r->E);
    if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
        return set_last_error(MOE_ERR_INVALID_ARG, "score = %d is neither softmax (0) nor sigmoid (1)", r->score);
    if (!std::isfinite(r->scale)) return set_last_error(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (r->n_groups < 0) return set_last_error(MOE_ERR_INVALID_ARG, "n_groups < 0");
    if (r->n_groups > 0) {
        if (r->n_groups > 32 || r->E % r->n_groups)
            return set_last_error(MOE_ERR_INVALID_ARG, "n_groups = %d must divide E and be <= 32", r->n_groups);
        if (r->topk_groups <= 0 || r->topk_groups > r->n_groups)
            return set_last_error(MOE_ERR_INVALID_ARG, "topk_groups = %d outside [1, n_groups]", r->topk_groups);
        if (r->topk_groups * (r->E / r->n_groups) < r->k)
            return set_last_error(MOE_ERR_INVALID_ARG, "topk_groups * (E / n_groups) < k");
        if (r->group_top != 1 && r->group_top != 2)
            return set_last_error(MOE_ERR_INVALID_ARG, "group_top = %d is neither 1 nor 2", r->group_top);
    }
    return MOE_OK;
}

moe_status_t check_tokens(const moe_score_rule_t* r, int32_t dtype, int64_t T) {
    const moe_status_t s = check_rule(r);
    if (s != MOE_OK) return s;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_F32)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is none of bf16 (0), f16 (1), f32 (2)", dtype);
    if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "T < 0");
    if (T * r->k > (1ll << 30) || T > (1ll << 30))
        return set_last_error(MOE_ERR_UNSUPPORTED, "T*k too large for 32-bit row indices");
    return MOE_OK;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

moe_status_t check_rows(const void* p, int64_t ld, int32_t dtype, const moe_score_rule_t* r) {
    if (!aligned(p, elem_bytes(dtype)))
        return set_last_error(MOE_ERR_INVALID_ARG, "logits and dlogits must be aligned to their elements");
    if (ld < r->E) return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row");
    return MOE_OK;
}

// Rows that can be read V elements at a time
bool wide_rows(const void* p, int64_t ld, int32_t dtype, int E) {
    const int V = per_lane(E), bytes = V * elem_bytes(dtype);
    return E % V == 0 && aligned(p, bytes) && ld % V == 0;
}

ScoreArgs args_of(const moe_score_rule_t* r, int64_t T) {
    ScoreArgs a{};
    a.T = T;
    a.E = r->E;
    a.k = r->k;
    a.n_groups = r->n_groups;
    a.topk_groups = r->topk_groups;
    a.group_top = r->group_top;
    a.sigmoid = r->score == MOE_SCORE_SIGMOID;
    a.renormalize = r->renormalize != 0;
    a.scale = r->scale;
    return a;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// Blocks of the first kernel where loads and losses are summed: kPerSm per SM, and at
// most as many as the workspace, whose size no GPU decides, holds sums of
int most_blocks(int64_t T) {
    const int64_t need = (T + kWarps - 1) / kWarps;
    return static_cast<int>(need < kLossBlocks ? need : kLossBlocks);
}
int loss_blocks(int64_t T) {
    const int most = most_blocks(T);
    return kPerSm * num_sms() < most ? kPerSm * num_sms() : most;
}

template <typename F>
cudaError_t by_type(int32_t dtype, int E, F&& go) {
    auto lanes = [&](auto t) {
        switch (per_lane(E)) {
            case 1: return go(t, std::integral_constant<int, 1>());
            case 2: return go(t, std::integral_constant<int, 2>());
            case 4: return go(t, std::integral_constant<int, 4>());
            default: return go(t, std::integral_constant<int, 8>());
        }
    };
    if (dtype == MOE_DTYPE_F32) return lanes(float());
    return dtype == MOE_DTYPE_BF16 ? lanes(__nv_bfloat16()) : lanes(__half());
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_scores_workspace_size(const moe_score_rule_t* rule, int64_t T) {
    if (check_tokens(rule, MOE_DTYPE_F32, T) != MOE_OK) return 0;
    const size_t blocks = most_blocks(T);
    return 2 * up(blocks * rule->E * 4) + up(blocks * 4) + 256;
}

extern "C" moe_status_t moe_route_scores(const moe_score_rule_t* rule, int32_t dtype, int64_t T, const void* logits,
                                         int64_t ld, const float* bias, int32_t* topk_idx, float* topk_w,
                                         int32_t* counts, float* losses, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t s = check_tokens(rule, dtype, T);
    if (s != MOE_OK) return s;
    if (!counts != !losses) return set_last_error(MOE_ERR_INVALID_ARG, "counts and losses come together");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (T == 0) {
        if (counts) {
            e = cudaMemsetAsync(counts, 0, static_cast<size_t>(rule->E) * 4, st);
            if (e == cudaSuccess) e = cudaMemsetAsync(losses, 0, 8, st);
        }
        return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "routing by scores: %s", cudaGetErrorString(e));
    }
    if (!logits || !topk_idx || !topk_w) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    s = check_rows(logits, ld, dtype, rule);
    if (s != MOE_OK) return s;
    ScoreArgs a = args_of(rule, T);
    a.logits = logits;
    a.ld = ld;
    a.wide = wide_rows(logits, ld, dtype, rule->E);
    a.bias = bias;
    a.idx = topk_idx;
    a.w = topk_w;
    if (counts) {
        const size_t need = moe_route_scores_workspace_size(rule, T);
        if (!ws || ws_bytes < need || !aligned(ws, 16))
            return set_last_error(MOE_ERR_WORKSPACE, "loads and losses need a 16-byte aligned workspace of %zu bytes", need);
        char* at = static_cast<char*>(ws);
        const size_t blocks = most_blocks(T), sums = up(blocks * rule->E * 4);
        a.share = reinterpret_cast<float*>(at);
        a.load = reinterpret_cast<int32_t*>(at + sums);
        a.z = reinterpret_cast<float*>(at + 2 * sums);
        a.part = reinterpret_cast<float*>(at + 2 * sums + up(blocks * 4));
        a.ticket = reinterpret_cast<uint32_t*>(a.part + 32);
        a.counts = counts;
        a.losses = losses;
        a.blocks = loss_blocks(T);
    }
    e = by_type(dtype, rule->E, [&](auto t, auto v) {
        using E_ = decltype(t);
        constexpr int V = decltype(v)::value;
        if (counts)
            return launch_pdl(k_route_scores<E_, V, true>, dim3(a.blocks), dim3(32 * kWarps), 0, st, a);
        const int64_t need = (T + kWarps - 1) / kWarps, most = static_cast<int64_t>(kPerSm) * num_sms();
        return launch_pdl(k_route_scores<E_, V, false>, dim3(static_cast<unsigned>(need < most ? need : most)),
                          dim3(32 * kWarps), 0, st, a);
    });
    if (e == cudaSuccess && counts)
        e = launch_pdl(k_route_losses, dim3((rule->E + kLossColumns - 1) / kLossColumns), dim3(kLossThreads), 0, st, a);
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "routing by scores: %s", cudaGetErrorString(e));
}

extern "C" moe_status_t moe_route_scores_bwd(const moe_score_rule_t* rule, int32_t dtype, int64_t T, const void* logits,
                                             int64_t ld, const int32_t* topk_idx, const float* dw, const int32_t* counts,
                                             const float* dlosses, void* dlogits, int64_t ldd, void* stream) {
    moe_status_t s = check_tokens(rule, dtype, T);
    if (s != MOE_OK) return s;
    if (!counts != !dlosses) return set_last_error(MOE_ERR_INVALID_ARG, "counts and dlosses come together");
    if (T == 0) return MOE_OK;
    if (!logits || !dlogits || (dw && !topk_idx)) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    s = check_rows(logits, ld, dtype, rule);
    if (s == MOE_OK) s = check_rows(dlogits, ldd, dtype, rule);
    if (s != MOE_OK) return s;
    ScoreArgs a = args_of(rule, T);
    a.logits = logits;
    a.ld = ld;
    a.wide = wide_rows(logits, ld, dtype, rule->E);
    a.idx = const_cast<int32_t*>(topk_idx);
    a.dw = dw;
    a.counts = const_cast<int32_t*>(counts);
    a.per_count = static_cast<float>(rule->E / (static_cast<double>(rule->k) * static_cast<double>(T) * static_cast<double>(T)));
    a.dlosses = dlosses;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.wide_out = wide_rows(dlogits, ldd, dtype, rule->E);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t need = (T + kWarps - 1) / kWarps, most = static_cast<int64_t>(kPerSmBwd) * num_sms();
    const dim3 grid(static_cast<unsigned>(need < most ? need : most));
    const cudaError_t e = by_type(dtype, rule->E, [&](auto t, auto v) {
        using E_ = decltype(t);
        constexpr int V = decltype(v)::value;
        return counts ? launch_pdl(k_route_scores_bwd<E_, V, true>, grid, dim3(32 * kWarps), 0, st, a)
                      : launch_pdl(k_route_scores_bwd<E_, V, false>, grid, dim3(32 * kWarps), 0, st, a);
    });
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "gradient of the scores: %s", cudaGetErrorString(e));
}
