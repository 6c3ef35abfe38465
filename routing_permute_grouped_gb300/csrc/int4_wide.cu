// int4_wide.cu -- products of 16-bit rows with 4-bit weights, many rows to a group.
//
//   y[r] = row_scale[r] * x[src[r] / div] W[e]^T   for the rows r of group e
// with W[e][n][k] = (code - zero) * scale, scale and zero per row n and group of
// k.  code - zero is a small integer, exact in 16 bits, so the tensor cores sum a
// group's products as they are, and each group's sum is scaled once, in fp32.
//
// The weights are the MMA's M side: 128 rows of W[e], widened in registers and
// written to tensor memory, from where tcgen05.mma takes its A operand; the token
// rows are its N side (16 to 64 of them, a multiple of 16).  A work item is such a
// panel of weight rows times a tile of token rows; the sum runs over chunks of 256
// elements (128 for groups of 64 and 32).  One CTA of 20 warps per SM:
//   warp 0       TMA of the codes (6 chunks of 16 KB in flight)
//   warps 1, 3   the token rows by cp.async, 80 KB of them in flight, whichever src picks
//   warp 2       issues the MMAs
//   warps 4-11   two warpgroups that take the items in turn: a chunk's sums (one per
//                group of scales) out of tensor memory, scaled and added in registers,
//                one weight row per thread; the epilogue beside the other's sums
//   warps 12-19  widen codes, two warpgroups that take the chunks in turn
//
// What bounds it: not one of these.  32 rows in each of 32 groups of 7168 x 2048 take 104
// us (2.5 TB/s; 39 us of bytes), 64 rows in each of 8 of 4096 x 4096 49 (350 TFLOP/s).
// With seven of eight MMAs, the widening's arithmetic, the sums' or three quarters of the
// token rows' loads left out, the first takes 96, 92, 96 or 100: a chunk is handed on four
// times, and tensor memory holds two of them (512 columns: two widened, two of sums).
// Measured and slower: chunks of 128, four of them in tensor memory (102 to 109); three
// widening warpgroups (108); both summing warpgroups on half of every tile's columns
// (107); sums by packed pairs (110); two issuing warps (115); token rows by 256 elements
// (123) or gathered by TMA; scales of the rows read before the sums (115).
//
// Few items and a long sum: the CTAs of a cluster split the sum; each hands its
// part of every column to the CTA that stores it, which adds the parts in the
// CTAs' order.
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/moe.h"
#include "int4.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kCodeBytes = 96 * 1024;  // of the codes in flight
constexpr int kRowBytes = 80 * 1024;   // of the token rows in flight
constexpr int kRowStages = 16;         // of 128 elements each, at most
constexpr int kThreads = 640;
// Registers per thread of the roles; together no more than the launch's 96 each.  (56,
// 120 and 88 spill in the loaders: 115 us where these take 110.)
constexpr int kIssueRegs = 80, kSumRegs = 120, kWidenRegs = 80;
static_assert(kIssueRegs + 2 * kSumRegs + 2 * kWidenRegs <= 5 * 96, "register split");
constexpr int kMaxSplit = 8;           // CTAs of a cluster

// A chunk's sums are one column per group and token; two chunks' of them and two
// widened chunks (half a column per element) share tensor memory.
template <int G>
struct Cfg {
    static constexpr int chunk = G == 128 ? 256 : 128;   // elements of the sum per step
    static constexpr int parts = chunk / G;              // groups of a chunk
    static constexpr int TN = G == 32 ? 32 : 64;         // token rows of a tile, at most
    static constexpr int d_cols = parts * TN;            // a chunk's sums
    static constexpr int d_bufs = 256 / d_cols;
    static constexpr uint32_t a_col = 256;               // the first widened chunk's column
    static constexpr int a_bufs = 512 / chunk;
    static constexpr int code_stage = 128 * chunk / 2;
    static constexpr int code_stages = kCodeBytes / code_stage;
    static constexpr int join = TN * 512;                // fp32 sums of the columns this CTA stores
    static constexpr int smem = 1024 + kCodeBytes + kRowBytes + join + 1024 + 4 * 260 * 4;
    static_assert(smem <= 232448, "shared memory budget");
    static_assert(d_bufs * d_cols <= 256 && a_bufs * chunk / 2 <= 256, "tensor memory budget");
};

struct Bars {
    uint64_t code_full[12], code_empty[12];
    uint64_t row_full[kRowStages], row_empty[kRowStages];
    uint64_t a_full[4], a_empty[4];
    uint64_t d_full[4], d_empty[4];
    uint64_t join_full[2], join_free[2], summed[2], drain;
    uint32_t tmem, abort;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

// A warp's items first, first + stride, ..: the lanes find 32 of them at a time.
struct Feed {
    Int4Item mine;
    int k = 32;
    __device__ __forceinline__ Int4Item next(const Int4Lists& s, int n_groups, int panels, int total, int t, int stride, int lane) {
        if (k == 32) {
            k = 0;
            const int64_t at = t + static_cast<int64_t>(lane) * stride;
            if (at < total) mine = int4_item(s, n_groups, panels, static_cast<int>(at));
        }
        Int4Item it;
        it.e = __shfl_sync(kAll, mine.e, k);
        it.panel = __shfl_sync(kAll, mine.panel, k);
        it.row = __shfl_sync(kAll, mine.row, k);
        it.rows = __shfl_sync(kAll, mine.rows, k);
        ++k;
        return it;
    }
};

// Stages of token rows that fit beside one another, for tiles of `wide` rows: 16, 10,
// 6 or 5 for 16, 32, 48 or 64
__device__ __forceinline__ int row_stages(int wide) { return min(kRowStages, kRowBytes / (wide * 256)); }

// First weight rows of a panel's two halves of 64.  With SwiGLU the halves are
// gate and up of the same 64 columns (interleaved per 128 in W).
struct Halves {
    int a, b;
};
__device__ __forceinline__ Halves halves_of(int panel, bool swiglu) {
    if (swiglu) {
        const int gate = (panel >> 1) * 256 + (panel & 1) * 64;
        return {gate, gate + 128};
    }
    return {panel * 128, panel * 128 + 64};
}

// Row `me` of the panel among the weight rows; past the last one, the last.
__device__ __forceinline__ int64_t weight_row(const Int4Product& p, int e, const Halves& h, int me) {
    const int n = me < 64 ? h.a + me : h.b + me - 64;
    return static_cast<int64_t>(e) * p.r.N + min(n, p.r.N - 1);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, M = 128, K = 16; by one lane.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A bounded wait of a converged warp.  Many warps wait at a time here, so that the
// hardware is told to suspend them for longer than it would by itself: polling took
// half of the issued instructions.
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort,
                                          uint64_t limit_ns = kWaitLimitNs) {
    const uint32_t at = smem_u32(bar);
    auto once = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(at), "r"(parity), "r"(20000u)
            : "memory");
        return __all_sync(kAll, ok != 0);
    };
    if (once()) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!once()) {
        if (__any_sync(kAll, *abort != 0)) return false;
        if (__any_sync(kAll, globaltimer_ns() - t0 > limit_ns)) return false;
    }
    return true;
}

template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Eight scales (16 bits each) or zero points (8) of a weight row, by the chunk:
// a row's are read eight groups at a time, one read ahead, where they are aligned
// for it, else each by itself, a chunk ahead.
template <int PARTS, typename E>
struct Stream {
    using Eight = std::conditional_t<sizeof(E) == 2, uint4, uint2>;
    const E* at;
    int groups, whole;
    uint32_t absent;
    Eight now, ahead;
    uint32_t one[PARTS];
    __device__ __forceinline__ Eight eight(int g) const {
        Eight v{};
        if (g < groups) v = *reinterpret_cast<const Eight*>(at + g);
        return v;
    }
    __device__ __forceinline__ void single(int c) {
#pragma unroll
        for (int j = 0; j < PARTS; ++j) one[j] = c * PARTS + j < groups ? at[c * PARTS + j] : absent;
    }
    __device__ __forceinline__ void start(const E* row, int n, int aligned, uint32_t none, int c) {
        at = row;
        groups = n;
        whole = aligned;
        absent = none;
        if (!row) return;
        if (whole) {
            now = eight(c * PARTS & ~7);
            ahead = eight((c * PARTS & ~7) + 8);
        } else {
            single(c);
        }
    }
    // Those of chunk c; the chunks follow one another.
    __device__ __forceinline__ void take(int c, uint32_t (&v)[PARTS]) {
        if (!at) {
#pragma unroll
            for (int j = 0; j < PARTS; ++j) v[j] = absent;
        } else if (whole) {
            const uint32_t* w = &now.x;
#pragma unroll
            for (int j = 0; j < PARTS; ++j) {
                const int g = (c * PARTS + j) & 7;
                if constexpr (sizeof(E) == 2) {
                    const uint32_t u = g & 4 ? (g & 2 ? w[3] : w[2]) : (g & 2 ? w[1] : w[0]);
                    v[j] = g & 1 ? u >> 16 : u & 0xFFFFu;
                } else {
                    v[j] = (g & 4 ? w[1] : w[0]) >> (8 * (g & 3)) & 0xFFu;
                }
            }
            if (((c + 1) * PARTS & 7) == 0) {
                now = ahead;
                ahead = eight((c + 1) * PARTS + 8);
            }
        } else {
#pragma unroll
            for (int j = 0; j < PARTS; ++j) v[j] = one[j];
            single(c + 1);
        }
    }
};

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 1)
    k_int4_wide(const __grid_constant__ CUtensorMap tW, const __grid_constant__ Int4Product p) {
    using C = Cfg<G>;
    constexpr int TN = C::TN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* s_rows = smem + kCodeBytes;
    uint8_t* s_join = s_rows + kRowBytes;
    Bars& bars = *reinterpret_cast<Bars*>(s_join + C::join);
    Int4Lists& lists = *reinterpret_cast<Int4Lists*>(reinterpret_cast<uint8_t*>(&bars) + 1024);
    volatile uint32_t* abort_flag = &bars.abort;

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    uint32_t split_;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split_));
    const int split = static_cast<int>(split_);
    const bool swiglu = p.swiglu != 0;
    const int panels = swiglu ? p.columns / 64 : (p.r.N + 127) / 128;
    const int chunks = (p.r.K + C::chunk - 1) / C::chunk, per = (chunks + split - 1) / split;
    const int c0 = min(rank * per, chunks), c1 = min(c0 + per, chunks);
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::code_stages; ++i) {
            mbar_init(bars.code_full + i, 1);
            mbar_init(bars.code_empty + i, 4);  // the warps that widen the chunk
        }
        for (int i = 0; i < kRowStages; ++i) {
            mbar_init(bars.row_full + i, 64);  // every lane of both loading warps
            mbar_init(bars.row_empty + i, 1);
        }
        for (int i = 0; i < C::a_bufs; ++i) {
            mbar_init(bars.a_full + i, 4);
            mbar_init(bars.a_empty + i, 1);
        }
        for (int i = 0; i < C::d_bufs; ++i) {
            mbar_init(bars.d_full + i, 1);
            mbar_init(bars.d_empty + i, 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.join_full + i, 4 * split);  // a summing warpgroup of every CTA of the cluster
            mbar_init(bars.join_free + i, 4 * split);
            mbar_init(bars.summed + i, 4);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
    }
    // tensor memory is taken only once the kernels before this one have finished
    pdl_wait();
    if (warp == 3) tmem_alloc(&bars.tmem, 512);
    const int total = uniform(int4_lists<TN, 16>(p.r, lists, panels));
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peers' barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem = uniform(bars.tmem);
    const int first = blockIdx.x / split, stride = gridDim.x / split;
    bool timed_out = false;
    // a warpgroup takes its registers with one instruction
    if (warp < 4) {
        give_registers<kIssueRegs>();
        if (warp == 0) {
            // ------------------------------------------------------------ codes
            Feed feed;
            Ring r;
            uint32_t armed = 0, armed_par = 0;  // stages with copies not yet seen landed
            for (int t = first; t < total && !timed_out; t += stride) {
                const Int4Item it = feed.next(lists, p.r.E, panels, total, t, stride, lane);
                const Halves h = halves_of(it.panel, swiglu);
                for (int c = c0; c < c1; ++c) {
                    if (!role_wait(bars.code_empty + r.s, r.ph ^ 1u, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    if (lane == 0) {
                        uint64_t* bar = bars.code_full + r.s;
                        const uint32_t dst = smem_u32(smem + r.s * C::code_stage);
                        mbar_arrive_expect_tx(bar, C::code_stage);
                        tma_load_3d(dst, &tW, c * (C::chunk / 2), h.a, it.e, bar);
                        tma_load_3d(dst + C::code_stage / 2, &tW, c * (C::chunk / 2), h.b, it.e, bar);
                    }
                    armed |= 1u << r.s;
                    armed_par = (armed_par & ~(1u << r.s)) | (r.ph << r.s);
                    r.next<C::code_stages>();
                }
            }
            if ((timed_out || *abort_flag) && lane == 0) {
                *abort_flag = 1;
                for (int i = 0; i < C::code_stages; ++i)
                    if (armed & (1u << i)) {
                        volatile uint32_t never = 0;
                        (void)mbar_wait(bars.code_full + i, (armed_par >> i) & 1u, &never);
                    }
            }
        } else if (warp == 1 || warp == 3) {
            // ------------------------------------------------------- token rows
            // each of the two warps takes 64 of a stage's 128 elements; a lane 16 bytes
            // of every fourth row, into the 128-byte swizzle, whose 8-row atoms of the
            // two halves alternate.  As many stages as tiles of this width leave room
            // for; where the width changes, they are all waited for first.
            Feed feed;
            const int half = warp >> 1, sub = lane >> 3, piece = lane & 7;
            const uint32_t even = sub * 128 + ((piece ^ sub) << 4), odd = (sub + 4) * 128 + ((piece ^ (sub + 4)) << 4);
            const uint32_t dst0 = smem_u32(s_rows) + half * 1024, pitch = static_cast<uint32_t>(p.ldx * 2);
            int n_stages = 0, s = 0;
            uint32_t used = 0;  // parity of each stage's uses
            auto load = [&](const Int4Item& it, auto quads) {
                constexpr int kQuads = decltype(quads)::value, wide = 4 * kQuads;
                // rows that are not stored, or stored as zeros, may be any; their numbers are
                // held and not their addresses, which would not fit beside one another
                uint32_t from[kQuads];
#pragma unroll
                for (int i = 0; i < kQuads; ++i)
                    from[i] = 4 * i + sub < it.rows ? max(int4_token_row(p, it.row + 4 * i + sub), 0) : 0;
                const uint8_t* at = static_cast<const uint8_t*>(p.x) + (c0 * C::chunk + half * 64 + piece * 8) * static_cast<int64_t>(2);
                for (int c = c0; c < c1; ++c) {
#pragma unroll
                    for (int u = 0; u < C::chunk / 128; ++u) {
                        if (!role_wait(bars.row_empty + s, (used >> s & 1u) ^ 1u, abort_flag)) {
                            timed_out = true;
                            return;
                        }
                        const uint32_t to_even = dst0 + s * wide * 256 + even, to_odd = dst0 + s * wide * 256 + odd;
                        const int k0 = c * C::chunk + u * 128;
                        if (k0 + 128 <= p.r.K) {
#pragma unroll
                            for (int i = 0; i < kQuads; ++i)
                                cp_async_16((i & 1 ? to_odd : to_even) + (i >> 1) * 2048, at + static_cast<uint64_t>(from[i]) * pitch + u * 256, 16);
                        } else {
                            const bool in = k0 + half * 64 + piece * 8 < p.r.K;
#pragma unroll
                            for (int i = 0; i < kQuads; ++i)
                                cp_async_16((i & 1 ? to_odd : to_even) + (i >> 1) * 2048,
                                            in ? at + static_cast<uint64_t>(from[i]) * pitch + u * 256 : static_cast<const uint8_t*>(p.x), in ? 16 : 0);
                        }
                        // not a wait for the copies and a proxy fence here: the fence waits for all
                        // that the warp has under way (127 us for 32 rows in each of 32 groups)
                        cp_async_arrive(bars.row_full + s);
                        used ^= 1u << s;
                        if (++s == row_stages(wide)) s = 0;
                    }
                    at += C::chunk * 2;
                }
            };
            for (int t = first; t < total && !timed_out; t += stride) {
                const Int4Item it = feed.next(lists, p.r.E, panels, total, t, stride, lane);
                const int wide = (it.rows + 15) & ~15;
                if (row_stages(wide) != n_stages) {
                    for (int i = 0; i < n_stages && !timed_out; ++i)
                        timed_out = !role_wait(bars.row_empty + i, (used >> i & 1u) ^ 1u, abort_flag);
                    n_stages = row_stages(wide);
                    s = 0;
                    if (timed_out) break;
                }
                if (wide == 16) load(it, std::integral_constant<int, 4>());
                else if (wide == 32) load(it, std::integral_constant<int, 8>());
                else if constexpr (TN == 64) {
                    if (wide == 48) load(it, std::integral_constant<int, 12>());
                    else load(it, std::integral_constant<int, 16>());
                }
            }
            // nothing of this CTA's shared memory may still be written to at exit
            cp_async_commit();
            cp_async_wait<0>();
        } else if (warp == 2) {
            // ------------------------------------------------------------- MMAs
            Feed feed;
            const uint32_t one = elect_one();
            // 8-row atoms 2048 bytes apart: those of the two halves alternate
            const uint64_t b0 = sdesc_sw128(smem_u32(s_rows)) + (static_cast<uint64_t>(1024u >> 4) << 32);
            Ring a, d;
            int n_stages = 0, s = 0;
            uint32_t used = 0;
            bool issued = false;
            for (int t = first; t < total && !timed_out; t += stride) {
                const Int4Item it = feed.next(lists, p.r.E, panels, total, t, stride, lane);
                const int wide = (it.rows + 15) & ~15;
                if (row_stages(wide) != n_stages) {
                    n_stages = row_stages(wide);
                    s = 0;
                }
                const uint32_t idesc = (1u << 4) | (Int4Wide<T>::format << 7) | (Int4Wide<T>::format << 10) |
                                       (static_cast<uint32_t>(wide >> 3) << 17) | (8u << 24);
                for (int c = c0; c < c1 && !timed_out; ++c) {
                    if (!role_wait(bars.d_empty + d.s, d.ph ^ 1u, abort_flag) || !role_wait(bars.a_full + a.s, a.ph, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    const uint32_t dcol = tmem + static_cast<uint32_t>(d.s * C::d_cols);
                    const uint32_t acol = tmem + C::a_col + static_cast<uint32_t>(a.s * (C::chunk / 2));
#pragma unroll
                    for (int u = 0; u < C::chunk / 128; ++u) {
                        if (!role_wait(bars.row_full + s, used >> s & 1u, abort_flag)) {
                            timed_out = true;
                            break;
                        }
                        fence_proxy_async_smem();  // the rows came through the generic proxy
                        tc_fence_after();
                        const uint32_t b = static_cast<uint32_t>(b0) + static_cast<uint32_t>(s * wide * 16);
                        // a branch, not a predicate on each: 110 us against 104 for 32 rows in each of
                        // 32 groups
                        if (one) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_tmem(dcol + ((u * 128 + k * 16) / G) * TN, acol + (u * 8 + k) * 8,
                                         b + (k >> 2) * 64 + (k & 3) * 2, static_cast<uint32_t>(b0 >> 32), idesc,
                                         k % (G / 16) != 0);
                            mma_commit(bars.row_empty + s);
                        }
                        __syncwarp();
                        issued = true;
                        used ^= 1u << s;
                        if (++s == n_stages) s = 0;
                    }
                    if (timed_out) break;
                    commit_if(one, bars.a_empty + a.s);
                    commit_if(one, bars.d_full + d.s);
                    a.next<C::a_bufs>();
                    d.next<C::d_bufs>();
                }
            }
            if ((timed_out || *abort_flag) && issued && one) {
                *abort_flag = 1;
                mma_commit(&bars.drain);
                volatile uint32_t never = 0;
                (void)mbar_wait(&bars.drain, 0, &never);
            }
        }
    } else if (warp < 12) {
        take_registers<kSumRegs>();
        // ------------------------------------------------- sums and epilogue
        const int q = warp & 3, me = q * 32 + lane;  // weight row of the panel
        const uint32_t quarter = tmem + (static_cast<uint32_t>(q * 32) << 16);
        Feed feed;
        Ring d;
        // The two warpgroups take the items in turn: one's epilogue runs beside the
        // other's sums.  Each item's barriers are those of its warpgroup, so that a
        // phase is waited for only once the phase before it has been: a parity says
        // no more than that.
        const int w = warp >> 3;
        int turn = 0;
        for (int t = first; t < total && !timed_out; t += stride, ++turn) {
            const Int4Item it = feed.next(lists, p.r.E, panels, total, t, stride, lane);
            if ((turn & 1) != w) {
                for (int c = c0; c < c1; ++c) d.next<C::d_bufs>();
                continue;
            }
            const uint32_t ph = turn >> 1 & 1, other_ph = w ? ph : ph ^ 1u;  // of the item before: none, at first
            const Halves hv = halves_of(it.panel, swiglu);
            const int wide = (it.rows + 15) & ~15;
            Stream<C::parts, uint16_t> scales;
            scales.start(static_cast<const uint16_t*>(p.scales) + weight_row(p, it.e, hv, me) * p.groups, p.groups, p.whole,
                         0u, c0);
            float acc[TN];
#pragma unroll
            for (int n = 0; n < TN; ++n) acc[n] = 0.0f;
            // the sums of the item before have been taken
            if (!role_wait(bars.summed + (w ^ 1), other_ph, abort_flag, sum_limit_ns(per))) {
                timed_out = true;
                break;
            }
            for (int c = c0; c < c1; ++c) {
                // a group past the row's end has sum 0, and scale 0
                uint32_t sbits[C::parts];
                scales.take(c, sbits);
                if (!role_wait(bars.d_full + d.s, d.ph, abort_flag)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < C::parts; ++j) {
                    const uint32_t col = quarter + static_cast<uint32_t>(d.s * C::d_cols + j * TN);
                    const float s = to_float<T>(__builtin_bit_cast(T, static_cast<uint16_t>(sbits[j])));
#pragma unroll
                    for (int n0 = 0; n0 < TN; n0 += 16) {
                        if (n0 >= wide) break;
                        uint32_t v[16];
                        tmem_ld16(col + n0, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int n = 0; n < 16; ++n) acc[n0 + n] = fmaf(__uint_as_float(v[n]), s, acc[n0 + n]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.d_empty + d.s);
                d.next<C::d_bufs>();
            }
            if (timed_out) break;
            if (lane == 0) mbar_arrive(bars.summed + w);
            // every CTA of the cluster stores wide / split columns: parts to them
            const int share = wide / split;
            if (!role_wait(bars.join_free + (w ^ 1), other_ph, abort_flag, sum_limit_ns(per))) {
                timed_out = true;  // the columns of the item before have not been read
                break;
            }
            if (split == 1) {
                float* dst = reinterpret_cast<float*>(s_join) + me;
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    if (n >= wide) break;
                    dst[n * 128] = acc[n];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.join_full + w);
            } else {
                fence_cluster();
                const uint32_t mine = smem_u32(s_join) + static_cast<uint32_t>(rank * share * 512 + me * 4);
                int to = 0, left = share;
                uint32_t dst = mapa_shared(mine, 0);
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    if (n >= wide) break;
                    if (left == 0) {
                        left = share;
                        dst = mapa_shared(mine, static_cast<uint32_t>(++to));
                    }
                    st_cluster_f32(dst, acc[n]);
                    dst += 512;
                    --left;
                }
                fence_cluster();
                __syncwarp();
                if (lane < split) mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_full + w), static_cast<uint32_t>(lane)));
            }
            if (!role_wait(bars.join_full + w, ph, abort_flag, sum_limit_ns(per))) {
                timed_out = true;
                break;
            }
            if (split > 1) fence_cluster();
            // a warp takes every fourth column (with SwiGLU, every fourth two): a
            // token, whose features lie along the lanes, four to each
            const float* join = reinterpret_cast<const float*>(s_join);
            T* out = static_cast<T*>(p.r.out);
            constexpr float up = 1.0f / Int4Wide<T>::unit;  // the codes were widened in units of their own
            auto sum4 = [&](int c, int f) {
                float4 v = *reinterpret_cast<const float4*>(join + c * 128 + f);
                for (int o = 1; o < split; ++o) {
                    const float4 w = *reinterpret_cast<const float4*>(join + (o * share + c) * 128 + f);
                    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                }
                v.x *= up, v.y *= up, v.z *= up, v.w *= up;
                return v;
            };
            const int each = swiglu ? 2 : 1;
            for (int cb = q * each; cb < min(share, it.rows - rank * share); cb += 4 * each) {
                const int c = cb + (swiglu ? lane >> 4 : 0), token = rank * share + c;
                const int f = swiglu ? 4 * (lane & 15) : 4 * lane, n = it.panel * (swiglu ? 64 : 128) + f;
                if (c >= share || token >= it.rows || n >= p.columns) continue;
                const int row = it.row + token;
                float4 v = sum4(c, f);
                if (swiglu) {
                    const float4 u = sum4(c, 64 + f);
                    v.x = v.x / (1.0f + expf(-v.x)) * u.x;
                    v.y = v.y / (1.0f + expf(-v.y)) * u.y;
                    v.z = v.z / (1.0f + expf(-v.z)) * u.z;
                    v.w = v.w / (1.0f + expf(-v.w)) * u.w;
                }
                const float g = p.r.row_scale ? ld_dep(p.r.row_scale + row) : 1.0f;
                v.x *= g, v.y *= g, v.z *= g, v.w *= g;
                if (p.src && int4_token_row(p, row) < 0) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                *reinterpret_cast<uint2*>(out + row * p.r.ldo + n) = make_uint2(pack2(T(), v.x, v.y), pack2(T(), v.z, v.w));
            }
            __syncwarp();
            if (split == 1) {
                if (lane == 0) mbar_arrive(bars.join_free + w);
            } else if (lane < split) {
                mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_free + w), static_cast<uint32_t>(lane)));
            }
        }
    } else {
        // ---------------------------------------------------------- widening
        give_registers<kWidenRegs>();
        Feed feed;
        const int mine = (warp - 12) >> 2, q = warp & 3, me = q * 32 + lane;
        const uint32_t quarter = tmem + (static_cast<uint32_t>(q * 32) << 16) + C::a_col;
        // 16-byte piece i of row `me` in the 128-byte or 64-byte swizzle
        const int turn = C::chunk == 256 ? me & 7 : (me >> 1) & 3;
        Ring s, a;
        int turns = 0;
        for (int t = first; t < total && !timed_out; t += stride) {
            const Int4Item it = feed.next(lists, p.r.E, panels, total, t, stride, lane);
            Stream<C::parts, uint8_t> zeros;
            zeros.start(p.zeros ? p.zeros + weight_row(p, it.e, halves_of(it.panel, swiglu), me) * p.groups : nullptr,
                        p.groups, p.whole, 8u, c0);
            for (int c = c0; c < c1; ++c) {
                uint32_t zero[C::parts];
                zeros.take(c, zero);
#pragma unroll
                for (int j = 0; j < C::parts; ++j) zero[j] = int4_zero<T>(zero[j]);
                if ((turns++ & 1) == mine) {
                    if (!role_wait(bars.code_full + s.s, s.ph, abort_flag) ||
                        !role_wait(bars.a_empty + a.s, a.ph ^ 1u, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    const uint4* row = reinterpret_cast<const uint4*>(smem + s.s * C::code_stage + me * (C::chunk / 2));
#pragma unroll
                    for (int h = 0; h < C::chunk / 64; ++h) {  // 64 elements, 32 columns
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 u = row[(2 * h + i) ^ turn];
                            const uint32_t z = zero[(2 * h + i) * 32 / G];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[16 * i + j] = int4_widen<T>(u.x, j, z);
                                v[16 * i + 4 + j] = int4_widen<T>(u.y, j, z);
                                v[16 * i + 8 + j] = int4_widen<T>(u.z, j, z);
                                v[16 * i + 12 + j] = int4_widen<T>(u.w, j, z);
                            }
                        }
                        tmem_st(quarter + static_cast<uint32_t>(a.s * (C::chunk / 2) + h * 32), v);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.code_empty + s.s);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.a_full + a.s);
                }
                s.next<C::code_stages>();
                a.next<C::a_bufs>();
            }
        }
    }
    if (timed_out) *abort_flag = 1;
    if (timed_out && p.r.status) atomicOr(p.r.status, kRaggedTimeout);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no peer still writes to this CTA's shared memory
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// CTAs that split a sum: as many as leave all items, of groups of equal lengths, to run
// at once; an item costs its start and its joining whatever is left of its sum.  By split
// 1, 2, 4 and 8, with groups of 128 elements: 64 rows with 4096 x 4096 weights (32 items)
// 35, 33, 29 and 37 us, with 1024 x 16384 (8 items) 74, 53, 39 and 31, 16 rows in each of
// 8 groups of 7168 x 2048 (448 items) 35, 47, 68 and 131.
int split_of(int64_t items, int chunks) {
    int split = 1;
    while (split < kMaxSplit && items * split * 2 <= num_sms() && chunks >= 4 * split) split *= 2;
    return split;
}

template <typename T, int G>
cudaError_t launch(const Int4Product& q, cudaStream_t st) {
    using C = Cfg<G>;
    Int4Product p = q;
    p.whole = p.groups % 8 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15) == 0 &&
              (reinterpret_cast<uintptr_t>(p.zeros) & 7) == 0;
    static int found[kMaxDevices][4] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    CUtensorMap tW;
    const uint64_t K = p.r.K, N = p.r.N, E = p.r.E;
    const uint64_t wd[3] = {K / 2, N, E}, ws[2] = {K / 2, N * (K / 2)};
    const uint32_t wb[3] = {C::chunk / 2, 64, 1};
    if (!make_tensor_map(&tW, p.codes, 3, wd, ws, wb, CU_TENSOR_MAP_DATA_TYPE_UINT8, C::chunk / 2)) return cudaErrorInvalidValue;
    const int64_t panels = p.swiglu ? p.columns / 64 : (p.r.N + 127) / 128;
    const int64_t items = panels * (p.r.R / C::TN + (p.r.R < p.r.E ? p.r.R : p.r.E));  // at most
    const int64_t used = p.r.R < p.r.E ? p.r.R : p.r.E, each = (p.r.R + used - 1) / used;  // groups with rows, theirs
    const int split = split_of(panels * used * ((each + C::TN - 1) / C::TN), static_cast<int>((K + C::chunk - 1) / C::chunk));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    int& n = found[dev][split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3];  // clusters at once
    if (!n) {
        cudaError_t e = cudaFuncSetAttribute(k_int4_wide<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
        if (e != cudaSuccess) return e;
        int most = num_sms();
        if (split > 1) {
            e = cudaOccupancyMaxActiveClusters(&most, k_int4_wide<T, G>, &cfg);
            if (e != cudaSuccess) return e;
        }
        n = most > 0 ? most : 1;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(split * (items < n ? items : n)));
    return cudaLaunchKernelEx(&cfg, k_int4_wide<T, G>, tW, p);
}

}  // namespace

template <typename T>
cudaError_t launch_int4_wide(int group, const Int4Product& p, cudaStream_t st) {
    if (group == 32) return launch<T, 32>(p, st);
    return group == 64 ? launch<T, 64>(p, st) : launch<T, 128>(p, st);
}
template cudaError_t launch_int4_wide<__nv_bfloat16>(int, const Int4Product&, cudaStream_t);
template cudaError_t launch_int4_wide<__half>(int, const Int4Product&, cudaStream_t);

}  // namespace moe
