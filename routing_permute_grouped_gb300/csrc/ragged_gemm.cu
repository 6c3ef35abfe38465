// ragged_gemm.cu -- matrix products grouped by expert on ragged row groups,
// bf16 or f16: y[r] = row_scale[r] * x[r] W[e]^T (or x[r] W[e]) and the weight
// gradient dW[e] = sum over e's rows of a[r]^T b[r].
//
// Both run on CTA pairs (tcgen05 cta_group::2, fp32 accumulators in tensor
// memory, two of them so that a tile's epilogue overlaps the next tile's MMAs),
// one persistent pair per two SMs, operands staged by TMA in 64-element steps
// of the sum.
//
// Product.  The operands are swapped: 256 rows of W[e] are the MMA's M (128 per
// CTA), a token tile of at most 256 rows its N, in steps of 32 -- a ragged
// group wastes at most 31 columns of one tile, where row tiles on the M side
// waste up to 255 rows.  The same kernel then serves two rows per expert (the
// weights stream through the SM once) and thousands.  W is K-major or, for x W
// and the data gradient, MN-major through the transposing bit of the MMA; no
// copy is laid out.  Sizes that the tiles do not divide are zero-filled by TMA
// on loads and cut off by the epilogue.
//
// Weight gradient.  The sum runs along the rows, so both operands are MN-major.
// The last step of a group holds rows of the next one: one warp of each CTA
// zeroes them in shared memory (both operands: a NaN of another group times
// zero is not zero) before the step is handed to the MMAs.  An empty group's
// tiles are written as zeros.
//
// Where a call has fewer tiles than the GPU has pairs and a long sum, two or four
// pairs of a cluster split the sum (SP) and join their fp32 parts through each
// other's shared memory, in an order that does not depend on timing.
//
// What bounds them: at the default layer's gate/up size (32768 rows, 8 experts,
// 7168 -> 4096) a launch by itself takes 1.02 to 1.04 ms, 1850 to 1890 TFLOP/s,
// with the tensor pipe 92 to 93 % busy at 1.62 GHz, the board's power limit; back
// to back 1.14 to 1.19 ms.  The data gradient of a 64-expert layer (98304 rows,
// 2048 -> 4096): 0.90 to 0.91 ms alone, 91 % busy.  The weight gradient: 0.93 ms,
// 81 % busy, waiting for loads (two 64-column boxes per operand and step).  Two
// rows for each of 256 experts: the weights' bytes over HBM.  Clusters of two
// pairs that share one operand by TMA multicast gained nothing (default 1.169
// against 1.187 ms, data gradient 1.069 against 1.062): fewer SMs hold clusters
// of four.
//
// Warp roles: warp 0 TMA producer, warp 1 tensor memory and MMA issue (even
// CTA), warps 2..9 epilogue, warp 10 (weight gradient) the zeroing of tails.
// Every wait is bounded; on a timeout the CTA flags the status word, lets its
// copies and MMAs in flight finish and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr int kBK = 64;                 // step of the sum
constexpr int kOpBytes = 128 * kBK * 2; // one operand of one CTA and stage: 16 KB
constexpr int kStage = 2 * kOpBytes;
constexpr int kChunk = 64 * kBK * 2;    // a 64 x 64 box of an MN-major operand
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int map = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    static constexpr uint32_t idesc = idesc_bf16_f32(256, 8) & ~(0x3Fu << 17);
};
template <>
struct Elem<__half> {  // operand formats 0 in bits [7,10) and [10,13)
    static constexpr int map = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    static constexpr uint32_t idesc = (1u << 4) | ((256u >> 4) << 24);
};

// ---------------------------------------------------------------- product --
// SP > 1 pairs (a cluster of 2 SP CTAs) share an item, each with its part of the
// sum: for calls with fewer items than pairs and long sums, like one expert's
// decode batch, whose time is the length of one item's chain of steps.
template <int SP>
struct Prod {
    static constexpr int TN = SP == 1 ? 256 : 64;  // token rows of a tile, at most
    static constexpr int stages = SP == 1 ? 6 : 5;
    static constexpr int stage = kOpBytes + TN / 2 * 128;
    static constexpr int join = (SP - 1) * kEpiWarps * 4096;
    static constexpr int smem = 1024 + stages * stage + kEpiStage + join + 1024 + static_cast<int>(sizeof(RaggedTiles));
    static_assert(smem <= 232448, "shared memory budget");
    static_assert(stage % 1024 == 0, "swizzled tiles need 1024-byte alignment");
};

template <typename T, bool WT, int SP>
__global__ void __cluster_dims__(2 * SP, 1, 1) __launch_bounds__(64 + 32 * kEpiWarps, 1)
    k_ragged_product(const __grid_constant__ CUtensorMap tW, const __grid_constant__ RowMaps tX,
                     const __grid_constant__ CUtensorMap tY, const RaggedArgs args) {
    using C = Prod<SP>;
    constexpr int S = C::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sOut = smem + S * C::stage;
    uint8_t* join = sOut + kEpiStage;
    PairBars<S>& bars = *reinterpret_cast<PairBars<S>*>(join + C::join);
    static_assert(sizeof(PairBars<S>) <= 1024, "barriers");
    RaggedTiles& tiles = *reinterpret_cast<RaggedTiles*>(join + C::join + 1024);
    volatile uint32_t* abort_flag = &bars.abort;

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t cta = rank & 1, lead = SP == 1 ? 0 : rank & ~1u;  // of the pair
    const bool leader = cta == 0;
    const uint16_t both = static_cast<uint16_t>(0x3u << lead);
    const int panels = (args.N + 255) / 256;
    const int all = (args.K + kBK - 1) / kBK, pair = static_cast<int>(rank >> 1);
    const int k0 = SP == 1 ? 0 : pair * all / SP, k1 = SP == 1 ? all : (pair + 1) * all / SP;  // this pair's steps
    pdl_trigger();
    pair_start(bars, 1, warp, SP > 1 ? SP - 1 : 1);
    if (warp == 2) ragged_tiles_build<C::TN>(args, tiles, panels, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = uniform(bars.tmem);
    const int total = uniform(tiles.first[args.E]);
    const int first = blockIdx.x / (2 * SP), stride = gridDim.x / (2 * SP);
    bool timed_out = false;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        // converged, one lane issuing, as the MMA warp
        const uint32_t one = elect_one();
        Ring r;
        uint32_t armed = 0, armed_par = 0;  // stages with copies not yet seen landed
        RaggedFeed feed;
        for (int t = first; t < total && !timed_out; t += stride) {
            const RaggedItem it = feed.next(tiles, args.E, panels, total, t, stride, lane);
            const int half = ((it.rows + 31) & ~31) / 2;  // token rows of each CTA
            const int xrow = it.row + half * static_cast<int>(cta);
            const int wrow = it.panel * 256 + 128 * static_cast<int>(cta);
            for (int k = k0; k < k1; ++k) {
                if (!warp_wait(bars.empty + r.s, r.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                const uint32_t full = mapa_shared(smem_u32(bars.full + r.s), lead);
                uint8_t* st = smem + r.s * C::stage;
                armed &= ~(1u << r.s);
                if (leader) mbar_arrive_expect_tx_if(one, bars.full + r.s, 2 * (kOpBytes + half * 128));
                if constexpr (WT) {
                    tma_load_3d_pair_if(one, st, &tW, wrow, k * kBK, it.e, full);
                    tma_load_3d_pair_if(one, st + kChunk, &tW, wrow + 64, k * kBK, it.e, full);
                } else {
                    tma_load_3d_pair_if(one, st, &tW, k * kBK, wrow, it.e, full);
                }
                load_rows(one, tX, st + kOpBytes, k * kBK, xrow, half, full);
                armed |= 1u << r.s;
                armed_par = (armed_par & ~(1u << r.s)) | (r.ph << r.s);
                r.next<S>();
            }
        }
        if ((timed_out || *abort_flag) && leader && lane == 0) {
            *abort_flag = 1;
            for (int i = 0; i < S; ++i)
                if (armed & (1u << i)) {
                    volatile uint32_t never = 0;
                    (void)mbar_wait(bars.full + i, (armed_par >> i) & 1u, &never);
                }
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------- MMA issuer
            // The warp stays converged and one lane issues: descriptors and
            // loop counters are then warp-uniform values, which the MMA takes
            // as they are.
            const uint32_t one = elect_one();
            const uint64_t wd0 = WT ? sdesc_sw128_mn(smem_u32(smem), kChunk) : sdesc_sw128(smem_u32(smem));
            const uint64_t xd0 = sdesc_sw128(smem_u32(smem + kOpBytes));
            constexpr uint32_t kWStep = (WT ? 2048 : 32) >> 4;  // 16 elements of the sum
            Ring r;
            Acc acc;
            bool issued = false, ready = false;
            RaggedFeed feed;
            for (int t = first; t < total && !timed_out; t += stride) {
                const RaggedItem it = feed.next(tiles, args.E, panels, total, t, stride, lane);
                const uint32_t n = (it.rows + 31) & ~31;
                const uint32_t idesc = Elem<T>::idesc | ((n >> 3) << 17) | (WT ? kTransA : 0u);
                if (!warp_wait(bars.tempty + acc.i, acc.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc.i * C::TN);
                for (int k = k0; k < k1; ++k) {
                    if (!ready && !warp_wait(bars.full + r.s, r.ph, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    const Ring next = r.after<S>();
                    const bool peek = mbar_test_wait(bars.full + next.s, next.ph);
                    const uint32_t at = static_cast<uint32_t>(r.s) * (C::stage >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        mma_bf16_pair_if(one, d, wd0 + (at + kk * kWStep), xd0 + (at + kk * 2), idesc,
                                         ((k - k0) | kk) != 0 ? 1u : 0u);
                    mma_commit_pair_if(one, bars.empty + r.s, both);
                    ready = __all_sync(0xFFFFFFFFu, peek);
                    issued = true;
                    r = next;
                }
                if (timed_out) break;
                mma_commit_pair_if(one, bars.tfull + acc.i, both);
                acc.next();
            }
            if ((timed_out || *abort_flag) && issued && one) {
                *abort_flag = 1;
                mma_commit_pair(&bars.drain, static_cast<uint16_t>(1u << rank));
                volatile uint32_t never = 0;
                (void)mbar_wait(&bars.drain, 0, &never);
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        if (!product_epilogue<T, C::TN, SP>(args, tY, tiles, bars, panels, total, first, stride, k1 - k0, tmem_base, warp - 2,
                                            lane, rank, sOut + (warp - 2) * 2048, 1.0f, [](int) { return 1.0f; }, join))
            timed_out = true;
        if (timed_out) *abort_flag = 1;
    }
    if (timed_out && args.status) atomicOr(args.status, kRaggedTimeout);
    pair_end(tmem_base, warp);
}

// -------------------------------------------------------- weight gradient --
// One staging buffer (32 rows x 128 bytes) per epilogue warp and a sixth stage:
// 1.067 against 1.094 ms with two buffers and five stages on the 64-expert
// layer's gradient, and as fast where the stores bound it (64 experts, 8 rows
// each: 6.3 TB/s).
constexpr int kGradStages = 6;
constexpr int kOutStage = kEpiWarps * 4096;
constexpr int kGradSmem = 1024 + kGradStages * kStage + kOutStage + 1024;
static_assert(kGradSmem <= 232448, "shared memory budget");

struct GradTile {
    int e, m, n;     // group, first row and column of the 256 x 256 output tile
    int row, rows;   // the group's rows; with several pairs, this pair's part
    int whole;       // the group's rows
};

__device__ __forceinline__ GradTile grad_tile(const RaggedArgs& a, int t) {
    const int nt = (a.N + 255) / 256, mt = (a.K + 255) / 256;
    GradTile g;
    g.e = t / (mt * nt);
    const int r = t - g.e * mt * nt;
    g.m = r / nt * 256;
    g.n = r % nt * 256;
    const int2 rows = group_rows(a, g.e);
    g.row = rows.x;
    g.rows = rows.y - rows.x;
    return g;
}

// A warp's tiles, found 32 at a time (see RaggedFeed).
template <int SP>
struct GradFeed {
    GradTile mine;
    int k = 32;
    __device__ __forceinline__ GradTile next(const RaggedArgs& a, int total, int t, int stride, int lane, int pair) {
        if (k == 32) {
            k = 0;
            const int64_t at = t + static_cast<int64_t>(lane) * stride;
            if (at < total) mine = grad_tile(a, static_cast<int>(at));
        }
        GradTile g;
        g.e = __shfl_sync(0xFFFFFFFFu, mine.e, k);
        g.m = __shfl_sync(0xFFFFFFFFu, mine.m, k);
        g.n = __shfl_sync(0xFFFFFFFFu, mine.n, k);
        g.row = __shfl_sync(0xFFFFFFFFu, mine.row, k);
        g.rows = g.whole = __shfl_sync(0xFFFFFFFFu, mine.rows, k);
        ++k;
        if constexpr (SP > 1) {  // whole steps of 64 rows
            const int steps = (g.whole + kBK - 1) / kBK;
            const int s0 = pair * steps / SP, s1 = (pair + 1) * steps / SP;
            g.row += s0 * kBK;
            g.rows = min(g.whole - s0 * kBK, (s1 - s0) * kBK);
        }
        return g;
    }
};

// The pairs of a cluster hold sums over parts of a group's rows.  Of the 128
// columns of an epilogue warp, pair p finishes the p-th 128 / SP: the warps send
// one another those columns in fp32 and add what they receive to their own, the
// other pairs' in ascending order.  What is sent lands in the receiver's pipeline
// stages: a cluster has one tile, so they are free once its sum is complete, which
// join_free says.  has: this pair had rows, and its accumulator is at taddr;
// limit: of each wait, in ns.  False on a timeout.
template <int SP>
__device__ __forceinline__ bool exchange_parts(PairBars<kGradStages>& bars, float (&f)[128 / SP], uint8_t* stages,
                                               uint32_t taddr, bool has, int ew, int lane, uint32_t rank,
                                               uint64_t limit) {
    constexpr int kPart = 128 / SP;
    constexpr int kBytes = kPart * 128;  // of a warp: 32 lanes x kPart fp32
    static_assert((SP - 1) * kEpiWarps * kBytes <= kGradStages * kStage, "the parts fit the stages");
    const volatile uint32_t* abort_flag = &bars.abort;
    const int pair = static_cast<int>(rank >> 1), cta = static_cast<int>(rank & 1);
    if (lane == 0)
        for (int o = 0; o < SP; ++o)
            if (o != pair) mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_free + ew), 2 * o + cta));
    if (!warp_wait(bars.join_free + ew, 0, abort_flag, limit)) return false;
    fence_cluster();
#pragma unroll 1
    for (int i = 1; i < SP; ++i) {
        const int to = (pair + i) % SP;  // not all at once to the same pair
        const int slot = pair < to ? pair : pair - 1;
        const uint32_t dst = mapa_shared(smem_u32(stages + (slot * kEpiWarps + ew) * kBytes), 2 * to + cta) + lane * 16;
#pragma unroll
        for (int c = 0; c < kPart; c += 32) {
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
            if (has) {
                tmem_ld32(taddr + to * kPart + c, v);
                tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                st_cluster_v4(dst + (c / 4 + j) * 512, __uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                              __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        }
        fence_cluster();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_full + ew), 2 * to + cta));
    }
    if (has) {
#pragma unroll
        for (int c = 0; c < kPart; c += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + pair * kPart + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) f[c + j] = __uint_as_float(v[j]);
        }
    }
    if (!warp_wait(bars.join_full + ew, 0, abort_flag, limit)) return false;
    fence_cluster();
#pragma unroll 1
    for (int o = 0; o < SP - 1; ++o) {
        const float4* src = reinterpret_cast<const float4*>(stages + (o * kEpiWarps + ew) * kBytes) + lane;
#pragma unroll
        for (int j = 0; j < kPart / 4; ++j) {
            const float4 w = src[j * 32];
            f[4 * j] += w.x;
            f[4 * j + 1] += w.y;
            f[4 * j + 2] += w.z;
            f[4 * j + 3] += w.w;
        }
    }
    return true;
}

template <typename T, int SP>
__global__ void __cluster_dims__(2 * SP, 1, 1) __launch_bounds__(96 + 32 * kEpiWarps, 1)
    k_ragged_wgrad(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB,
                   const __grid_constant__ CUtensorMap tOut, const RaggedArgs args) {
    constexpr int S = kGradStages;
    constexpr int kPart = 128 / SP;  // columns of a warp's 128 that this pair finishes
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sOut = smem + S * kStage;
    PairBars<S>& bars = *reinterpret_cast<PairBars<S>*>(sOut + kOutStage);
    volatile uint32_t* abort_flag = &bars.abort;

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t cta = rank & 1, lead = SP == 1 ? 0 : rank & ~1u;  // of the pair
    const bool leader = cta == 0;
    const uint16_t both = static_cast<uint16_t>(0x3u << lead);
    const int pair = static_cast<int>(rank >> 1);
    pdl_trigger();
    // a stage is full when both CTAs say so (and its bytes have landed)
    pair_start(bars, 2, warp, SP > 1 ? SP - 1 : 1, SP > 1 ? SP - 1 : 1);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = uniform(bars.tmem);
    const int total = args.E * ((args.N + 255) / 256) * ((args.K + 255) / 256);
    const int first = blockIdx.x / (2 * SP), stride = gridDim.x / (2 * SP);
    bool timed_out = false;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        const uint32_t one = elect_one();
        Ring r;
        uint32_t armed = 0, armed_par = 0, tails = 0, tail_par = 0, tail_ph = 0;
        GradFeed<SP> feed;
        for (int t = first; t < total && !timed_out; t += stride) {
            const GradTile g = feed.next(args, total, t, stride, lane, pair);
            const int ac = g.m + 128 * static_cast<int>(cta), bc = g.n + 128 * static_cast<int>(cta);
            for (int k = 0; k < g.rows; k += kBK) {
                if (!warp_wait(bars.empty + r.s, r.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                uint8_t* st = smem + r.s * kStage;
                const uint32_t bit = 1u << r.s;
                // a tail's bytes go to the CTA's own barrier: the zeroing warp
                // hands that stage on
                const bool tail = g.rows - k < kBK;
                armed &= ~bit;
                tails &= ~bit;
                if (tail) {
                    tails |= bit;
                    tail_par = (tail_par & ~bit) | (tail_ph & bit);
                    tail_ph ^= bit;
                } else {
                    armed |= bit;
                    armed_par = (armed_par & ~bit) | (r.ph << r.s);
                }
                const uint32_t bar = tail ? mapa_shared(smem_u32(bars.tail + r.s), rank)
                                          : mapa_shared(smem_u32(bars.full + r.s), lead);
                const int row = g.row + k;
                if (tail)
                    mbar_arrive_expect_tx_if(one, bars.tail + r.s, kStage);
                else if (leader)
                    mbar_arrive_expect_tx_if(one, bars.full + r.s, 2 * kStage);
                else if (one)
                    mbar_arrive_cluster_relaxed(bar);
                tma_load_2d_pair_if(one, st, &tA, ac, row, bar);
                tma_load_2d_pair_if(one, st + kChunk, &tA, ac + 64, row, bar);
                tma_load_2d_pair_if(one, st + kOpBytes, &tB, bc, row, bar);
                tma_load_2d_pair_if(one, st + kOpBytes + kChunk, &tB, bc + 64, row, bar);
                r.next<S>();
            }
        }
        if ((timed_out || *abort_flag) && lane == 0) {
            *abort_flag = 1;
            volatile uint32_t never = 0;
            for (int i = 0; i < S; ++i) {
                if (leader && (armed & (1u << i)))
                    (void)mbar_wait(bars.full + i, (armed_par >> i) & 1u, &never);
                if (tails & (1u << i)) (void)mbar_wait(bars.tail + i, (tail_par >> i) & 1u, &never);
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = Elem<T>::idesc | ((256u >> 3) << 17) | kTransA | kTransB;
            const uint32_t one = elect_one();
            const uint64_t ad0 = sdesc_sw128_mn(smem_u32(smem), kChunk);
            const uint64_t bd0 = sdesc_sw128_mn(smem_u32(smem + kOpBytes), kChunk);
            Ring r;
            Acc acc;
            bool issued = false, ready = false;
            GradFeed<SP> feed;
            for (int t = first; t < total && !timed_out; t += stride) {
                const GradTile g = feed.next(args, total, t, stride, lane, pair);
                if (g.rows == 0) continue;  // the epilogue writes zeros
                if (!warp_wait(bars.tempty + acc.i, acc.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc.i * 256);
                for (int k = 0; k < g.rows; k += kBK) {
                    if (!ready && !warp_wait(bars.full + r.s, r.ph, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    const Ring next = r.after<S>();
                    const bool peek = mbar_test_wait(bars.full + next.s, next.ph);
                    const uint32_t at = static_cast<uint32_t>(r.s) * (kStage >> 4);
                    const int rest = g.rows - k;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)  // 16 rows per MMA
                        if (kk * 16 < rest)
                            mma_bf16_pair_if(one, d, ad0 + (at + kk * (2048 >> 4)), bd0 + (at + kk * (2048 >> 4)),
                                             idesc, (k | kk) != 0 ? 1u : 0u);
                    mma_commit_pair_if(one, bars.empty + r.s, both);
                    ready = __all_sync(0xFFFFFFFFu, peek);
                    issued = true;
                    r = next;
                }
                if (timed_out) break;
                mma_commit_pair_if(one, bars.tfull + acc.i, both);
                acc.next();
            }
            if ((timed_out || *abort_flag) && issued && one) {
                *abort_flag = 1;
                mma_commit_pair(&bars.drain, static_cast<uint16_t>(1u << rank));
                volatile uint32_t never = 0;
                (void)mbar_wait(&bars.drain, 0, &never);
            }
        }
    } else if (warp == 2 + kEpiWarps) {
        // ------------------------------------------------- zeroing of tails
        Ring r;
        uint32_t tail_ph = 0;
        int64_t ahead = 0;  // steps from the last tail to the next
        GradFeed<SP> feed;
        for (int t = first; t < total && !timed_out; t += stride) {
            const GradTile g = feed.next(args, total, t, stride, lane, pair);
            const int steps = (g.rows + kBK - 1) / kBK, rest = g.rows % kBK;
            for (int k = 0; k + 1 < steps; ++k) r.next<S>();
            if (steps == 0) continue;
            ahead += steps;
            if (rest) {
                if (!warp_wait(bars.tail + r.s, (tail_ph >> r.s) & 1u, abort_flag, sum_limit_ns(ahead))) {
                    timed_out = true;
                    break;
                }
                ahead = 0;
                tail_ph ^= 1u << r.s;
                // rows [rest, next multiple of 16): one 128-byte row in each of
                // the four 64-column chunks (a row stays in its own 128 bytes
                // under the swizzle)
                uint8_t* st = smem + r.s * kStage;
                const int n = ((rest + 15) & ~15) - rest;
                for (int i = lane; i < n * 32; i += 32) {
                    const int row = rest + (i >> 5), c = (i >> 3) & 3;
                    *reinterpret_cast<uint4*>(st + c * kChunk + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(bars.full + r.s), lead));
            }
            r.next<S>();
        }
    } else {
        // ------------------------------------------------------ epilogue
        // Each warp owns 32 rows of M (its tensor-memory lane quarter) and
        // half of the tile's columns (with several pairs, finishes its part of
        // them), and stores them through TMA from boxes of 32 x 64 (four pairs:
        // 32 x 32) staged in shared memory; TMA cuts off what lies past M or N.
        const int q = warp & 3, ew = warp - 2;
        const int c0 = (ew >> 2) * 128;
        Acc acc;
        uint8_t* stage = sOut + ew * 4096;
        GradFeed<SP> feed;
        for (int t = first; t < total; t += stride) {
            const GradTile g = feed.next(args, total, t, stride, lane, pair);
            const int m = g.m + 128 * static_cast<int>(cta) + q * 32;
            const int n = g.n + c0;
            uint32_t pk[kPart / 2];
            uint32_t taddr = 0;
            const uint64_t limit = sum_limit_ns(g.whole / kBK + 1);
            if (g.rows) {
                if (!warp_wait(bars.tfull + acc.i, acc.ph, abort_flag, limit)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
                taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc.i * 256 + c0);
            }
            if constexpr (SP == 1) {
                if (g.rows) {
#pragma unroll
                    for (int c = 0; c < 128; c += 64) {
                        uint32_t v[2][32];
                        tmem_ld32(taddr + c, v[0]);
                        tmem_ld32(taddr + c + 32, v[1]);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            pk[c / 2 + i] = pack2(T(), __uint_as_float(v[i >> 4][2 * (i & 15)]),
                                                  __uint_as_float(v[i >> 4][2 * (i & 15) + 1]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) pk[i] = 0u;
                }
            } else {
                float f[kPart];
#pragma unroll
                for (int i = 0; i < kPart; ++i) f[i] = 0.f;
                if (g.whole && !exchange_parts<SP>(bars, f, smem, taddr, g.rows != 0, ew, lane, rank, limit)) {
                    timed_out = true;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kPart / 2; ++i) pk[i] = pack2(T(), f[2 * i], f[2 * i + 1]);
            }
            if (g.rows) {
                // handed back before the stores; they are not what the MMA
                // side waits for, so the arrive need not release them
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(bars.tempty + acc.i), lead));
                acc.next();
            }
            constexpr int kBox = kPart < 64 ? kPart : 64;  // columns per box
#pragma unroll
            for (int c = 0; c < kPart; c += kBox) {
                const int nc = n + pair * kPart + c;
                if (m >= args.K || nc >= args.N) continue;
                if (lane == 0) bulk_wait_read<0>();  // the previous store has read the buffer
                __syncwarp();
                uint8_t* sb = stage + lane * kBox * 2;
#pragma unroll
                for (int j = 0; j < kBox / 8; ++j) {  // 16-byte chunks of a row of 128 or 64 bytes
                    const uint32_t* u = pk + c / 2 + 4 * j;
                    const int at = kBox == 64 ? j ^ (lane & 7) : j ^ ((lane >> 1) & 3);
                    *reinterpret_cast<uint4*>(sb + (at << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tOut, stage, nc, m, g.e);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        if (timed_out) *abort_flag = 1;
    }
    if (timed_out && args.status) atomicOr(args.status, kRaggedTimeout);
    pair_end(tmem_base, warp);
}

// --------------------------------------------------------------- launches --
// Items of tiles of tn token rows, at most: every group with rows may round up.
int64_t most_items(const RaggedArgs& a, int tn) {
    const int64_t groups = a.R < a.E ? a.R : a.E;
    return (a.R + (tn - 1) * groups) / tn * ((a.N + 255) / 256);
}

template <typename T, bool WT, int SP>
cudaError_t launch_product(const RaggedArgs& a, const void* x, int64_t ldx, const void* w, cudaStream_t st) {
    using C = Prod<SP>;
    static bool ready[kMaxDevices] = {};
    const uint64_t N = a.N, K = a.K, R = a.R, E = a.E;
    CUtensorMap tW, tY;
    RowMaps tX;
    const uint64_t wd[3] = {WT ? N : K, WT ? K : N, E};
    const uint64_t ws[2] = {wd[0] * 2, N * K * 2};
    const uint32_t wb[3] = {64, WT ? 64u : 128u, 1};
    if (!make_tensor_map(&tW, w, 3, wd, ws, wb, Elem<T>::map) ||
        !make_row_maps(&tX, x, R, K, static_cast<uint64_t>(ldx) * 2, 64, Elem<T>::map) ||
        !make_out_map(&tY, a, Elem<T>::map))
        return cudaErrorInvalidValue;
    const int64_t items = most_items(a, C::TN);
    return launch_pairs<SP>(k_ragged_product<T, WT, SP>, items, 64 + 32 * kEpiWarps, C::smem, ready, st, tW, tX, tY, a);
}

// Few items and a long sum: the sum is split over the pairs of a cluster, four
// or two, as many as let every item run at once.  One expert, 16 rows, 7168 ->
// 2048: 13.7 us with four pairs, 24.8 without; 200 rows: 18.6 against 31.4 with
// two; 64 rows, 7168 -> 4096: 20.3 against 26.1 with two, 30.9 with four, of
// which not all 16 clusters fit; 64 rows, 2048 -> 7168: 12.0 against 11.1 with
// two, so two pairs want the longer sum.
template <typename T, bool WT>
cudaError_t product(const RaggedArgs& a, const void* x, int64_t ldx, const void* w, cudaStream_t st) {
    static int four[kMaxDevices] = {}, two[kMaxDevices] = {};
    constexpr int kThreads = 64 + 32 * kEpiWarps;
    const int64_t items = most_items(a, Prod<2>::TN);
    if (a.K >= 16 * kBK && items <= num_sms() / 4) {
        if (items <= resident_clusters<4>(k_ragged_product<T, WT, 4>, kThreads, Prod<4>::smem, four))
            return launch_product<T, WT, 4>(a, x, ldx, w, st);
        if (a.K >= 50 * kBK &&
            items <= resident_clusters<2>(k_ragged_product<T, WT, 2>, kThreads, Prod<2>::smem, two))
            return launch_product<T, WT, 2>(a, x, ldx, w, st);
    }
    return launch_product<T, WT, 1>(a, x, ldx, w, st);
}

template <typename T, int SP>
cudaError_t launch_wgrad(const RaggedArgs& a, const void* x, int64_t ldx, const void* y, int64_t ldy,
                         cudaStream_t st) {
    static bool ready[kMaxDevices] = {};
    const uint64_t M = a.K, N = a.N, R = a.R, E = a.E;
    CUtensorMap tA, tB, tOut;
    const uint64_t ad[2] = {M, R}, as[1] = {static_cast<uint64_t>(ldx) * 2};
    const uint64_t bd[2] = {N, R}, bs[1] = {static_cast<uint64_t>(ldy) * 2};
    const uint64_t od[3] = {N, M, E}, os[2] = {N * 2, M * N * 2};
    const uint32_t box[2] = {64, 64}, obox[3] = {SP == 4 ? 32u : 64u, 32, 1};
    if (!make_tensor_map(&tA, x, 2, ad, as, box, Elem<T>::map) || !make_tensor_map(&tB, y, 2, bd, bs, box, Elem<T>::map) ||
        !make_tensor_map(&tOut, a.out, 3, od, os, obox, Elem<T>::map, SP == 4 ? 64 : 128))
        return cudaErrorInvalidValue;
    const int64_t items = static_cast<int64_t>(E) * ((N + 255) / 256) * ((M + 255) / 256);
    // split sums: one tile per cluster
    if (items > (SP > 1 ? num_sms() / (2 * SP) : INT32_MAX)) return cudaErrorInvalidValue;
    return launch_pairs<SP>(k_ragged_wgrad<T, SP>, items, 96 + 32 * kEpiWarps, kGradSmem, ready, st, tA, tB, tOut, a);
}

// Few tiles and many rows (a router's or an adapter's gradient, few small
// experts): the rows are split over the pairs of a cluster, four or two, as many
// as let every tile run at once.  bf16, one group, without and with: 8192 rows,
// 2048 x 512: 39.3 and 25.6 us (two pairs); 7168 x 256: 40.3 and 29.1 (two); 4096
// rows, 512 x 512: 21.9 and 14.0 (four; 16.1 with two); 2048 rows: 13.5 and 11.8;
// 1024 rows: 9.2 and 10.7.  Eight groups of 2048 rows: 14.6 and 14.8.  So it starts
// at 2048 rows per group; the average is what the host knows of them.
template <typename T>
cudaError_t wgrad(const RaggedArgs& a, const void* x, int64_t ldx, const void* y, int64_t ldy, cudaStream_t st) {
    static int four[kMaxDevices] = {}, two[kMaxDevices] = {};
    constexpr int kThreads = 96 + 32 * kEpiWarps;
    const int64_t items = static_cast<int64_t>(a.E) * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    if (a.R / a.E >= 32 * kBK && items <= num_sms() / 4) {
        if (items <= resident_clusters<4>(k_ragged_wgrad<T, 4>, kThreads, kGradSmem, four))
            return launch_wgrad<T, 4>(a, x, ldx, y, ldy, st);
        if (items <= resident_clusters<2>(k_ragged_wgrad<T, 2>, kThreads, kGradSmem, two))
            return launch_wgrad<T, 2>(a, x, ldx, y, ldy, st);
    }
    return launch_wgrad<T, 1>(a, x, ldx, y, ldy, st);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status_t check_ragged(int32_t dtype, int64_t R, int32_t A, int32_t B, int32_t E) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    if (R < 0 || A <= 0 || B <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (A % 8 || B % 8)
        return set_last_error(MOE_ERR_UNSUPPORTED, "dimensions %d and %d must be multiples of 8", A, B);
    if (A > kRaggedMaxDim || B > kRaggedMaxDim)
        return set_last_error(MOE_ERR_UNSUPPORTED, "dimensions %d and %d must be at most 2^30", A, B);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm(int32_t dtype, int64_t R, int32_t N, int32_t K, int32_t E, const void* x,
                                         int64_t ldx, const void* w, int32_t w_transposed, const int32_t* offsets,
                                         const float* row_scale, void* y, int64_t ldy, uint32_t* status,
                                         void* stream) {
    const moe_status_t s = check_ragged(dtype, R, N, K, E);
    if (s != MOE_OK) return s;
    if (R == 0) return MOE_OK;
    if (!x || !w || (!offsets && E != 1) || !y) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(w) || !aligned16(y))
        return set_last_error(MOE_ERR_INVALID_ARG, "x, w and y must be 16-byte aligned");
    if (ldx < K || ldx % 8 || ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG,
                              "row strides must cover the row and be multiples of 8 elements");
    RaggedArgs a{};
    a.offsets = offsets;
    a.R = static_cast<int32_t>(R);
    a.N = N;
    a.K = K;
    a.E = E;
    a.row_scale = row_scale;
    a.out = y;
    a.ldo = ldy;
    a.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == MOE_DTYPE_BF16)
        e = w_transposed ? product<__nv_bfloat16, true>(a, x, ldx, w, st) : product<__nv_bfloat16, false>(a, x, ldx, w, st);
    else
        e = w_transposed ? product<__half, true>(a, x, ldx, w, st) : product<__half, false>(a, x, ldx, w, st);
    return e == cudaSuccess ? MOE_OK
                            : set_last_error(MOE_ERR_CUDA, "grouped product: %s", cudaGetErrorString(e));
}

extern "C" moe_status_t moe_grouped_wgrad(int32_t dtype, int64_t R, int32_t M, int32_t N, int32_t E, const void* a_,
                                          int64_t lda, const void* b, int64_t ldb, const int32_t* offsets, void* out,
                                          uint32_t* status, void* stream) {
    const moe_status_t s = check_ragged(dtype, R, M, N, E);
    if (s != MOE_OK) return s;
    if (!out || (R > 0 && (!a_ || !b || (!offsets && E != 1)))) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(out) || (R > 0 && (!aligned16(a_) || !aligned16(b))))
        return set_last_error(MOE_ERR_INVALID_ARG, "a, b and out must be 16-byte aligned");
    if (R > 0 && (lda < M || lda % 8 || ldb < N || ldb % 8))
        return set_last_error(MOE_ERR_INVALID_ARG,
                              "row strides must cover the row and be multiples of 8 elements");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (R == 0) {
        e = cudaMemsetAsync(out, 0, static_cast<size_t>(E) * M * N * 2, st);
    } else {
        RaggedArgs a{};
        a.offsets = offsets;
        a.R = static_cast<int32_t>(R);
        a.N = N;
        a.K = M;
        a.E = E;
        a.out = out;
        a.status = status;
        e = dtype == MOE_DTYPE_BF16 ? wgrad<__nv_bfloat16>(a, a_, lda, b, ldb, st)
                                    : wgrad<__half>(a, a_, lda, b, ldb, st);
    }
    return e == cudaSuccess ? MOE_OK
                            : set_last_error(MOE_ERR_CUDA, "grouped weight gradient: %s", cudaGetErrorString(e));
}
