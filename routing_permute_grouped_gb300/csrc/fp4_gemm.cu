// fp4_gemm.cu -- the grouped product on 4-bit rows and weights with block
// scales: y[r] = row_scale[r] * gx * gw[e] * sum_k x[r, k] W[e][n, k].
//
// The schedule of the 16-bit product (ragged_gemm.cu): 256 rows of W[e] are
// the M of a CTA pair's MMAs, a token tile of at most 224 (MX) or 192 (NV) rows
// the N, in steps of 32.  The MMAs (tcgen05 kind::mxf4 / kind::mxf4nvf4, K = 64)
// multiply the e2m1 codes with their block scales as they are, so nothing is
// widened: a step of 256 elements is 128 bytes of each row.
//
// Scales.  The MMA wants them in tensor memory as 32-bit words (four bytes
// along K), word of row r in lane r % 32 and column r / 32, repeated in the
// four lane quarters.  In global memory they are row-major.  One warp of each
// CTA copies 16 bytes of every row of the tile (a scale group: 512 elements of
// MX, 256 of NV) into shared memory with cp.async, several groups ahead.  Four
// warps, one per lane quarter, read a group back, lane l the four words of rows
// l, l + 32, l + 64, ..., and store them to tensor memory word by word; the
// transposition is a renaming of registers.  (Laying the words out in shared
// memory for tcgen05.cp needs the writes published to the tensor core of both
// CTAs: that cluster-scope release made a decode step over 256 experts 884 us
// instead of 507.)  Bytes past K are cleared on the way (they may hold
// anything), rows past the operand repeat its last row and reach no stored
// result.  A step's barrier is full when its codes have landed and its scales
// are written: one wait per step, because a wait costs the MMA warp some 100
// cycles even when there is nothing to wait for (445 against 405 us with two).
//
// What bounds it (default gate/up product of 8 experts, 32768 rows, 7168 ->
// 4096, MX: 293 to 330 us, 5.8 to 6.6 PFLOP/s): the turn of the two scale
// buffers.  A step's scales can be stored once the MMAs of two steps before are
// complete, and its own MMAs start only after the store, its hand-over and the
// issue.  Counted in the kernel at that size, of 627 cycles per step, of which
// its four MMAs run 432 (tensor pipe 70 % busy): the MMA warp waits 260 for a
// step's codes and scales (ready at once in 2 % of the steps), issues the MMAs
// in 130 and commits in 44; a layout warp waits 270 for a free buffer and 70 for
// a group of scales, stores and hands on in 115 and reads and rearranges the
// rest; the TMA warp is busy for 510.  The loads alone took 252 us.
// Decode (two rows for each of 256 experts) runs at the weights' bytes over HBM.
// Short sums (K = 1024: 216 to 232 us for 98304 rows of 64 experts, N = 4096) are
// bound by the epilogue: the MMAs of a tile run 40 % of its time.
// NV has twice the scale words and tiles of 192 rows: 391 to 396 us where MX
// takes 293 to 297, 259 where it takes 216.
//
// A scale buffer in tensor memory is written again once its MMAs are complete.
//
// Warp roles: warp 0 TMA producer, warp 1 tensor memory and MMA issue (even
// CTA), warp 2 scale loads, warps 4..7 scale layout, warps 8..15 epilogue.
// Every wait is bounded, as in ragged_gemm.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr int kStep = 256;                // step of the sum: 128 bytes of codes
constexpr int kWBytes = 128 * 128;        // weight codes of one CTA and stage
constexpr int kEpi0 = 8;                  // first epilogue warp
constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);

// A step's cost outside its MMAs is the same for every tile, and an MMA runs N / 2
// cycles, so the widest tile is the fastest.  Two accumulators and two scale
// buffers (the words of one step, two of MX and four of NV, each 4 columns of A
// and 8 of B) must fit 512 columns of tensor memory: 224 token rows for MX, 192
// for NV (MX with 192: 342 against 324 us).
template <bool NV>
struct Cfg {
    static constexpr int TN = NV ? 192 : 224;  // token rows of a tile, at most
    static constexpr int pieces = 4 + TN / 32;  // 32-row pieces of a tile's scales: weights, tokens
    static constexpr int stage = kWBytes + TN / 2 * 128;
    static constexpr int stages = NV ? 6 : 5;
    static constexpr int raw = 7;               // scale groups in shared memory
    static constexpr int raw_bytes = pieces * 512;
    static constexpr int words = NV ? 4 : 2;    // of a step's scales
    static constexpr int bufs = 2;              // scale buffers
    static constexpr uint32_t cols = words * 12;
    static constexpr uint32_t scale_col = 2 * TN;  // the first one's tensor-memory column
    static constexpr int smem =
        1024 + stages * stage + raw * raw_bytes + kEpiStage + 1024 + static_cast<int>(sizeof(RaggedTiles));
    static_assert(scale_col + bufs * cols <= 512, "tensor memory budget");
    static_assert(smem <= 232448, "shared memory budget");
    static_assert(stage % 1024 == 0, "swizzled tiles need 1024-byte alignment");
};

template <int RAW>
struct ScaleBars {
    uint64_t raw_full[RAW], raw_empty[RAW];  // groups in shared memory
};

template <bool NV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_ragged_product_fp4(const __grid_constant__ CUtensorMap tW, const __grid_constant__ RowMaps tX,
                         const __grid_constant__ CUtensorMap tY, const uint8_t* w_scales, const uint8_t* x_scales,
                         const int pitch, const RaggedArgs args) {
    using C = Cfg<NV>;
    constexpr int S = C::stages;
    constexpr int kGroup = NV ? 256 : 512;  // elements under 16 scale bytes
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* raw = smem + S * C::stage;
    uint8_t* sOut = raw + C::raw * C::raw_bytes;
    PairBars<S>& bars = *reinterpret_cast<PairBars<S>*>(sOut + kEpiStage);
    ScaleBars<C::raw>& sb = *reinterpret_cast<ScaleBars<C::raw>*>(&bars + 1);
    static_assert(sizeof(PairBars<S>) % 8 == 0 && sizeof(PairBars<S>) + sizeof(ScaleBars<C::raw>) <= 1024, "barriers");
    RaggedTiles& tiles = *reinterpret_cast<RaggedTiles*>(sOut + kEpiStage + 1024);
    volatile uint32_t* abort_flag = &bars.abort;

    const int warp = uniform(static_cast<int>(threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int panels = (args.N + 255) / 256;
    const int steps = (args.K + kStep - 1) / kStep;
    const int groups = (args.K + kGroup - 1) / kGroup;
    pdl_trigger();
    if (threadIdx.x == 32) {
        for (int i = 0; i < C::raw; ++i) {
            mbar_init(sb.raw_full + i, 32);  // every lane's copies
            mbar_init(sb.raw_empty + i, 4);  // every layout warp
        }
        fence_mbar_init();
    }
    __syncwarp();
    // a step is full when its codes have landed and the four layout warps of
    // both CTAs have written its scales
    pair_start(bars, 9, warp);
    if (warp == 2) ragged_tiles_build<C::TN>(args, tiles, panels, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = uniform(bars.tmem);
    const int total = uniform(tiles.first[args.E]);
    const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
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
            const int xrow = it.row + half * static_cast<int>(rank);
            const int wrow = it.panel * 256 + 128 * static_cast<int>(rank);
            for (int k = 0; k < steps; ++k) {
                if (!warp_wait(bars.empty + r.s, r.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                const uint32_t full = mapa_shared(smem_u32(bars.full + r.s), 0);
                uint8_t* st = smem + r.s * C::stage;
                armed &= ~(1u << r.s);
                if (leader) mbar_arrive_expect_tx_if(one, bars.full + r.s, 2 * (kWBytes + half * 128));
                tma_load_3d_pair_if(one, st, &tW, k * 128, wrow, it.e, full);
                load_rows(one, tX, st + kWBytes, k * 128, xrow, half, full);
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
            // converged, one lane issuing, as in ragged_gemm.cu
            constexpr uint32_t idesc0 = idesc_e2m1_f32(256, 8, !NV) & ~(0x3Fu << 17);
            const uint32_t one = elect_one();
            const uint64_t wd0 = sdesc_sw128(smem_u32(smem)), xd0 = sdesc_sw128(smem_u32(smem + kWBytes));
            Ring r;
            Acc acc;
            Ring buf;  // scale buffer
            bool issued = false, ready = false;
            RaggedFeed feed;
            for (int t = first; t < total && !timed_out; t += stride) {
                const RaggedItem it = feed.next(tiles, args.E, panels, total, t, stride, lane);
                const uint32_t n = (it.rows + 31) & ~31;
                const uint32_t idesc = idesc0 | ((n >> 3) << 17);
                if (!warp_wait(bars.tempty + acc.i, acc.ph ^ 1u, abort_flag)) {
                    timed_out = true;
                    break;
                }
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc.i * C::TN);
                for (int k = 0; k < steps; ++k) {
                    if (!ready && !warp_wait(bars.full + r.s, r.ph, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    // the next stage is looked at while this one's MMAs are
                    // issued: a wait costs even when there is nothing to wait for
                    const Ring next = r.after<S>();
                    const bool peek = mbar_test_wait(bars.full + next.s, next.ph);
                    const uint32_t at = static_cast<uint32_t>(r.s) * (C::stage >> 4);
                    const uint32_t sa = tmem_base + C::scale_col + static_cast<uint32_t>(buf.s) * C::cols;
                    const int left = args.K - k * kStep;
                    if (one) {
                        auto mma = [&](int kk) {  // 64 elements of each 128-byte row
                            const int word = NV ? kk : kk / 2;
                            const uint32_t byte = NV ? 0u : static_cast<uint32_t>(kk & 1) * 2u;
                            mma_e2m1_pair<NV>(d, wd0 + (at + kk * 2), xd0 + (at + kk * 2),
                                              idesc | (byte << 4) | (byte << 29), sa + word * 4,
                                              sa + C::words * 4 + word * 8, (k | kk) != 0 ? 1u : 0u);
                        };
                        if (left >= kStep) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) mma(kk);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                if (kk * 64 < left) mma(kk);
                        }
                        // read by the scale warps too: a step's scale buffer is
                        // free with its stage
                        mma_commit_pair(bars.empty + r.s, 0x3);
                    }
                    ready = __all_sync(0xFFFFFFFFu, peek);
                    issued = true;
                    buf.next<C::bufs>();
                    r = next;
                }
                if (timed_out) break;
                mma_commit_pair_if(one, bars.tfull + acc.i, 0x3);
                acc.next();
            }
            if ((timed_out || *abort_flag) && issued && one) {
                *abort_flag = 1;
                mma_commit_pair(&bars.drain, 0x1);
                volatile uint32_t never = 0;
                (void)mbar_wait(&bars.drain, 0, &never);
            }
        }
    } else if (warp == 2) {
        // ---------------------------------------------------- scale loads
        int s = 0;
        uint32_t ph = 0;
        RaggedFeed feed;
        for (int t = first; t < total && !timed_out; t += stride) {
            const RaggedItem it = feed.next(tiles, args.E, panels, total, t, stride, lane);
            const int64_t w_last = static_cast<int64_t>(it.e + 1) * args.N - 1;
            const int64_t w0 = static_cast<int64_t>(it.e) * args.N + it.panel * 256 + 128 * static_cast<int>(rank);
            const uint8_t* wp[4];
            const uint8_t* xp[C::TN / 32];
#pragma unroll
            for (int c = 0; c < 4; ++c) wp[c] = w_scales + min(w0 + c * 32 + lane, w_last) * pitch;
#pragma unroll
            for (int c = 0; c < C::TN / 32; ++c)
                xp[c] = x_scales + static_cast<int64_t>(it.row + min(c * 32 + lane, it.rows - 1)) * pitch;
            for (int g = 0; g < groups; ++g) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(sb.raw_empty + s, ph ^ 1u, abort_flag))) {
                    timed_out = true;
                    break;
                }
                const uint32_t dst = smem_u32(raw + s * C::raw_bytes) + lane * 16;
#pragma unroll
                for (int c = 0; c < 4; ++c) cp_async_16(dst + c * 512, wp[c] + g * 16, 16);
#pragma unroll
                for (int c = 0; c < C::TN / 32; ++c)
                    if (c * 32 < it.rows) cp_async_16(dst + (4 + c) * 512, xp[c] + g * 16, 16);
                cp_async_arrive(sb.raw_full + s);
                if (++s == C::raw) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // nothing of this CTA's shared memory may still be written to at exit
        cp_async_commit();
        cp_async_wait<0>();
    } else if (warp == 3) {
        // no part: the layout warps start at a multiple of four
    } else if (warp < kEpi0) {
        // --------------------------------------------------- scale layout
        const int valid = args.K / (NV ? 16 : 32);  // scale bytes of a row
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int s = 0;
        uint32_t ph = 0;
        Ring buf;
        // the stage of the step whose buffer is written next, C::bufs steps ago
        Ring old, cur;  // cur: its own
        int fresh = C::bufs;  // buffers not yet written
        for (int t = first; t < total && !timed_out; t += stride) {
            for (int g = 0; g < groups; ++g) {
                const int left = valid - g * 16;  // bytes of this group inside K
                uint4 v[C::pieces];
                if (!warp_wait(sb.raw_full + s, ph, abort_flag)) {
                    timed_out = true;
                    break;
                }
                const uint4* src = reinterpret_cast<const uint4*>(raw + s * C::raw_bytes) + lane;
#pragma unroll
                for (int c = 0; c < C::pieces; ++c) v[c] = src[c * 32];
                __syncwarp();
                if (lane == 0) mbar_arrive(sb.raw_empty + s);
                if (left < 16) {
                    uint32_t m[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int b = left - 4 * q;
                        m[q] = b >= 4 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
                    }
#pragma unroll
                    for (int c = 0; c < C::pieces; ++c)
                        v[c] = make_uint4(v[c].x & m[0], v[c].y & m[1], v[c].z & m[2], v[c].w & m[3]);
                }
                if (++s == C::raw) {
                    s = 0;
                    ph ^= 1u;
                }
#pragma unroll
                for (int h = 0; h < 4 / C::words; ++h) {  // the group's buffers
                    if (4 * C::words * h >= left) break;
                    // the MMAs that last read this buffer are complete
                    if (fresh == 0 && !warp_wait(bars.empty + old.s, old.ph, abort_flag)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    uint32_t a[4 * C::words], b[8 * C::words];
#pragma unroll
                    for (int q = 0; q < C::words; ++q) {
                        auto word = [&](int c) {
                            const int i = C::words * h + q;
                            return i == 0 ? v[c].x : i == 1 ? v[c].y : i == 2 ? v[c].z : v[c].w;
                        };
#pragma unroll
                        for (int c = 0; c < 4; ++c) a[4 * q + c] = word(c);
#pragma unroll
                        for (int c = 0; c < 8; ++c) b[8 * q + c] = c < C::TN / 32 ? word(4 + (c < C::TN / 32 ? c : 0)) : 0u;
                    }
                    const uint32_t dst = tmem_base + quarter + C::scale_col + static_cast<uint32_t>(buf.s) * C::cols;
                    tmem_st(dst, a);
                    tmem_st(dst + 4 * C::words, b);
                    tmem_st_wait();
                    // the words are in tensor memory; the MMA side reads
                    // nothing else of this warp's, so the arrive releases
                    // nothing
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(bars.full + cur.s), 0));
                    buf.next<C::bufs>();
                    cur.next<S>();
                    if (fresh)
                        --fresh;
                    else
                        old.next<S>();
                }
                if (timed_out) break;
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        const float gx = args.x_scale ? ld_dep(args.x_scale) : 1.0f;
        if (!product_epilogue<__nv_bfloat16, C::TN, 1>(
                args, tY, tiles, bars, panels, total, first, stride, steps, tmem_base, warp - kEpi0, lane, rank,
                sOut + (warp - kEpi0) * 2048, gx,
                [&](int e) { return args.w_scale ? ld_dep(args.w_scale + e) : 1.0f; }))
            timed_out = true;
    }
    if (timed_out) *abort_flag = 1;
    if (timed_out && args.status) atomicOr(args.status, kRaggedTimeout);
    pair_end(tmem_base, warp);
}

template <bool NV>
cudaError_t launch_fp4(const RaggedArgs& a, const void* xq, const uint8_t* xs, const void* wq, const uint8_t* ws,
                       int pitch, cudaStream_t st) {
    using C = Cfg<NV>;
    static bool ready[kMaxDevices] = {};
    const uint64_t N = a.N, KB = a.K / 2, R = a.R, E = a.E;  // KB bytes of codes per row
    CUtensorMap tW, tY;
    RowMaps tX;
    const uint64_t wd[3] = {KB, N, E}, wst[2] = {KB, N * KB};
    const uint32_t wb[3] = {128, 128, 1};
    if (!make_tensor_map(&tW, wq, 3, wd, wst, wb, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !make_row_maps(&tX, xq, R, KB, KB, 128, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !make_out_map(&tY, a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16))
        return cudaErrorInvalidValue;
    const int64_t items = (R / C::TN + (R < E ? R : E)) * ((N + 255) / 256);  // at most
    return launch_pairs(k_ragged_product_fp4<NV>, items, kThreads, C::smem, ready, st, tW, tX, tY, ws, xs, pitch,
                              a);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm_fp4(int32_t fmt, int64_t R, int32_t N, int32_t K, int32_t E, const void* x_codes,
                                             const void* x_scales, const void* w_codes, const void* w_scales,
                                             const int32_t* offsets, const float* x_scale, const float* w_scale,
                                             const float* row_scale, void* y, int64_t ldy, uint32_t* status,
                                             void* stream) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV)
        return set_last_error(MOE_ERR_INVALID_ARG, "format = %d is neither MX (0) nor NV (1)", fmt);
    if (R < 0 || N <= 0 || K <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (K % 32 || N % 8)
        return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d must be a multiple of 32 and N = %d of 8", K, N);
    if (K > kRaggedMaxDim || N > kRaggedMaxDim)
        return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d and N = %d must be at most 2^30", K, N);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    if (R == 0) return MOE_OK;
    if (!x_codes || !x_scales || !w_codes || !w_scales || (!offsets && E != 1) || !y)
        return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y))
        return set_last_error(MOE_ERR_INVALID_ARG, "codes, scales and y must be 16-byte aligned");
    if (ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    RaggedArgs a{};
    a.offsets = offsets;
    a.R = static_cast<int32_t>(R);
    a.N = N;
    a.K = K;
    a.E = E;
    a.row_scale = row_scale;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.out = y;
    a.ldo = ldy;
    a.status = status;
    const uint8_t* xs = static_cast<const uint8_t*>(x_scales);
    const uint8_t* ws = static_cast<const uint8_t*>(w_scales);
    const int pitch = static_cast<int>(moe_fp4_scale_stride(fmt, K));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = fmt == MOE_FP4_NV ? launch_fp4<true>(a, x_codes, xs, w_codes, ws, pitch, st)
                                            : launch_fp4<false>(a, x_codes, xs, w_codes, ws, pitch, st);
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit grouped product: %s", cudaGetErrorString(e));
}
