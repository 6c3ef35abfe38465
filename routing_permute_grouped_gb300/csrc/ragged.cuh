// ragged.cuh -- what the grouped products on ragged row groups share: the
// launch description and the reading of the group offsets.
//
// Token rows are sorted by group (expert): group e owns rows
// [offsets[e], offsets[e + 1]) of the row-major operands, of any size; rows
// before the first group and past the last belong to none.  The offsets live on
// the device, so nothing of the launch depends on them.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

constexpr int kRaggedMaxGroups = 256;
constexpr int kRaggedMaxDim = 1 << 30;  // of a matrix: (K + 255) / 256, 2 K and the like stay within 32 bits
constexpr uint32_t kRaggedBadGroup = 0x4u;  // MOE_DEVERR_SEGMENT

struct RaggedArgs {
    const int32_t* offsets;  // [E + 1], or null: one group of all rows
    int32_t R, N, K, E;      // rows, output columns, sum length (wgrad: M is K here), groups
    const float* row_scale;  // [R] or null
    const float* x_scale;    // [1] or null: 4-bit rows' tensor scale
    const float* w_scale;    // [E] or null: 4-bit weights' tensor scales
    void* out;
    int64_t ldo;             // output row stride (elements)
    uint32_t* status;        // device error word, may be null
};

// Rows [x, y) of group e; empty and flagged when they do not lie in [0, R].
__device__ __forceinline__ int2 group_rows(const RaggedArgs& a, int e, bool* bad = nullptr) {
    if (!a.offsets) return make_int2(0, a.R);
    const int lo = ld_dep(a.offsets + e);
    const int hi = ld_dep(a.offsets + e + 1);
    if (lo < 0 || hi < lo || hi > a.R) {
        if (a.status) atomicOr(a.status, kRaggedBadGroup);
        if (bad) *bad = true;
        return make_int2(0, 0);
    }
    return make_int2(lo, hi);
}

// ------------------------------------------------------------ work list --
// The products put the weights on the MMA's M side (256 rows of W[e] across a
// CTA pair) and the token rows on its N side, whose extent is free in steps of
// 32: a group of any size then costs its own rows rounded up to 32, not a
// multiple of the tile.  A group of len rows is cut into ceil(len / TN) equal
// token tiles; a work item is one token tile times one 256-row weight panel.
struct RaggedTiles {
    int first[kRaggedMaxGroups + 1];  // a group's first work item
    int lo[kRaggedMaxGroups], hi[kRaggedMaxGroups];
    int tiles[kRaggedMaxGroups];      // its token tiles
    int width[kRaggedMaxGroups];      // their rows, a multiple of 32 (<= TN)
};

struct RaggedItem {
    int e, panel;
    int row, rows;  // token rows [row, row + rows)
};

// One warp fills the list from the offsets.
template <int TN>
__device__ void ragged_tiles_build(const RaggedArgs& a, RaggedTiles& s, int panels, int lane) {
    int running = 0, end = 0;  // work items, and the end of the rows of the groups so far
    bool skipped = false;
    for (int base = 0; base < a.E; base += 32) {
        const int e = base + lane;
        int n = 0;
        bool bad = false;
        int2 g = make_int2(0, 0);
        if (e < a.E) g = group_rows(a, e, &bad);
        skipped |= __any_sync(0xFFFFFFFFu, bad);
        if (skipped) {  // only then can groups overlap: each starts past the ends of those before it
            int top = g.y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, top, o);
                if (lane >= o) top = max(top, y);
            }
            top = __shfl_up_sync(0xFFFFFFFFu, top, 1);
            g.x = min(max(g.x, lane ? max(top, end) : end), g.y);
        }
        end = max(end, __reduce_max_sync(0xFFFFFFFFu, g.y));
        if (e < a.E) {
            s.lo[e] = g.x;
            s.hi[e] = g.y;
            const int len = g.y - g.x, tiles = (len + TN - 1) / TN;
            s.tiles[e] = tiles;
            s.width[e] = tiles ? ((len + tiles - 1) / tiles + 31) & ~31 : 0;
            n = tiles * panels;
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (e < a.E) s.first[e] = running + x - n;
        running += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    if (lane == 0) s.first[a.E] = running;
}

// Item t: its group by bisection; inside a group, token tiles pass over eight
// panels at a time, so the items in flight share both operands in L2.
__device__ __forceinline__ RaggedItem ragged_item(const RaggedTiles& s, int n_groups, int panels, int t) {
    int e = 0, end = n_groups;  // first[e] <= t < first[end]
    while (end - e > 1) {
        const int mid = (e + end) >> 1;
        if (s.first[mid] <= t)
            e = mid;
        else
            end = mid;
    }
    RaggedItem it;
    it.e = e;
    const unsigned tiles = s.tiles[e], width = s.width[e];
    const unsigned i = t - s.first[e];
    const unsigned block = i / (tiles * 8), rest = i - block * tiles * 8;
    const unsigned wide = min(8u, panels - block * 8);
    const unsigned tile = rest / wide;
    it.panel = block * 8 + rest - tile * wide;
    it.row = s.lo[e] + tile * width;
    it.rows = min(static_cast<int>(width), s.hi[e] - it.row);
    return it;
}

// A warp's items first, first + stride, ...: the lanes find 32 of them at a time,
// and each is then four shuffles, which also make it warp-uniform.  Finding an
// item alone takes some 500 cycles, which every role of the pipeline would
// spend at every tile.
struct RaggedFeed {
    RaggedItem mine;
    int k = 32;
    __device__ __forceinline__ RaggedItem next(const RaggedTiles& s, int n_groups, int panels, int total, int t,
                                               int stride, int lane) {
        if (k == 32) {
            k = 0;
            const int64_t at = t + static_cast<int64_t>(lane) * stride;
            if (at < total) mine = ragged_item(s, n_groups, panels, static_cast<int>(at));
        }
        RaggedItem it;
        it.e = __shfl_sync(0xFFFFFFFFu, mine.e, k);
        it.panel = __shfl_sync(0xFFFFFFFFu, mine.panel, k);
        it.row = __shfl_sync(0xFFFFFFFFu, mine.row, k);
        it.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, k);
        ++k;
        return it;
    }
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float lo, float hi) { return pack_bf16x2(lo, hi); }
__device__ __forceinline__ uint32_t pack2(__half, float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Epilogue of the products for 32 accumulator columns: tokens row .. row + 31
// (`rows` of them are stored) times the warp's 32 features n0 .. n0 + 31, one
// feature per tensor-memory lane.  The accumulator is read in matrix-fragment
// form (v), packed to 16 bits and stored transposed through stmatrix into 2 KB
// of shared memory, [token][64 bytes] in the 64-byte swizzle, from where TMA
// stores it and cuts off the features past N.  The chunk that a group's last
// token cuts is copied by the lanes: the rows after it are another group's.
// (Copying every chunk that way, 64 bytes of eight rows per store instruction,
// kept the load/store pipe 72 % busy on short sums: the 64-expert 4-bit down
// projection took 256 us instead of 232.)
// gate is the factor of token row + lane.
template <typename T>
__device__ __forceinline__ void store_transposed(const RaggedArgs& a, const CUtensorMap& tY, const uint32_t (&v)[2][16],
                                                 int row, int rows, int n0, int lane, float gate, uint8_t* stage) {
    if (lane == 0) bulk_wait_read<0>();  // the previous chunk has left the buffer
    __syncwarp();
    const uint32_t sbase = smem_u32(stage);
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 8 tokens
        const float g0 = __shfl_sync(0xFFFFFFFFu, gate, 8 * j + 2 * (lane & 3));
        const float g1 = __shfl_sync(0xFFFFFFFFu, gate, 8 * j + 2 * (lane & 3) + 1);
        uint32_t p[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {  // 8 features
            const uint32_t* u = v[f >> 1] + 4 * j + 2 * (f & 1);
            p[f] = pack2(T(), __uint_as_float(u[0]) * g0, __uint_as_float(u[1]) * g1);
        }
        const int token = 8 * j + (lane & 7), f = lane >> 3;
        stmatrix_x4_trans(sbase + token * 64 + ((f ^ ((token >> 1) & 3)) << 4), p[0], p[1], p[2], p[3]);
    }
    if (rows >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && n0 < a.N) {
            tma_store_2d(&tY, stage, n0, row);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    const int f = lane & 3;
    if (n0 + 8 * f < a.N) {
        T* out = static_cast<T*>(a.out) + static_cast<int64_t>(row) * a.ldo + n0 + 8 * f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int token = 8 * i + (lane >> 2);
            if (token < rows)
                *reinterpret_cast<uint4*>(out + token * a.ldo) =
                    *reinterpret_cast<const uint4*>(stage + token * 64 + ((f ^ ((token >> 1) & 3)) << 4));
        }
    }
}

// ---------------------------------------------------- CTA-pair pipelines --
constexpr int kEpiWarps = 8;
constexpr int kEpiStage = kEpiWarps * 2048;  // the products' store staging
constexpr uint32_t kRaggedTimeout = 0x2u;  // MOE_DEVERR_TIMEOUT

// The barriers of a pipeline of S stages and two accumulators, and what a
// pair shares; the first 1 KB of shared memory.
template <int S>
struct PairBars {
    uint64_t full[S], empty[S], tail[S], tfull[2], tempty[2], join_full[kEpiWarps], join_free[kEpiWarps], drain;
    uint32_t tmem, abort;
};

// The value of lane 0 of a converged warp.  The compiler cannot see that what
// comes from memory is the same in every lane; told so, it keeps loop counters,
// descriptors and addresses of the issuing warps in uniform registers, which
// is where TMA and the MMAs take them from.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// A bounded wait of a converged warp; the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort,
                                          uint64_t limit_ns = kWaitLimitNs) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, limit_ns));
}
// The limit of a wait for a whole sum of that many steps, which may take longer
// than kWaitLimitNs: 2^30 rows of one group's weight gradient run for 4.4 s.  A
// step takes 0.26 us where its loads bound it.
__device__ __forceinline__ uint64_t sum_limit_ns(int64_t steps) {
    return kWaitLimitNs + static_cast<uint64_t>(steps) * 2000u;
}

struct Ring {  // stage and its parity
    int s = 0;
    uint32_t ph = 0;
    template <int S>
    __device__ __forceinline__ void next() {
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
    }
    template <int S>
    __device__ __forceinline__ Ring after() const {
        Ring r = *this;
        r.next<S>();
        return r;
    }
};

struct Acc {  // accumulator and its parity
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        i ^= 1;
        if (i == 0) ph ^= 1u;
    }
};

template <int S>
__device__ __forceinline__ void pair_start(PairBars<S>& b, uint32_t full_count, int warp, uint32_t joins = 1,
                                           uint32_t frees = 1) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(b.full + i, full_count);
            mbar_init(b.empty + i, 1);
            mbar_init(b.tail + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b.tfull + i, 1);
            mbar_init(b.tempty + i, 2 * kEpiWarps);  // every epilogue warp of both CTAs
        }
        for (int i = 0; i < kEpiWarps; ++i) {
            mbar_init(b.join_full + i, joins);  // the cluster's other pairs
            mbar_init(b.join_free + i, frees);
        }
        mbar_init(&b.drain, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    // tensor memory is taken only once the kernels before this one have
    // finished (and released theirs)
    pdl_wait();
    if (warp == 1) tmem_alloc_pair(&b.tmem, 512);
}

// Token rows as TMA boxes of 64 and 16 rows of 128 bytes.  (Boxes of 16 alone:
// 1.22 against 1.17 ms on the data gradient of a 64-expert layer, whose tiles
// are 200 to 250 rows; a map for every power of two saves loads that do not
// bound the kernels, and costs short calls the time to encode it.)
struct RowMaps {
    CUtensorMap box64, box16;
};
__device__ __forceinline__ void load_rows(uint32_t one, const RowMaps& m, uint8_t* dst, int x, int row, int rows,
                                          uint32_t full) {
    int i = 0;
    for (; i + 64 <= rows; i += 64) tma_load_2d_pair_if(one, dst + i * 128, &m.box64, x, row + i, full);
    for (; i < rows; i += 16) tma_load_2d_pair_if(one, dst + i * 128, &m.box16, x, row + i, full);
}
inline bool make_row_maps(RowMaps* m, const void* x, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_cols,
                          int dtype) {
    const uint64_t dims[2] = {cols, rows}, strides[1] = {stride};
    const uint32_t box64[2] = {box_cols, 64}, box16[2] = {box_cols, 16};
    return make_tensor_map(&m->box64, x, 2, dims, strides, box64, dtype) &&
           make_tensor_map(&m->box16, x, 2, dims, strides, box16, dtype);
}

__device__ __forceinline__ void pair_end(uint32_t tmem_base, int warp) {
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// The epilogue warps of the products (`ew` of kEpiWarps): a warp owns 32 of the
// CTA's 128 features (its tensor-memory lane quarter) and every other 32-token
// chunk of a tile.  Short sums leave little time per tile, so nothing waits in
// line: the next item and its routing weights are fetched while a tile is
// stored, a chunk is read from tensor memory while the one before it is
// stored, and the accumulator goes back before the last chunk's stores.
//
// With SP > 1 pairs in the cluster, each holds its part of the same sums: the
// others' warps write theirs (fp32, 4 KB per warp) into the first pair's shared
// memory (`join`), whose warps add them in the pairs' order and store.
template <typename T, int TN, int SP, int S, typename Scale>
__device__ __forceinline__ bool product_epilogue(const RaggedArgs& args, const CUtensorMap& tY,
                                                 const RaggedTiles& tiles, PairBars<S>& bars,
                                                 int panels, int total, int first, int stride, int steps,
                                                 uint32_t tmem_base, int ew, int lane, uint32_t rank, uint8_t* stage, float common,
                                                 Scale scale_of, uint8_t* join = nullptr) {
    constexpr int kChunks = (TN + 32) / 64;
    const int q = (threadIdx.x >> 5) & 3, odd = ew >> 2;
    const volatile uint32_t* abort_flag = &bars.abort;
    RaggedFeed feed;
    uint32_t join_ph = 0;
    RaggedItem it{};
    float gate[kChunks], scale = 1.0f;
    // item t, its scale and the routing weight of this lane's token of each
    // chunk; nothing is computed with them before they are needed
    auto fetch = [&](int t) {
        if (t >= total) return;
        it = feed.next(tiles, args.E, panels, total, t, stride, lane);
        scale = scale_of(it.e);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int token = odd * 32 + i * 64 + lane;
            gate[i] = args.row_scale && token < it.rows ? ld_dep(args.row_scale + it.row + token) : 1.0f;
        }
    };
    fetch(first);
    Acc acc;
    for (int t = first; t < total; t += stride) {
        if (!warp_wait(bars.tfull + acc.i, acc.ph, abort_flag, sum_limit_ns(steps))) {
            if (lane == 0) bulk_wait_all();
            return false;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc.i * TN);
        uint32_t v[2][2][16];
        auto load = [&](int i) {
            tmem_ld_frag32(taddr + odd * 32 + i * 64, v[i & 1][0]);
            tmem_ld_frag32(taddr + odd * 32 + i * 64 + (16u << 16), v[i & 1][1]);
        };
        const RaggedItem now = it;
        float g[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) g[i] = gate[i] * scale * common;
        const int n0 = now.panel * 256 + static_cast<int>(rank & 1) * 128 + q * 32;
        if (odd * 32 < now.rows) load(0);
        fetch(t + stride);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = odd * 32 + i * 64;
            tmem_ld_wait();
            if (c + 64 < now.rows && i + 1 < kChunks) {
                load(i + 1);
            } else if (c < now.rows || i == 0) {
                // the last read is complete; the MMA side reads nothing that
                // this warp stores, so the arrive need not release it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(bars.tempty + acc.i), rank & ~1u));
            }
            if (c >= now.rows) break;
            if constexpr (SP > 1) {
                static_assert(kChunks == 1, "one chunk per warp and tile");
                uint32_t* f = &v[0][0][0];
                const uint32_t pair = rank >> 1;
                if (pair > 0) {
                    // the first pair has read this warp's part of the last tile
                    bool ok = warp_wait(bars.join_free + ew, join_ph ^ 1u, abort_flag, sum_limit_ns(steps));
                    join_ph ^= 1u;
                    if (!ok) return false;
                    fence_cluster();
                    const uint32_t dst =
                        mapa_shared(smem_u32(join + ((pair - 1) * kEpiWarps + ew) * 4096), rank & 1u) + lane * 16;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_cluster_v4(dst + k * 512, __uint_as_float(f[4 * k]), __uint_as_float(f[4 * k + 1]),
                                      __uint_as_float(f[4 * k + 2]), __uint_as_float(f[4 * k + 3]));
                    fence_cluster();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_full + ew), rank & 1u));
                    break;
                }
                bool ok = warp_wait(bars.join_full + ew, join_ph, abort_flag, sum_limit_ns(steps));
                join_ph ^= 1u;
                if (!ok) {
                    if (lane == 0) bulk_wait_all();
                    return false;
                }
                fence_cluster();
#pragma unroll
                for (int o = 0; o < SP - 1; ++o) {
                    const float4* src = reinterpret_cast<const float4*>(join + (o * kEpiWarps + ew) * 4096) + lane;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 w = src[k * 32];
                        f[4 * k] = __float_as_uint(__uint_as_float(f[4 * k]) + w.x);
                        f[4 * k + 1] = __float_as_uint(__uint_as_float(f[4 * k + 1]) + w.y);
                        f[4 * k + 2] = __float_as_uint(__uint_as_float(f[4 * k + 2]) + w.z);
                        f[4 * k + 3] = __float_as_uint(__uint_as_float(f[4 * k + 3]) + w.w);
                    }
                }
                __syncwarp();
                if (lane == 0)
                    for (int o = 1; o < SP; ++o)
                        mbar_arrive_cluster(mapa_shared(smem_u32(bars.join_free + ew), rank + 2 * o));
            }
            store_transposed<T>(args, tY, v[i & 1], now.row + c, now.rows - c, n0, lane, g[i], stage);
        }
        acc.next();
    }
    if (lane == 0) bulk_wait_all();
    return true;
}

// Tensor map of the products' output: boxes of 32 features x 32 tokens.
inline bool make_out_map(CUtensorMap* m, const RaggedArgs& a, int dtype) {
    const uint64_t dims[2] = {static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.R)};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.ldo) * 2};
    const uint32_t box[2] = {32, 32};
    return make_tensor_map(m, a.out, 2, dims, strides, box, dtype, 64);
}

// Launches `kernel` (clusters of SP pairs) on as many clusters as the GPU has
// SMs for, but no more than there are items.
template <int SP = 1, typename... KArgs, typename... Args>
cudaError_t launch_pairs(void (*kernel)(KArgs...), int64_t items, int threads, int smem, bool (&ready)[kMaxDevices],
                         cudaStream_t stream, Args&&... args) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    const int64_t most = num_sms() / (2 * SP);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(2 * SP * (items < most ? items : most))), dim3(threads), smem,
                      stream, std::forward<Args>(args)...);
}

// Clusters of SP pairs of `kernel` that the GPU holds at once (a cluster stays
// inside one graphics processing cluster, so fewer than its SMs give); 0 if the
// query fails.  found: the answers per device, plus one.
template <int SP, typename K>
int64_t resident_clusters(K kernel, int threads, int smem, int (&found)[kMaxDevices]) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) return 0;
    if (!found[dev]) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 * SP;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * SP);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 0) {
            (void)cudaGetLastError();
            n = 0;
        }
        found[dev] = n + 1;
    }
    return found[dev] - 1;
}

// ---------------------------------------------------------- 4-bit values --
// Eight e2m1 codes (lowest nibble first) -> four pairs of f16; every e2m1 value
// is an f16 value.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t q, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
}
// The nearest e2m1 codes of eight values (v[0] in the lowest nibble), ties to
// even, saturating at +-6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// Power-of-two block scale 2^(code - 127); code 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7FC00000u : (code == 0u ? 0x00400000u : code << 23));
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(code));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

}  // namespace moe
