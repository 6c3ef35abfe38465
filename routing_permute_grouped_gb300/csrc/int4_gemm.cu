// int4_gemm.cu -- products of 16-bit rows with 4-bit weights, few rows to a group.
//
//   y[r] = row_scale[r] * x[src[r] / div] W[e]^T   for the rows r of group e
// with W[e][n][k] = (code - zero) * scale, scale and zero per row n and group of
// k.  code - zero is a small integer, exact in 16 bits, so the tensor cores sum a
// group's products as they are, and each group's sum is scaled once, in fp32.
//
// Few token rows: the weights' bytes set the pace, and what has to keep up with
// them is the widening of the codes.  So no weight is handed from warp to warp: a
// warp streams 32 weight rows (with SwiGLU 16 of gate and the same 16 of up), with
// their scales and zero points, by cp.async into a ring of its own, a step of 128
// elements (256 for groups of 128) ahead, widens them in registers as the A operand of
// mma.m16n8k16 and multiplies them by up to 8 token rows, whose B operands it reads
// from two blocks of token rows that the CTA's 8 warps share.  Two CTAs to an SM.
// (The same product with the widened weights written to tensor memory for
// tcgen05.mma, int4_wide.cu, spends as much again on handing chunks on: 2 rows in
// each of 220 groups of 7168 x 2048 545 us, here 330.)
//
// That decode batch reads 1.72 GB at 5.2 TB/s, 78 % of a copy's rate.  Its loads alone
// take 287 us and its arithmetic alone 291: 298 instructions for 32 x 128 weights, 60 % of
// the issue slots with the 16 warps that the registers leave.  Measured on the way there:
// or-ing the codes into a mantissa, three shifts instead of one, 306 instructions;
// scales and zero points through L1 instead of shared memory 385 us; token rows through
// L1 420; three CTAs to an SM spill.
//
// The order of k inside a group is free as long as both operands share it: a lane
// takes whole 32-bit words, and one word's eight elements are its part of two
// steps of 16.  All of a step's elements lie in one group of scales, so a lane's
// part is 4, 2 or 1 words for groups of 128, 64 or 32.
//
// Few items: the warps of a CTA split the sum and add their parts in order.
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/moe.h"
#include "int4.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kChunk = 128;   // elements of the sum that a lane's four words and its neighbours' make
constexpr int kStages = 2;    // steps of a warp's codes in shared memory

constexpr int kWarps = 8;     // of a CTA, two CTAs to an SM
constexpr int kTile = 8;      // token rows of an item, at most
constexpr int kRowBytes = 18 * 1024;  // of a block of token rows

// d (+)= a b on 16 weight rows, 8 token rows and 16 elements
template <typename T, bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define MOE_MMA(type)                                                                                                     \
    if constexpr (FIRST)                                                                                                  \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};" \
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                              \
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));                                   \
    else                                                                                                                  \
        asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};" \
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                              \
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
    if constexpr (std::is_same_v<T, __half>) {
        MOE_MMA("f16");
    } else {
        MOE_MMA("bf16");
    }
#undef MOE_MMA
}

// Where piece `piece` (16 bytes) of a token row's 256 bytes of a chunk lies: eight
// lanes that read their B operands together (two rows, four pieces) meet no bank twice.
template <int WORDS>
__device__ __forceinline__ int row_place(int row, int piece) {
    if (WORDS == 4) piece = (piece & 3) << 2 | piece >> 2;
    return piece ^ (WORDS == 2 ? row & 1 : (row & 1) << 2);
}

template <typename T, int G>
struct Warp {
    static constexpr int parts = kChunk / G, words = 4 / parts;  // groups of a chunk, words of a lane in each
    static constexpr int halves = G == 128 ? 2 : 1;              // chunks of a step
    static constexpr int groups = halves * parts, step = halves * kChunk;
    // of a step: codes, then scales and (four bytes with) zero points of a row per lane
    static constexpr int code_bytes = halves * 32 * 64, stage_bytes = code_bytes + 32 * (2 * groups + 4);
    const Int4Product& p;
    const uint8_t* codes[4];  // this lane's 16 bytes of the next step's first chunk, of its four weight rows
    const uint16_t* scales;   // of the weight row lane % 4 of the four
    const uint8_t* zeros;
    uint32_t put, get, par, par_zero;  // this lane's places in the first of the warp's stages
    int lane, t4;             // lane % 4

    // 32 rows x 64 bytes of every chunk; a row's 16-byte pieces in an order that its
    // number gives, so that reading one piece of eight rows meets no bank twice.
    // left: bytes of the row from the lane's first on.  Past its end any codes will
    // do (its last ones), with token rows that read as zero.
    __device__ __forceinline__ void load(uint32_t stage, int left) const {
#pragma unroll
        for (int h = 0; h < halves; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async_16(put + stage + 2048 * h + 512 * i, codes[i] + min(h * 64, left - 16), 16);
    }
    __device__ __forceinline__ void load_whole(uint32_t stage) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < halves; ++h) cp_async_16(put + stage + 2048 * h + 512 * i, codes[i] + h * 64, 16);
    }
    // The lane's words of group j of the chunk, in rows lane / 4 + 8 i.
    __device__ __forceinline__ void codes_of(uint32_t stage, int j, uint32_t (&q)[4][words]) const {
        uint32_t at = get + stage;
        if constexpr (words == 2) at ^= j << 5;
        if constexpr (words == 1) at ^= j << 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (words == 4)
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(q[i][0]), "=r"(q[i][1]), "=r"(q[i][2]), "=r"(q[i][3])
                             : "r"(at + 512 * i)
                             : "memory");
            else if constexpr (words == 2)
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(q[i][0]), "=r"(q[i][1]) : "r"(at + 512 * i) : "memory");
            else
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q[i][0]) : "r"(at + 512 * i) : "memory");
        }
    }
    // Scales and zero points of step c come by way of shared memory as well, where they
    // can be copied four bytes at a time (`whole`); else they are read as they are
    // needed, with a scale of 0 past the last group, where the sums are 0 (an infinite
    // scale of the last one would make them NaN).
    __device__ __forceinline__ void load_params(uint32_t stage, int c) const {
        const int at = min(c * groups, p.groups - groups);
        const uint32_t dst = par + stage;
        if constexpr (groups == 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(scales + at) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(scales + at) : "memory");
        if (p.zeros)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(par_zero + stage), "l"(zeros + (at & ~3)) : "memory");
    }
    __device__ __forceinline__ void params(uint32_t stage, int c, float (&scale)[groups], uint32_t (&zero)[groups]) const {
        uint32_t s[groups], z[groups];
        if (p.whole) {
            const uint32_t at = par + stage;
            uint32_t v[groups / 2], w = 0x08080808u;
            if constexpr (groups == 4)
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at) : "memory");
            else
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(at) : "memory");
            if (p.zeros) {
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(par_zero + stage) : "memory");
                if constexpr (groups == 2) w >>= (min(c * groups, p.groups - groups) & 2) * 8;
            }
#pragma unroll
            for (int j = 0; j < groups; ++j) {
                s[j] = v[j / 2] >> (16 * (j & 1)) & 0xFFFFu;
                z[j] = w >> (8 * j) & 0xFFu;
            }
        } else {
#pragma unroll
            for (int j = 0; j < groups; ++j) {
                const int at = min(c * groups + j, p.groups - 1);
                s[j] = at < c * groups + j ? 0u : scales[at];
                z[j] = p.zeros ? zeros[at] : 8u;
            }
        }
#pragma unroll
        for (int j = 0; j < groups; ++j) {
            scale[j] = to_float<T>(__builtin_bit_cast(T, static_cast<uint16_t>(s[j])));
            zero[j] = int4_zero<T>(z[j]);
        }
    }

    // sum[m]: 16 weight rows m by 8 token rows; x: the step's first element of this lane's
    // token row in shared memory, 256 bytes for a chunk, pieces placed by row_place
    __device__ __forceinline__ void take(uint32_t stage, uint32_t x, int odd, const float (&scales_)[groups],
                                         const uint32_t (&zeros_)[groups], float (&sum)[2][4]) const {
        uint4 ahead;
        auto fetch = [&](int w) {  // the lane's word w of the step
            const int at = w / 4 * 256 + (row_place<words>(0, (w % 4 / words * 4 + t4) * words + w % words) << 4 ^ odd);
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(ahead.x), "=r"(ahead.y), "=r"(ahead.z), "=r"(ahead.w)
                         : "r"(x + at)
                         : "memory");
        };
        fetch(0);
#pragma unroll
        for (int hj = 0; hj < groups; ++hj) {
            const int half = hj / parts, j = hj % parts;
            float scale[4];
            uint32_t zero[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                scale[i] = __shfl_sync(kAll, scales_[hj], (lane & ~3) | i);
                zero[i] = __shfl_sync(kAll, zeros_[hj], (lane & ~3) | i);
            }
            uint32_t q[4][words];
            codes_of(stage + 2048 * half, j, q);
            float part[2][4];
#pragma unroll
            for (int u = 0; u < words; ++u) {
                const uint4 b = ahead;
                if (hj * words + u + 1 < groups * words) fetch(hj * words + u + 1);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t a[4];
                        a[0] = int4_widen<T>(q[2 * m][u], 2 * h, zero[2 * m]);
                        a[1] = int4_widen<T>(q[2 * m + 1][u], 2 * h, zero[2 * m + 1]);
                        a[2] = int4_widen<T>(q[2 * m][u], 2 * h + 1, zero[2 * m]);
                        a[3] = int4_widen<T>(q[2 * m + 1][u], 2 * h + 1, zero[2 * m + 1]);
                        if (u == 0 && h == 0)
                            mma<T, true>(part[m], a, b.x, b.y);
                        else
                            mma<T, false>(part[m], a, h ? b.z : b.x, h ? b.w : b.y);
                    }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[m][i] = fmaf(part[m][i], scale[2 * m + (i >> 1)], sum[m][i]);
        }
    }
};

struct Shared {
    Int4Lists lists;
    uint64_t full[2], empty[2];  // blocks of token rows
    int from[2][kTile];            // an item's token rows
    uint32_t abort;
};

template <typename T, int G>
__device__ __forceinline__ void run_item(const Int4Product& p, const Int4Item& it, Shared& sh, uint8_t* ring, uint8_t* s_rows,
                                         int& blocks_so_far, int& turn_of, bool& timed_out) {
    using W = Warp<T, G>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    // Set once a wait of the CTA has run out: the other warps' waits end as well, and no sum is
    // stored any more.  (Leaving the blocks and items there and then: decode 330 -> 336 us, for
    // registers.)
    volatile uint32_t* abort_flag = &sh.abort;
    const int split = p.split, part = warp & (split - 1), block = it.panel * (kWarps / split) + warp / split;
    // the warp's weight rows: 16 from a on and 16 from b on
    const int a0 = p.swiglu ? (block >> 3) * 256 + (block & 7) * 16 : block * 32, b0 = a0 + (p.swiglu ? 128 : 16);
    const bool live = a0 < p.r.N;
    const int64_t first = static_cast<int64_t>(it.e) * p.r.N + g;
    // N is a multiple of 8: rows past the last one are read as others, and not stored
    auto row = [&](int i) {
        const int r = i < 2 ? a0 + 8 * i : b0 + 8 * (i - 2);
        return first + (r < p.r.N ? r : live ? a0 : 0);
    };
    const int* from = sh.from[turn_of & 1];  // of the item before the last one no one reads any more
    if (threadIdx.x < it.rows) sh.from[turn_of & 1][threadIdx.x] = max(int4_token_row(p, it.row + threadIdx.x), 0);
    ++turn_of;
    __syncthreads();
    // Token rows, in blocks of `columns` elements, two in shared memory.  Columns of the
    // product past the item's rows are not stored: any row will do for them.
    const int held = it.rows > 4 ? 8 : it.rows > 2 ? 4 : it.rows;  // rows with a place
    const int super = split * W::step, supers = (p.r.K + super - 1) / super;
    const int each = min(supers, kRowBytes / (held * 2) / super), columns = each * super;
    const int n_blocks = (supers + each - 1) / each;
    auto load_rows = [&](int b) {
        const int use = blocks_so_far + b, buf = use & 1;
        timed_out = timed_out || !warp_wait(sh.empty + buf, (use >> 1 & 1) ^ 1, &sh.abort);
        if (timed_out) *abort_flag = 1;  // before what comes may lie over rows that others read
        const uint32_t dst = smem_u32(s_rows) + buf * kRowBytes;
        const int piece = threadIdx.x & 15, slot = threadIdx.x >> 4, chunks = columns / kChunk;
        auto copy = [&](int r, int c) {  // chunk c of row r
            const int k = b * columns + c * kChunk + piece * 8;
            const bool in = k < p.r.K;
            cp_async_16(dst + (r * chunks + c) * 256 + (row_place<W::words>(r, piece) << 4),
                        static_cast<const T*>(p.x) + (from[r] * p.ldx + (in ? k : 0)), in ? 16 : 0);
        };
        for (int c = slot; c < chunks; c += 2 * kWarps)
            for (int r = 0; r < it.rows; ++r) copy(r, c);
        cp_async_arrive(sh.full + buf);
    };
    W w{p};
#pragma unroll
    for (int i = 0; i < 4; ++i) w.codes[i] = p.codes + row(i) * (p.r.K / 2) + part * (W::step / 2) + t4 * 16;
    w.scales = static_cast<const uint16_t*>(p.scales) + row(t4) * p.groups;
    w.zeros = p.zeros + row(t4) * p.groups;
    const uint32_t stages = smem_u32(ring + warp * kStages * W::stage_bytes), mine = stages + g * 64;
    w.par = stages + W::code_bytes + lane * 2 * W::groups;
    w.par_zero = stages + W::code_bytes + 64 * W::groups + lane * 4;
    const int turn = g >> 1 & 3;
    w.put = mine + ((t4 ^ turn) << 4);
    w.get = W::words == 4 ? w.put : W::words == 2 ? mine + (((t4 >> 1) ^ turn) << 4) + (t4 & 1) * 8 : mine + (turn << 4) + t4 * 4;
    w.lane = lane;
    w.t4 = t4;
    const int steps = (p.r.K + W::step - 1) / W::step;
    int ahead = part;  // the next step to load
    auto load = [&](uint32_t stage) {
        if (ahead < steps) {
            if ((ahead + 1) * W::step <= p.r.K)
                w.load_whole(stage);
            else
                w.load(stage, p.r.K / 2 - ahead * (W::step / 2) - t4 * 16);
            if (p.whole) w.load_params(stage, ahead);
        }
        cp_async_commit();
        ahead += split;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.codes[i] += split * (W::step / 2);
    };
    load_rows(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i * W::stage_bytes);
    float sum[2][4] = {};
    uint32_t stage = 0;
    const int mine_of = g & (held - 1), odd = row_place<W::words>(mine_of, 0) << 4;
    for (int b = 0; b < n_blocks; ++b) {
        if (b + 1 < n_blocks) load_rows(b + 1);
        const int use = blocks_so_far + b, buf = use & 1;
        timed_out = timed_out || !warp_wait(sh.full + buf, use >> 1 & 1, &sh.abort);
        if (timed_out) *abort_flag = 1;
        uint32_t x = smem_u32(s_rows) + buf * kRowBytes + mine_of * columns * 2 + part * (W::step * 2);
        const int end = min((b + 1) * each * split, steps);
        for (int c = b * each * split + part; c < end; c += split) {
            cp_async_wait<kStages - 2>();
            __syncwarp();  // every lane's copies, and the reads of the stage that is filled next
            load(stage == 0 ? (kStages - 1) * W::stage_bytes : stage - W::stage_bytes);
            float s[W::groups];
            uint32_t z[W::groups];
            w.params(stage, c, s, z);
            w.take(stage, x, odd, s, z, sum);
            x += super * 2;
            stage = stage == (kStages - 1) * W::stage_bytes ? 0 : stage + W::stage_bytes;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.empty + buf);
    }
    blocks_so_far += n_blocks;
    // the codes were widened in units of their own
#pragma unroll
    for (int v = 0; v < 8; ++v) (&sum[0][0])[v] *= 1.0f / Int4Wide<T>::unit;
    __syncwarp();  // the next item's copies come after these reads
    if (split > 1) {  // the parts to the first of the warps, in order, through the ring's memory
        float* join = reinterpret_cast<float*>(ring);
        cp_async_wait<0>();
        __syncthreads();
        if (part > 0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) join[(warp * 8 + v) * 32 + lane] = (&sum[0][0])[v];
        }
        __syncthreads();
        if (part == 0)
            for (int o = 1; o < split; ++o)
#pragma unroll
                for (int v = 0; v < 8; ++v) (&sum[0][0])[v] += join[((warp + o) * 8 + v) * 32 + lane];
        __syncthreads();
        if (part > 0) return;
    }
    if (!live || *abort_flag) return;
    // lane: token rows 2 t4 and 2 t4 + 1, weight rows g and g + 8 of each 16
    T* out = static_cast<T*>(p.r.out);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int token = 2 * t4 + j, to = it.row + token;
        if (token >= it.rows) continue;
        const float f = p.r.row_scale ? ld_dep(p.r.row_scale + to) : 1.0f;
        const bool none = p.src && int4_token_row(p, to) < 0;
        T* y = out + to * p.r.ldo;
        if (p.swiglu) {
            const int col = block * 16 + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float gate = sum[0][2 * h + j];
                const float v = gate / (1.0f + expf(-gate)) * sum[1][2 * h + j] * f;
                y[col + 8 * h] = from_float<T>(none ? 0.0f : v);
            }
        } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = a0 + 16 * m + 8 * h + g;
                    if (col < p.columns) y[col] = from_float<T>(none ? 0.0f : sum[m][2 * h + j] * f);
                }
        }
    }
}

template <typename T, int G>
__global__ void __launch_bounds__(32 * kWarps, 2) k_int4_product(const __grid_constant__ Int4Product p) {
    __shared__ Shared sh;
    extern __shared__ __align__(128) uint8_t ring[];
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.full + i, 32 * kWarps);
            mbar_init(sh.empty + i, kWarps);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    pdl_wait();
    const int blocks = (p.r.N + 31) / 32, per = kWarps / p.split, panels = (blocks + per - 1) / per;
    const int total = int4_lists<kTile, 1>(p.r, sh.lists, panels);
    uint8_t* rows = ring + kWarps * kStages * Warp<T, G>::stage_bytes;
    int blocks_so_far = 0, turn_of = 0;  // blocks of token rows, items
    bool timed_out = false;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Int4Item it = int4_item(sh.lists, p.r.E, panels, t);
        run_item<T, G>(p, it, sh, ring, rows, blocks_so_far, turn_of, timed_out);
    }
    cp_async_commit();
    cp_async_wait<0>();  // nothing may still be written to shared memory at exit
    if (timed_out && p.r.status) atomicOr(p.r.status, kRaggedTimeout);
}

// Warps that split a sum, as far as the token rows of their steps fit a block: the
// number that makes the fewest steps of the CTAs that run one after another, an item's
// start and end counted as kItemSteps.
// One token on 8 experts of 4096 x 7168, by split 1, 2 and 4: 47, 43 and 45 us (events
// around single calls; 40 back to back); one row of 1024 x 4096, by 1 and 8: 35 and 12.
constexpr int kItemSteps = 4;
int split_of(int64_t blocks, int64_t tiles, int64_t rows, int steps, int step) {
    const int held = rows > 4 ? 8 : rows > 2 ? 4 : static_cast<int>(rows);  // of the longest tile
    int best = 1;
    int64_t least = INT64_MAX;
    for (int split = 1; split <= kWarps && (split == 1 || split * held * step * 2 <= kRowBytes); split *= 2) {
        const int64_t items = (blocks * split + kWarps - 1) / kWarps * tiles, ctas = 2 * num_sms();
        const int64_t cost = (items + ctas - 1) / ctas * ((steps + split - 1) / split + kItemSteps);
        if (cost < least) least = cost, best = split;
    }
    return best;
}

template <typename T, int G>
cudaError_t launch(const Int4Product& q, cudaStream_t st) {
    using W = Warp<T, G>;
    constexpr int kSmem = kWarps * kStages * W::stage_bytes + 2 * kRowBytes;
    static_assert(2 * (kSmem + static_cast<int>(sizeof(Shared)) + 1024 + 64) <= 233472, "shared memory budget");
    Int4Product p = q;
    const int64_t blocks = (p.r.N + 31) / 32;
    const int64_t tiles = p.r.R / kTile + (p.r.R < p.r.E ? p.r.R : p.r.E);  // at most
    p.split = split_of(blocks, tiles, p.r.R, (p.r.K + W::step - 1) / W::step, W::step);
    p.whole = p.groups % (p.zeros ? 4 : W::groups) == 0 && (reinterpret_cast<uintptr_t>(p.scales) & (2 * W::groups - 1)) == 0 &&
              (reinterpret_cast<uintptr_t>(p.zeros) & 3) == 0;
    const int64_t per = kWarps / p.split, items = (blocks + per - 1) / per * tiles, most = 2 * num_sms();
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_int4_product<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_pdl(k_int4_product<T, G>, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(32 * kWarps),
                      kSmem, st, p);
}

template <typename T>
cudaError_t product(int group, const Int4Product& p, cudaStream_t st) {
    // Wide tiles read a group's weights once for up to 64 rows, but need more rows than a
    // narrow tile's 8, and enough work: their warps hand every chunk on, 20 us at least.
    // Narrow and wide, in us: 8 rows in each of 32 groups of 7168 x 2048 59 and 92, 12 rows
    // 104 and 94, 32 rows 203 and 104; 16 rows in 4 groups of 1024 x 7168 (2^29 products)
    // 20 and 27, 16 rows in 8 groups of 7168 x 2048 (2^31) 39 and 35, 64 rows of 1024 x 16384
    // (2^30) 39 and 31.  E counts groups without rows, which the host cannot tell: 2000 rows in
    // 8 groups of 2048 x 4096 take 80 us, the same rows where those are 8 of 256 groups 229, in
    // narrow tiles, and 2100 rows there 104, in wide ones.
    if (p.r.R > 8ll * p.r.E && static_cast<double>(p.r.R) * p.r.N * p.r.K >= 0x1p30) return launch_int4_wide<T>(group, p, st);
    if (group == 32) return launch<T, 32>(p, st);
    return group == 64 ? launch<T, 64>(p, st) : launch<T, 128>(p, st);
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm_int4(int32_t group, int32_t dtype, int64_t R, int32_t N, int32_t K, int32_t E,
                                              const void* x, int64_t x_rows, int64_t ldx, const int32_t* src,
                                              int32_t src_div, const void* w_codes, const void* w_scales,
                                              const void* w_zeros, const int32_t* offsets, const float* row_scale,
                                              int32_t swiglu, void* y, int64_t ldy, uint32_t* status, void* stream) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    const moe_status_t s = static_cast<moe_status_t>(check_int4_row(group, K));
    if (s != MOE_OK) return s;
    if (R < 0 || N <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (N % (swiglu ? 128 : 8))
        return set_last_error(MOE_ERR_UNSUPPORTED, "N = %d is not a multiple of %d", N, swiglu ? 128 : 8);
    if (N > kRaggedMaxDim / 2) return set_last_error(MOE_ERR_UNSUPPORTED, "N = %d is more than 2^29", N);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    if (R == 0) return MOE_OK;
    if (!x || !w_codes || !w_scales || (!offsets && E != 1) || !y)
        return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(y, 16) || !aligned(w_scales, 2))
        return set_last_error(MOE_ERR_INVALID_ARG, "x, w_codes and y must be 16-byte aligned, w_scales 2-byte");
    if (ldx < K || ldx % 8 || ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "row strides must cover the row and be multiples of 8 elements");
    if (ldx > kRaggedMaxDim || ldy > kRaggedMaxDim)
        return set_last_error(MOE_ERR_UNSUPPORTED, "a row stride is more than 2^30");
    if (src ? (src_div <= 0 || x_rows <= 0) : x_rows < R)
        return set_last_error(MOE_ERR_INVALID_ARG, "x has too few rows, or src_div <= 0");
    Int4Product p{};
    p.r.offsets = offsets;
    p.r.R = static_cast<int32_t>(R);
    p.r.N = swiglu ? 2 * N : N;
    p.r.K = K;
    p.r.E = E;
    p.r.row_scale = row_scale;
    p.r.out = y;
    p.r.ldo = ldy;
    p.r.status = status;
    p.x = x;
    p.ldx = ldx;
    p.x_rows = static_cast<int32_t>(x_rows < INT32_MAX ? x_rows : INT32_MAX);
    p.columns = N;
    p.swiglu = swiglu != 0;
    p.src = src;
    p.src_div = src_div;
    p.codes = static_cast<const uint8_t*>(w_codes);
    p.scales = w_scales;
    p.zeros = static_cast<const uint8_t*>(w_zeros);
    p.groups = (K + group - 1) / group;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == MOE_DTYPE_BF16 ? product<__nv_bfloat16>(group, p, st)
                                                  : product<__half>(group, p, st);
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit weight product: %s", cudaGetErrorString(e));
}
