// Projection in 8-bit integers with a scale per token and per output channel:
//   out[n][o] = (sum_k x8[n][k] w8[o][k]) x_scale[n] w_scale[o]
// on tcgen05 (kind::i8, 32-bit integer accumulators).  |sum| <= 65,536 x 128^2
// = 2^30, so the sum is exact, in any order.  Both operands are K-major bytes,
// read by TMA in chunks of 128 columns (128-byte swizzle); columns past d_in,
// rows past n_tok and d_out read as zero.
//
// Two kernels:
//  * split: few tokens, or few tiles.  Bound by the weights' bytes at decode
//    sizes.  A CTA takes 128 channels (MMA M) against up to 256 tokens (MMA N);
//    the K axis is cut over the CTAs of a cluster, so that every SM streams
//    weights even where there are fewer tiles than SMs, and the partial sums
//    meet in distributed shared memory: no workspace, no second launch.
//  * wide: many tokens.  Persistent clusters of two CTAs issue cta_group::2 MMAs
//    of 256 tokens x 256 channels (each SM supplies half of each operand); two
//    accumulators in tensor memory let the epilogue of one tile run under the
//    MMAs of the next.  Bound by what L2 delivers to the SMs: 2,048 tokens
//    through 1,536 x 24,576 take 57 us, 617 MB of operand tiles at 10.8 TB/s,
//    the tensor pipe 75 % busy while its SM works (ncu).

#include <cuda.h>

#include "common.cuh"
#include "layer.h"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace mla {
namespace {

constexpr int kSms = 148;
constexpr uint32_t kChunk = 128;                 // columns (bytes) of one K chunk
constexpr uint32_t kOpBytes = 128 * kChunk;      // a chunk of 128 operand rows (16 KB)

// An int8 matrix, rows row_bytes apart, in boxes of 128 columns x box_rows.
bool make_map_i8(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t row_bytes,
                 uint32_t box_rows) {
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {kChunk, box_rows};
    return encode_tiled_cached(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
}

// The bound of every mbarrier wait, and the test hook's withheld load.
struct WaitBound {
    uint64_t timeout_ns;
    int withhold;   // 1: the first CTA (or pair) never issues its first load of the activations
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             int32_t* status, const WaitBound& bound) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait_suspend(bar, parity, 100000)) {
        if (*abort_flag) return false;
        if (ptx::global_timer_ns() - t0 > bound.timeout_ns) {
            *abort_flag = 1;
            raise_status(status, MLA_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// after an abort: copies still in flight get time to land before shared memory is released
__device__ __forceinline__ void settle_copies(volatile int* abort_flag) {
    if (!*abort_flag) return;
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 200000ull) {
    }
}

__device__ __forceinline__ float scaled(int sum, float sx, float sw) { return static_cast<float>(sum) * sx * sw; }

// ---------------------------------------------------------------------------
// split
// ---------------------------------------------------------------------------

// Dynamic shared memory at which blocks with `cols` columns of tensor memory
// fill the SM's shared memory (1 KB of it reserved per block) no later than its
// 512 columns, alone or mixed with others that keep to this.
constexpr size_t kSmSmem = 233472;
constexpr size_t tmem_share(uint32_t cols) { return kSmSmem / 512 * cols - 1024; }

constexpr int kSplitThreads = 256;
constexpr int kMaxCluster = 8;
// A CTA's ring at most (shorter where K is): with one CTA per SM, with two
constexpr uint32_t kSplitRing = 200 * 1024;
constexpr uint32_t kSplitRingHalf = 108 * 1024;

struct SplitArgs {
    CUtensorMap tm_w;   // w8 [d_out][d_in], boxes 128 x 128
    CUtensorMap tm_x;   // x8 [n_tok][d_in], boxes 128 x nt
    const float* x_scale;
    const float* w_scale;
    uint16_t* out;
    int32_t* status;
    int n_tok, d_out, nt, chunks, stages;
    uint32_t idesc, tmem_cols, ring_bytes;
    WaitBound bound;
};

__global__ void __launch_bounds__(kSplitThreads) linear_i8_split_kernel(const __grid_constant__ SplitArgs p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const int S = p.stages;
    const uint32_t stage_bytes = kOpBytes + static_cast<uint32_t>(p.nt) * kChunk;
    const uint32_t bars = sbase + p.ring_bytes;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (S + s); };
    const uint32_t done = bars + 8 * (2 * S);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.ring_bytes + 8 * (2 * S + 1));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.ring_bytes + 8 * (2 * S + 1) + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = static_cast<int>(ptx::cluster_size()), rank = static_cast<int>(ptx::cluster_rank());
    const int o0 = static_cast<int>(blockIdx.x) / parts * 128, n0 = blockIdx.y * p.nt;
    const int c0 = static_cast<int>(static_cast<long>(p.chunks) * rank / parts);
    const int c1 = static_cast<int>(static_cast<long>(p.chunks) * (rank + 1) / parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    // The weights' first chunks on their way into L2 while the kernel before
    // this one still runs (a prefetch changes no data, and L2 is coherent with
    // that kernel's writes, so it may precede the wait).
    if (warp == 0) {
        if (lane == 0) {
            ptx::prefetch_tmap(&p.tm_w);
            ptx::prefetch_tmap(&p.tm_x);
        }
        if (c0 + lane < c1 && lane < S)
            ptx::tma_prefetch_2d(&p.tm_w, static_cast<int>(kChunk) * (c0 + lane), o0);
    }
    if (warp == 1) {
        ptx::tmem_alloc1(ptx::smem_u32(tmem_slot), p.tmem_cols);
        ptx::tmem_relinquish1();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();   // the codes come from earlier kernels; the output may still be read by them

    if (warp == 0) {
        // chunk c into stage c mod S; a thread's copies run one after another,
        // so consecutive stages come from different threads
        for (int c = 0; c < c1 - c0; ++c) {
            const int s = c % S;
            bool ok = true;
            if (lane == (c & 7)) {
                ok = wait_bounded(empty(s), ((c / S) & 1) ^ 1, abort_flag, p.status, p.bound);
                if (ok) {
                    const uint32_t st = sbase + s * stage_bytes;
                    const int k = static_cast<int>(kChunk) * (c0 + c);
                    ptx::mbar_arrive_expect_tx(full(s), stage_bytes);
                    ptx::tma_load_2d(st, &p.tm_w, k, o0, full(s));
                    const bool withheld = c == 0 && (blockIdx.x | blockIdx.y) == 0 && p.bound.withhold;
                    if (!withheld) ptx::tma_load_2d(st + kOpBytes, &p.tm_x, k, n0, full(s));
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
        }
    } else if (warp == 1) {
        bool ok = true;
        for (int c = 0; c < c1 - c0 && ok; ++c) {
            const int s = c % S;
            ok = __all_sync(0xffffffffu, wait_bounded(full(s), (c / S) & 1, abort_flag, p.status, p.bound));
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                const uint32_t st = sbase + s * stage_bytes;
                const uint64_t a = ptx::smem_desc_sw128(st, 16, 1024), b = ptx::smem_desc_sw128(st + kOpBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma1_i8_ss(tmem, a + ((32 * kk) >> 4), b + ((32 * kk) >> 4), p.idesc, (c | kk) ? 1u : 0u);
                ptx::mma1_commit(empty(s));
            }
            __syncwarp();
        }
        // completes when every MMA issued above has (also on the abort path)
        if (ptx::elect_one()) ptx::mma1_commit(done);
    }
    __syncwarp();
    wait_bounded(done, 0, abort_flag, p.status, p.bound);
    settle_copies(abort_flag);
    __syncthreads();   // every copy into the ring has landed and been read
    griddep_launch_dependents();

    // Partial sums to shared memory as [token][128 channels] (a warp writes 32
    // consecutive channels), then the cluster's CTAs share the outputs: each
    // adds its vectors of four channels over all parts.  A thread keeps its
    // four channels, and takes kOutStep tokens at a time: one at a time, and
    // with 128 threads, this took longer than the product of 256 tokens.
    int* part = reinterpret_cast<int*>(smem);
    const int valid = min(p.nt, p.n_tok - n0);
    ptx::tc_fence_after();
    for (int j0 = 16 * (warp >> 2); j0 < valid; j0 += 32) {
        uint32_t r[16];
        ptx::tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + j0, r);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(j0 + j) * 128 + (threadIdx.x & 127)] = static_cast<int>(r[j]);
    }
    const int c4 = 4 * lane, o = o0 + c4;
    const bool in = o < p.d_out;
    float sw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sw[k] = in ? p.w_scale[o + k] : 0.f;
    ptx::tc_fence_before();
    ptx::cluster_sync();
    constexpr int kOutStep = 4, kWarps = kSplitThreads / 32;
    const int stride = parts * kWarps;   // tokens between a warp's
    for (int j = rank * kWarps + warp; j < valid; j += kOutStep * stride) {
        int4 sum[kOutStep];
        float sx[kOutStep];
#pragma unroll
        for (int u = 0; u < kOutStep; ++u) {
            sum[u] = make_int4(0, 0, 0, 0);
            sx[u] = j + u * stride < valid ? p.x_scale[n0 + j + u * stride] : 0.f;
        }
        for (int q = 0; q < parts; q += 2) {
            int4 v[2][kOutStep];   // two parts of all the tokens requested together
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int u = 0; u < kOutStep; ++u)
                    v[w][u] = q + w < parts && j + u * stride < valid
                                  ? ptx::ld_cluster_int4(ptx::map_to_rank(
                                        sbase + 512u * static_cast<uint32_t>(j + u * stride) + 16u * lane, q + w))
                                  : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int u = 0; u < kOutStep; ++u)
                    sum[u].x += v[w][u].x, sum[u].y += v[w][u].y, sum[u].z += v[w][u].z, sum[u].w += v[w][u].w;
        }
#pragma unroll
        for (int u = 0; u < kOutStep; ++u)
            if (in && j + u * stride < valid)
                *reinterpret_cast<uint2*>(p.out + static_cast<size_t>(n0 + j + u * stride) * p.d_out + o) =
                    make_uint2(pack_bf16x2(scaled(sum[u].x, sx[u], sw[0]), scaled(sum[u].y, sx[u], sw[1])),
                               pack_bf16x2(scaled(sum[u].z, sx[u], sw[2]), scaled(sum[u].w, sx[u], sw[3])));
    }
    ptx::cluster_sync();   // the other CTAs have read this one's sums
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc1(tmem, p.tmem_cols);
}

// ---------------------------------------------------------------------------
// wide
// ---------------------------------------------------------------------------

constexpr int kWideThreads = 320;                // loads, MMAs, 8 x epilogue
constexpr int kWideStages = 6;
constexpr uint32_t kWideStage = 2 * kOpBytes;    // this CTA's 128 tokens and 128 channels
constexpr uint32_t kOffStage = kWideStages * kWideStage;       // epilogue staging: 4 KB per warp
constexpr uint32_t kOffScales = kOffStage + 8 * 4096;      // the tile's 256 channel scales
constexpr uint32_t kOffWideBars = kOffScales + 1024;
enum { W_FULL = 0, W_EMPTY = W_FULL + kWideStages, W_ACC_FULL = W_EMPTY + kWideStages, W_ACC_FREE = W_ACC_FULL + 2,
       W_DRAIN = W_ACC_FREE + 2, W_BARS = W_DRAIN + 1 };
constexpr uint32_t kWideSmem = 232448;   // all of it, with all of the tensor memory
static_assert(kOffWideBars + 8 * W_BARS + 16 + 1024 <= kWideSmem && kWideSmem >= tmem_share(512), "shared memory budget");

struct WideArgs {
    CUtensorMap tm_x;     // x8 [n_tok][d_in], boxes 128 x 128
    CUtensorMap tm_w;     // w8 [d_out][d_in], boxes 128 x 128
    CUtensorMap tm_out;   // out [n_tok][d_out] bf16, boxes 64 x 32 (stores)
    CUtensorMap tm_w_cut; // w8, boxes 128 x (128 / cut)
    const float* x_scale;
    const float* w_scale;
    int32_t* status;
    int n_tok, d_out, chunks, m_tiles;
    int whole;            // 256 x 256 tiles, in front of
    int pieces;           // pieces of 256 / cut channels of the others
    int cut;              // 1, 2 or 4
    WaitBound bound;
};

// The tiles of a cluster: t = cluster, cluster + clusters, .. < whole + pieces.
// Tiles beyond whole rounds of all clusters are cut into pieces where these
// still make one round: 768 tiles over 74 clusters end in 56 half tiles.
struct WideTile {
    int n0, o0, cols;   // first token and channel, channels
};

__device__ __forceinline__ WideTile wide_tile(const WideArgs& p, int t) {
    const bool cut = t >= p.whole;
    const int s = t - p.whole;
    const int tile = cut ? p.whole + s / p.cut : t;
    const int cols = cut ? 256 / p.cut : 256;
    return WideTile{(tile % p.m_tiles) * 256, (tile / p.m_tiles) * 256 + (cut ? (s % p.cut) * cols : 0), cols};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
linear_i8_wide_kernel(const __grid_constant__ WideArgs p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    auto bar = [&](int i) { return sbase + kOffWideBars + 8u * static_cast<uint32_t>(i); };
    auto leader_bar = [&](int i) { return ptx::map_to_rank(bar(i), 0); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffWideBars + 8 * W_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffWideBars + 8 * W_BARS + 4);
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWideStages; ++s) {
            ptx::mbar_init(bar(W_FULL + s), 1);     // leader: both CTAs' bytes
            ptx::mbar_init(bar(W_EMPTY + s), 1);    // each CTA: MMA commit
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(W_ACC_FULL + b), 1);   // each CTA: MMA commit
            ptx::mbar_init(bar(W_ACC_FREE + b), 16);  // leader: 8 epilogue warps x 2 CTAs
        }
        ptx::mbar_init(bar(W_DRAIN), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tm_x);
        ptx::prefetch_tmap(&p.tm_w);
        ptx::prefetch_tmap(&p.tm_out);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp == 0) {
        // tiles in order of channels, all token tiles of a channel tile in a
        // row: the clusters work on the same weights at the same time
        int e = 0;
        bool ok = true;
        for (int t = cluster; t < p.whole + p.pieces && ok; t += clusters) {
            const WideTile w = wide_tile(p, t);
            const int n0 = w.n0 + 128 * rank, o0 = w.o0 + w.cols / 2 * rank;
            const void* tm_w = w.cols == 256 ? static_cast<const void*>(&p.tm_w) : &p.tm_w_cut;
            const uint32_t tx = 2 * (kOpBytes + static_cast<uint32_t>(w.cols / 2) * kChunk);   // both CTAs'
            for (int c = 0; c < p.chunks; ++c, ++e) {
                const int s = e % kWideStages;
                bool good = true;
                if (lane == s) {
                    good = wait_bounded(bar(W_EMPTY + s), ((e / kWideStages) & 1) ^ 1, abort_flag, p.status, p.bound);
                    if (good) {
                        const uint32_t st = sbase + s * kWideStage;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(bar(W_FULL + s), tx);
                        const bool withheld = e == 0 && blockIdx.x == 0 && p.bound.withhold;
                        if (!withheld)
                            ptx::tma_load_2d_pair_normal(st, &p.tm_x, static_cast<int>(kChunk) * c, n0, leader_bar(W_FULL + s));
                        ptx::tma_load_2d_pair_normal(st + kOpBytes, tm_w, static_cast<int>(kChunk) * c, o0,
                                                     leader_bar(W_FULL + s));
                    }
                }
                if (!__all_sync(0xffffffffu, good)) { ok = false; break; }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int e = 0, i = 0;
            bool ok = true;
            for (int t = cluster; t < p.whole + p.pieces && ok; t += clusters, ++i) {
                const int b = i & 1;
                const uint32_t idesc = ptx::idesc_i8_s32(256, wide_tile(p, t).cols);
                ok = __all_sync(0xffffffffu, wait_bounded(bar(W_ACC_FREE + b), ((i >> 1) & 1) ^ 1, abort_flag, p.status, p.bound));
                if (!ok) break;
                ptx::tc_fence_after();
                for (int c = 0; c < p.chunks; ++c, ++e) {
                    const int s = e % kWideStages;
                    ok = __all_sync(0xffffffffu, wait_bounded(bar(W_FULL + s), (e / kWideStages) & 1, abort_flag, p.status, p.bound));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint32_t st = sbase + s * kWideStage;
                        const uint64_t a = ptx::smem_desc_sw128(st, 16, 1024),
                                       w = ptx::smem_desc_sw128(st + kOpBytes, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_pair_i8_ss(tmem + 256 * b, a + ((32 * kk) >> 4), w + ((32 * kk) >> 4), idesc,
                                                (c | kk) ? 1u : 0u);
                        ptx::mma_commit_pair(bar(W_EMPTY + s), 0x3);
                        if (c == p.chunks - 1) ptx::mma_commit_pair(bar(W_ACC_FULL + b), 0x3);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                // let every MMA this warp issued finish before the teardown frees anything
                if (ptx::elect_one()) ptx::mma_commit_pair(bar(W_DRAIN), 0x1);
                __syncwarp();
                const uint64_t t0 = ptx::global_timer_ns();
                while (!ptx::mbar_try_wait(bar(W_DRAIN), 0) && ptx::global_timer_ns() - t0 < p.bound.timeout_ns) {
                }
            }
        }
    } else {
        // two warps per tensor-memory lane quadrant, 128 of the 256 channels each
        // (with one the epilogue, not the MMAs, set the pace: 63 us for 2,048
        // tokens through 1,536 x 24,576)
        const int wq = warp & 3, half = (warp - 2) >> 2;
        const int st = (warp - 2) * 32 + lane;
        float* scales = reinterpret_cast<float*>(smem + kOffScales);
        unsigned char* stage = smem + kOffStage + (warp - 2) * 4096;
        const uint32_t stage_u = sbase + kOffStage + (warp - 2) * 4096;
        const int x7 = lane & 7;
        int i = 0;
        for (int t = cluster; t < p.whole + p.pieces; t += clusters, ++i) {
            const WideTile tile = wide_tile(p, t);
            const int row0 = tile.n0 + 128 * rank + 32 * wq, o0 = tile.o0;
            // groups of 64 channels of this warp: half, half + 2
            const int groups = row0 < p.n_tok ? (min(tile.cols, p.d_out - o0) + 63) / 64 : 0;
            const int last = groups > half + 2 ? half + 2 : half;
            const int b = i & 1;
            ptx::named_bar_sync(1, 256);   // every warp has read the last tile's scales
            scales[st] = o0 + st < p.d_out ? p.w_scale[o0 + st] : 0.f;
            const float sx = row0 + lane < p.n_tok ? p.x_scale[row0 + lane] : 0.f;
            ptx::named_bar_sync(2, 256);
            bool ok = wait_bounded(bar(W_ACC_FULL + b), (i >> 1) & 1, abort_flag, p.status, p.bound);
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int q = half; q < groups && ok; q += 2) {   // the same for the whole warp
                uint32_t r[2][32];
                const uint32_t src = tmem + (static_cast<uint32_t>(wq * 32) << 16) + 256 * b + 64 * q;
                ptx::tmem_ld32(src, r[0]);
                ptx::tmem_ld32(src + 32, r[1]);
                ptx::tmem_wait_ld();
                if (q == last) {   // the accumulator has been read: the MMAs may have it back
                    // (relaxed: a cluster-scope release held the warp for over 2,000 cycles)
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_bar(W_ACC_FREE + b));
                }
                // 32 rows x 64 bf16 in the store box's swizzled layout
                if (lane == 0) ptx::bulk_wait_read_all();   // the last store has read its box
                __syncwarp();
                unsigned char* my_row = stage + lane * 128;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 w0 = *reinterpret_cast<const float4*>(scales + 64 * q + 8 * k);
                    const float4 w1 = *reinterpret_cast<const float4*>(scales + 64 * q + 8 * k + 4);
                    auto v = [&](int j) { return static_cast<int>(r[k >> 2][(8 * k + j) & 31]); };
                    *reinterpret_cast<uint4*>(my_row + ((k ^ x7) * 16)) =
                        make_uint4(pack_bf16x2(scaled(v(0), sx, w0.x), scaled(v(1), sx, w0.y)),
                                   pack_bf16x2(scaled(v(2), sx, w0.z), scaled(v(3), sx, w0.w)),
                                   pack_bf16x2(scaled(v(4), sx, w1.x), scaled(v(5), sx, w1.y)),
                                   pack_bf16x2(scaled(v(6), sx, w1.z), scaled(v(7), sx, w1.w)));
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_2d(&p.tm_out, stage_u, o0 + 64 * q, row0);
                    ptx::bulk_commit_group();
                }
            }
            if (groups <= half || !ok) {   // a warp without columns here
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_bar(W_ACC_FREE + b));
            }
        }
        if (lane == 0) ptx::bulk_wait_all();
    }
    settle_copies(abort_flag);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// choice of kernel and shape, by estimates in cycles
// ---------------------------------------------------------------------------

// Token tile and K parts of the split kernel: the loads of the busiest SM at 50
// bytes a cycle, and for each wave of CTAs the latency of its first loads and
// its epilogue.  Parts are a power of two (others leave SMs of a GPC unused) of
// two chunks at least.  Products alone, measured: 32 tokens through 16,384 x
// 5,120 (40 channel tiles) 30.0, 18.9 and 29.4 us with 2, 4 and 7 parts; 897
// tokens through 272 x 464 (with the quantisation) 26 us with token tiles of
// 256, 9 with 64.
struct SplitPlan {
    long cost;
    int tok_tiles, parts;
};

SplitPlan split_plan(int n_tok, int chunks, int d_out) {
    SplitPlan best{-1, 1, 1};
    const int o_tiles = (d_out + 127) / 128;
    for (int most = 256; most >= 64; most /= 2) {
        const int tt = (n_tok + most - 1) / most;
        const int nt = ((n_tok + tt - 1) / tt + 15) / 16 * 16;
        const long stage = kOpBytes + static_cast<long>(nt) * kChunk;
        const int slots = (nt <= 64 ? 2 : 1) * kSms;   // CTAs resident at once
        for (int k = 1; k <= kMaxCluster && (k == 1 || 2 * k <= chunks); k *= 2) {
            const long ctas = static_cast<long>(o_tiles) * tt * k, waves = (ctas + slots - 1) / slots;
            const long in_wave = ctas < slots ? ctas : slots;
            const long loads = (chunks + k - 1) / k * stage / 50 * (in_wave > kSms ? in_wave : kSms) / kSms;
            const long cost = waves * (loads + 3000 + 10 * nt + 20 * nt / k);
            if (best.cost < 0 || cost < best.cost) best = SplitPlan{cost, tt, k};
        }
    }
    return best;
}

// The wide kernel: rounds of all clusters, 620 cycles a chunk (its two operand
// chunks per SM at about 50 bytes a cycle).  At 5,120 columns, measured: 32
// tiles (512 tokens, 4,096 channels) 16.9 us split and 17.8 wide, 60 tiles 33
// and 19; at 512 columns 32 tiles 7.3 and 7.1, 80 tiles 20 and 10.
long wide_cost(int n_tok, int chunks, int d_out) {
    const long tiles = static_cast<long>((n_tok + 255) / 256) * ((d_out + 255) / 256);
    return 6000 + (tiles + kSms / 2 - 1) / (kSms / 2) * (chunks * 620L + 500);
}

// Test hook state: the next launch withholds one load and uses this wait bound.
std::atomic<uint64_t> g_test_wait_limit_ns{0};

WaitBound next_bound() {
    const uint64_t limit = g_test_wait_limit_ns.exchange(0);
    return limit != 0 ? WaitBound{limit, 1} : WaitBound{2000000000ull, 0};
}

int chunks_of(int d_in) { return (d_in + static_cast<int>(kChunk) - 1) / static_cast<int>(kChunk); }

// Launch shape of the split kernel.  Its dynamic shared memory is at least its
// tensor memory's share of an SM: tcgen05.alloc waits without a bound for free
// columns, and the CTAs of a cluster for each other, so clusters that waited
// for one another's columns on different SMs would wait forever.  Blocks that
// fit an SM together never ask for more than its columns.  (The decode keeps to
// the same rule; the projections' CTAs need no others to finish.)
struct SplitShape {
    int nt, stages;              // tokens of a tile, ring stages
    uint32_t ring_bytes, tmem_cols;
    size_t smem;                 // dynamic shared memory
};

SplitShape split_shape(int n_tok, int chunks, const SplitPlan& plan) {
    SplitShape s;
    s.nt = ((n_tok + plan.tok_tiles - 1) / plan.tok_tiles + 15) / 16 * 16;
    const bool two = s.nt <= 64;   // two CTAs per SM
    const uint32_t stage = kOpBytes + static_cast<uint32_t>(s.nt) * kChunk;
    const int most = (chunks + plan.parts - 1) / plan.parts;   // chunks of one CTA
    s.stages = static_cast<int>((two ? kSplitRingHalf : kSplitRing) / stage);
    if (s.stages > most) s.stages = most;
    s.ring_bytes = s.stages * stage;
    if (s.ring_bytes < static_cast<uint32_t>(s.nt) * 512) s.ring_bytes = static_cast<uint32_t>(s.nt) * 512;
    s.tmem_cols = 32;
    while (s.tmem_cols < static_cast<uint32_t>(s.nt)) s.tmem_cols *= 2;
    s.smem = s.ring_bytes + 8 * (2 * s.stages + 1) + 16 + 1024;
    const size_t least = tmem_share(s.tmem_cols);
    if (s.smem < least) s.smem = least;
    return s;
}

cudaError_t launch_split(const int8_t* x8, long ld_x, const float* x_scale, const int8_t* w8, const float* w_scale,
                         uint16_t* out, int n_tok, int d_in, int d_out, const SplitPlan& plan, int32_t* status,
                         cudaStream_t stream) {
    SplitArgs p;
    const int o_tiles = (d_out + 127) / 128;
    p.chunks = chunks_of(d_in);
    const int tok_tiles = plan.tok_tiles, parts = plan.parts;
    const SplitShape shape = split_shape(n_tok, p.chunks, plan);
    p.nt = shape.nt, p.stages = shape.stages, p.ring_bytes = shape.ring_bytes, p.tmem_cols = shape.tmem_cols;
    p.idesc = ptx::idesc_i8_s32(128, p.nt);
    p.x_scale = x_scale, p.w_scale = w_scale, p.out = out, p.status = status;
    p.n_tok = n_tok, p.d_out = d_out, p.bound = next_bound();
    if (!make_map_i8(&p.tm_w, w8, d_in, d_out, d_in, 128) || !make_map_i8(&p.tm_x, x8, d_in, n_tok, ld_x, p.nt))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = allow_smem_once(linear_i8_split_kernel, static_cast<int>(kSplitRing + 2048), smem_set);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(linear_i8_split_kernel, dim3(o_tiles * parts, tok_tiles), dim3(kSplitThreads), parts, shape.smem,
                              stream, p);
}

cudaError_t launch_wide(const int8_t* x8, long ld_x, const float* x_scale, const int8_t* w8, const float* w_scale,
                        uint16_t* out, int n_tok, int d_in, int d_out, int32_t* status, cudaStream_t stream) {
    WideArgs p;
    p.chunks = chunks_of(d_in);
    p.m_tiles = (n_tok + 255) / 256;
    const int tiles = p.m_tiles * ((d_out + 255) / 256);
    const int most = kSms / 2, rest = tiles % most;
    p.cut = tiles < most || rest == 0 ? 1 : (4 * rest <= most ? 4 : (2 * rest <= most ? 2 : 1));
    p.whole = p.cut > 1 ? tiles - rest : tiles;
    p.pieces = p.cut > 1 ? rest * p.cut : 0;
    p.x_scale = x_scale, p.w_scale = w_scale, p.status = status;
    p.n_tok = n_tok, p.d_out = d_out, p.bound = next_bound();
    if (!make_map_i8(&p.tm_w, w8, d_in, d_out, d_in, 128) ||
        !make_map_i8(&p.tm_w_cut, w8, d_in, d_out, d_in, 128 / p.cut) ||
        !make_map_i8(&p.tm_x, x8, d_in, n_tok, ld_x, 128) ||
        !make_map_2d(&p.tm_out, out, d_out, n_tok, static_cast<uint64_t>(d_out) * 2, 64, 32))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = allow_smem_once(linear_i8_wide_kernel, static_cast<int>(kWideSmem), smem_set);
    if (e != cudaSuccess) return e;
    const int clusters = tiles < most ? tiles : most;
    return launch_pdl(linear_i8_wide_kernel, dim3(2 * clusters), dim3(kWideThreads), kWideSmem, stream, p);
}

}  // namespace

namespace {

// The kernel that serves a product: wide, or split with this plan.
bool choose_wide(int n_tok, int chunks, int d_out, SplitPlan* plan) {
    *plan = split_plan(n_tok, chunks, d_out);
    return wide_cost(n_tok, chunks, d_out) < plan->cost;
}

}  // namespace

cudaError_t launch_linear_i8(const int8_t* x8, long ld_x, const float* x_scale, const int8_t* w8,
                             const float* w_scale, uint16_t* out, int n_tok, int d_in, int d_out, int32_t* status,
                             cudaStream_t stream) {
    SplitPlan plan;
    if (choose_wide(n_tok, chunks_of(d_in), d_out, &plan))
        return launch_wide(x8, ld_x, x_scale, w8, w_scale, out, n_tok, d_in, d_out, status, stream);
    return launch_split(x8, ld_x, x_scale, w8, w_scale, out, n_tok, d_in, d_out, plan, status, stream);
}

void linear_i8_arm_timeout_test(uint64_t wait_limit_ns) { g_test_wait_limit_ns.store(wait_limit_ns); }

LinearShape linear_i8_shape(int n_tok, int d_in, int d_out) {
    SplitPlan plan;
    if (choose_wide(n_tok, chunks_of(d_in), d_out, &plan)) return LinearShape{2, 512, kWideSmem};
    const SplitShape s = split_shape(n_tok, chunks_of(d_in), plan);
    return LinearShape{plan.parts, static_cast<int>(s.tmem_cols), s.smem};
}

}  // namespace mla
