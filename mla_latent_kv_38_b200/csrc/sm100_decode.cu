// Absorbed MLA decode on the 5th-generation tensor cores (tcgen05), DeepSeek-V2
// head shape: d_c = 512 latent columns + d_r = 64 RoPE columns per cache row,
// heads in blocks of 128.
//
// What is computed (DeepSeek-V3 report notes eq. (10) with the absorbed query
// of "MLA(Multi-head Latent Attention): DeepSeek-V2 논문정리", "Key에 대한 수식
// 전개" / "Value에 대한 수식 전개"):
//   S = [q_abs ; q^R] . [c ; k^R]^T * scale   (M = 128 heads, K = 576)
//   causal mask, online softmax (exp2 domain)
//   O = P . c                                  (M = 128 heads, N = 512, K = keys)
// Every head reads every cache row, so both products are dense contractions
// with M = heads; the cache is streamed from HBM once.
//
// Mapping onto B200:
//  * A cluster of two CTAs (two SMs) issues cta_group::2 MMAs with M = 128: CTA
//    r owns heads [64r, 64r+64).  In the paired layout each SM's tensor memory
//    holds its 64 rows spread over all 128 lanes (lanes 0-63 take the first
//    half of N, lanes 64-127 the second), so O (64 heads x 512, fp32) takes 256
//    columns per SM and one S buffer (N = 256 keys) 128 columns; O and two S
//    buffers fill the 512 columns.
//  * A tile is 4 cache pages (256 keys).  S = [q_abs ; q^R] . K^T runs as 9 MMA
//    groups of K = 64 columns, N = 256: the pair's B operand is split by keys,
//    so each CTA loads its own 2 pages (128 keys x 576 columns).  O += P . V
//    runs as 2 x N = 256 per 16 keys: the B operand is split by latent
//    columns, so each CTA loads all 4 pages of its 256 latent columns (these
//    second reads hit L2).
//  * All operands arrive by TMA (128-byte swizzle) in two rings, each with one
//    producer warp and one in-order MMA consumer: 24 KB S entries (one
//    64-column chunk of the CTA's 2 pages and of its 64 query rows; the query
//    is re-read from L2 each tile, which leaves shared memory to the rings) and
//    32 KB V entries (the CTA's 4 latent chunks of one page, one 3-D box).  The
//    loads run at DRAM latency, so the bytes in flight per SM set the rate; a
//    thread's TMA copies run one after another, so every ring slot has its own
//    issuing thread.
//  * Warp roles per CTA: warp 0 S producer, warp 1 tensor-memory allocation
//    and (CTA 0) the S MMAs, warp 2 (CTA 0) the P.V MMAs, warp 3 V producer,
//    warps 4-11 softmax and epilogue (two warps per tensor-memory lane
//    quadrant).  S is double buffered and free again once its scores are in
//    registers; P is written to shared memory in two key halves, each released
//    as soon as its MMAs complete.  The running max is rescaled lazily (only
//    when it grows by 2^8).
//  * What bounds it with the cache in L2 (64 x 4 tokens of 128 heads behind 8,192
//    shared keys, 490 us): the loads.  A tile takes 344 KB per SM at 12.4 TB/s
//    over all SMs, which is what TMA boxes of this shape reach with 192 KB in
//    flight per SM; its MMAs need two thirds of that time.  Keeping the query in
//    shared memory takes 72 KB off each tile and as much off the rings: 480 us
//    there, 110 instead of 108 us for a shard's batch of short units.
//  * Work: the tiles of all (sequence, token, head block) units are laid end
//    to end and cut into contiguous ranges, one per cluster (persistent, 74
//    clusters on 148 SMs).  Each CTA computes the cut from the sequence
//    lengths itself (a block-wide scan), so no separate scheduling launch
//    precedes the decode unless the unit count is very large.  A bound on the
//    parts per unit moves each cut to the next allowed split point.  A unit
//    covered by one cluster is written directly in bf16; otherwise each
//    cluster writes an fp32 partial and its log-sum-exp, merged by a
//    reduction kernel.
//  * Every mbarrier wait is bounded by the global timer: on expiry the kernel
//    sets MLA_STATUS_TIMEOUT and unwinds instead of hanging.

#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "sm100_decode.h"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace mla {
namespace {

constexpr int kThreads = 384;   // 12 warps: S loads, S MMAs, P.V MMAs, V loads, 8 x softmax
// Registers per thread: 168 at launch (65,536 / 384, rounded down to 8); then
// the load / MMA warpgroup gives registers up to the two softmax warpgroups.
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsIssue = 80;
constexpr uint32_t kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr int kClusters = 74;                     // 148 SMs / 2
constexpr int kDc = 512, kDr = 64, kRow = 576;    // row = c^KV || k^R
constexpr int kPage = 64;                         // cache rows per page (TMA box height)
constexpr int kTilePages = 4;                     // a tile = 4 pages = 256 keys (MMA N)
constexpr int kChunks = 9;                        // 64-column chunks of a row (8 latent + 1 RoPE)
constexpr int kSRing = 4;                         // 24 KB entries, S operand stream (query chunk + key chunks)
constexpr int kVRing = 3;                         // 32 KB entries, P.V operand stream
constexpr int kSLaneGroups = 4;                   // S ring slots are issued by this many groups of lanes in turn

constexpr uint32_t kBox = 8192;                   // one page x 64 columns (128 B rows)
constexpr uint32_t kSEntry = 3 * kBox;            // chunk c of the CTA's 2 pages (keys) and of its 64 query rows
constexpr uint32_t kVEntry = 4 * kBox;            // the CTA's 4 latent chunks of one page
constexpr uint32_t kPBytes = 4 * kBox;            // 64 heads x 256 keys (4 blocks of 64 keys)
constexpr uint32_t kOffSRing = 0;
constexpr uint32_t kOffVRing = kOffSRing + kSRing * kSEntry;
constexpr uint32_t kOffP = kOffVRing + kVRing * kVEntry;
constexpr uint32_t kOffXmax = kOffP + kPBytes;    // 4 x 64 floats: partial row maxima (or sums)
constexpr uint32_t kOffBar = kOffXmax + 1024;
constexpr uint32_t kMaxBars = 40;
constexpr uint32_t kOffMisc = kOffBar + 8 * kMaxBars;   // tmem base, abort flag
constexpr uint32_t kOffCuts = kOffMisc + 64;      // cluster boundaries (75 ints)
constexpr uint32_t kOffSlice = kOffCuts + 320;    // key counts of the cluster's units
// Dynamic shared memory: the buffers above from a 1024-byte aligned base.
constexpr uint32_t kSmemBytes = 232448;
constexpr int kSliceCap = static_cast<int>((kSmemBytes - 1024 - kOffSlice) / 4);
// Units up to which every CTA computes the schedule itself (the scan's scratch
// is the ring area).  The key counts of the cluster's units go to shared
// memory when they fit, else to the CTA's own region of the workspace.
constexpr int kInKernelUnits = 2048;
static_assert(kOffSlice + 1024 <= kSmemBytes, "shared memory budget");
static_assert(4 * (5 * kInKernelUnits + 3 + kClusters + 1 + 48) <= static_cast<int>(kOffP - kOffSRing), "schedule scratch");
static_assert(4 * (kClusters + 1) <= 320, "cut area");
static_assert(kSRing % kSLaneGroups == 0, "each lane group keeps its own ring slots");
static_assert(4 * kSLaneGroups <= 32, "lane groups of the S producer warp");
static_assert(8 * 16384 <= kOffP, "the last epilogue's staging (16 KB per softmax warp) lies in the rings");

enum {
    BAR_SR_FULL = 0,                         // + slot (leader: both CTAs' bytes)
    BAR_SR_EMPTY = BAR_SR_FULL + kSRing,     // + slot (each CTA, MMA commit)
    BAR_VR_FULL = BAR_SR_EMPTY + kSRing,
    BAR_VR_EMPTY = BAR_VR_FULL + kVRing,
    BAR_S_FULL = BAR_VR_EMPTY + kVRing,      // + S buffer
    BAR_S_FREE = BAR_S_FULL + 2,             // + S buffer (leader, 8 warps x 2 CTAs)
    BAR_P_FULL = BAR_S_FREE + 2,             // + P half (leader, 4 warps x 2 CTAs; half 0: all 8 x 2)
    BAR_P_FREE = BAR_P_FULL + 2,             // + P half (each CTA, MMA commit)
    BAR_TAIL_READY = BAR_P_FREE + 2,         // each CTA, MMA thread arrives remotely
    BAR_TAIL_DONE = BAR_TAIL_READY + 1,      // leader, 8 warps x 2 CTAs
    BAR_DRAIN = BAR_TAIL_DONE + 1,           // S issuer's own drain on abort
    BAR_DRAIN_PV = BAR_DRAIN + 1,            // P.V issuer's
    BAR_X_FREE = BAR_DRAIN_PV + 1,           // + row group: its 4 warps have read the exchanged values
    BAR_X_FULL = BAR_X_FREE + 2,             // + row group: its 4 warps have written them
    NUM_BARS = BAR_X_FULL + 2
};
static_assert(NUM_BARS <= static_cast<int>(kMaxBars), "barrier area");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;                    // 2 x 128 columns (paired layout)
constexpr uint32_t kTmemS = 256;                  // 2 x 128 columns

constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, 256, 0, 0);
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, 256, 0, 1);

constexpr uint32_t kSuspendHintNs = 100000;      // a waiting thread sleeps up to 0.1 ms per try
constexpr float kRescaleThreshold = 8.0f;         // log2 units

// How the query rows are cut into units of work (described at unit_keys).
struct UnitMap {
    int n_h, n_hb, B, T_q, max_blocks;
    // the shared decode only:
    int n_shared;      // pages that every sequence begins with
    int n_prefix;      // units of the shared keys; 0: every unit walks the shared pages, then its own
    int n_rows;        // query rows of the batch
    int tok_per_unit;  // whole tokens of a sequence in one unit (1 when n_h > 64)
    int own_rows;      // rows of a sequence unit's partial slot, a multiple of 32
};

struct Sm100Params {
    CUtensorMap tm_pool;      // pool as [rows][576], box 64 cols x 64 rows
    CUtensorMap tm_pool_v;    // pool as [chunk][rows][64], box 64 cols x 64 rows x 4 chunks
    CUtensorMap tm_qa;        // q_abs as [n_tok*n_h][512], box 64 x 64
    CUtensorMap tm_qr;        // q_r   as [n_tok*n_h][64],  box 64 x 64
    CUtensorMap tm_out;       // out_latent as [n_tok*n_h][512] bf16, box 64 x 32 (stores)
    CUtensorMap tm_part;      // part_o as [(C+U)*128][512] fp32, box 32 x 32 (stores)
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t* prefix;          // (U + 1) exclusive prefix of pages per unit (schedule kernel only)
    int32_t* unit_kv;         // (U) keys per unit (schedule kernel only)
    int32_t* kv_cta;          // (148 x U) per-CTA key counts when the slice exceeds shared memory
    int4* unit_meta;          // (U) {kv_len, first cluster, parts, sequence}
    const int4* cluster_info; // (C) {first page, end page, first unit, last unit} (schedule kernel only)
    uint16_t* out_latent;
    float* out_lse;
    float* part_o;            // (C + U) slots x 128 rows x 512
    float* part_lse;          // (C + U) slots x 128
    int32_t* status;
    const int32_t* shared_table;   // (n_shared) blocks of the shared pages (shared decode only)
    const uint16_t* pool;          // for single rows (shared decode only)
    UnitMap um;
    int U, num_blocks, max_splits;
    int in_kernel_schedule;   // 1: each CTA computes the schedule; 0: the schedule kernel did
    int withhold_load;        // test hook: 1 = never issue the first S entry's load of CTA 0
    uint64_t timeout_ns;      // bound of every wait
    float scale_log2;
};

// Two bf16 values with infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
    return v;
}

// NaN in each of the 32 values whose bf16 counterpart in `row` is not finite.
__device__ __forceinline__ void nan_where_infinite(uint32_t (&o)[32], const uint16_t* row) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint4 v = reinterpret_cast<const uint4*>(row)[k];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if ((w[e] & 0x7F80u) == 0x7F80u) o[8 * k + 2 * e] = 0x7FC00000u;
            if ((w[e] & 0x7F800000u) == 0x7F800000u) o[8 * k + 2 * e + 1] = 0x7FC00000u;
        }
    }
}

template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(uint32_t addr, uint32_t parity, volatile int* abort_flag,
                                         int32_t* status, uint64_t timeout_ns) {
    if (ptx::mbar_try_wait<kCluster>(addr, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    while (true) {
        if (ptx::mbar_try_wait_suspend<kCluster>(addr, parity, kSuspendHintNs)) return true;
        if (*abort_flag) return false;
        if (ptx::global_timer_ns() - t0 > timeout_ns) {
            *abort_flag = 1;
            raise_status(status, MLA_STATUS_TIMEOUT);
            return false;
        }
    }
}

// ---------------------------------------------------------------------------
// Work schedule.  Units are numbered token-major: u = (t B + b) n_hb + hb
// for query token t of sequence b and head block hb, so that the T_q units
// of one sequence lie a quarter (for T_q = 4) of the work apart and run on
// different clusters at the same time, at the same relative position in the
// cache: their page reads meet in L2 instead of streaming the cache from
// HBM T_q times.  Unit u covers the keys 0 .. kv - 1 of query row (b, t),
// kv = L_b - T_q + t + 1, i.e. ceil(kv / 64) pages; a sequence whose length
// is out of range has no pages (its outputs are defined as zero / -inf by
// the merge kernel).  pf is the exclusive prefix of the page counts, T =
// pf[U] the total.
//
// Shared decode (kShared).  A unit of a sequence takes as many whole tokens as
// fit its 128 rows (tok_per_unit, at most 64; t then counts such groups); a
// token's row sees kv minus the tokens behind it in the unit.  The shared
// pages are either walked by every sequence unit in front of its own
// (n_prefix = 0), or by n_prefix units of their own in front of the others:
// 128 consecutive query rows of the whole batch, whatever their sequence.
// The sequence units then begin behind the shared pages.
// ---------------------------------------------------------------------------

struct UnitIdx {
    int b, t, hb;
};

__device__ __forceinline__ UnitIdx unit_index(int u, int n_hb, int B) {
    const int r = u / n_hb;
    const int t = r / B;
    return UnitIdx{r - t * B, t, u - r * n_hb};
}

template <bool kShared>
__device__ __forceinline__ int unit_keys(const int32_t* seq_lens, int u, const UnitMap& um) {
    if constexpr (kShared) {
        const int own0 = um.n_shared * kPage;
        if (u < um.n_prefix) return own0;
        const UnitIdx x = unit_index(u - um.n_prefix, um.n_hb, um.B);
        const int L = seq_lens[x.b];
        if (L < um.T_q + own0 || L > um.max_blocks * kPage) return 0;
        return L - um.T_q + min(um.T_q, (x.t + 1) * um.tok_per_unit) - (um.n_prefix > 0 ? own0 : 0);
    } else {
        const UnitIdx x = unit_index(u, um.n_hb, um.B);
        const int L = seq_lens[x.b];
        return (L >= um.T_q && L <= um.max_blocks * kPage) ? L - um.T_q + x.t + 1 : 0;
    }
}

// Whether u is the first unit of a sequence (the one that reports its length).
template <bool kShared>
__device__ __forceinline__ bool first_of_sequence(int u, const UnitMap& um) {
    if constexpr (kShared) u -= um.n_prefix;
    return u >= 0 && u < um.B * um.n_hb && u % um.n_hb == 0;
}

// Last of n entries with a[v] <= g (a ascending, a[0] <= g), narrowed to an
// eighth with each round of independent loads.
__device__ __forceinline__ int last_at_or_below(const int32_t* a, int n, int g) {
    int lo = 0;
    while (n > 1) {
        const int step = (n + 7) >> 3;
        int k = 0;
#pragma unroll
        for (int j = 1; j < 8; ++j) k += j * step < n && a[lo + j * step] <= g;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Last unit v with pf[v] <= g (for g < T: the unit holding page g).
__device__ __forceinline__ int unit_of_page(const int32_t* pf, int U, int g) { return last_at_or_below(pf, U, g); }

// Work is cut at whole tiles (4 pages, 256 keys, counted from each unit's
// start), so that a range that crosses a unit boundary carries no extra
// partial tile.  The cut balances a cost per cluster: 4 per tile (quarter
// tiles) plus kSegCost for every unit segment it starts, which stands for
// the epilogue and pipeline restart of a segment (measured at about 1.5
// tiles).  wf is the exclusive prefix of the units' costs, W = wf[U]; raw cut
// c lies at cost floor(c W / C), rounded to the nearest tile of the unit it
// falls in.  With max_splits = s > 0 it then moves up to the next allowed
// cut, where unit u's P tiles are cut into k = min(s, P) pieces at
// tf[u] + floor(j P / k), j = 0 .. k, so no unit lies in more than s ranges.
// (A shared decode of few pages was no faster cut by single pages: the merge of
// the additional partials takes what the shorter tiles save.)
constexpr int kSegCost = 6;

__device__ __forceinline__ int unit_cost(int tiles) { return 4 * tiles + (tiles > 0 ? kSegCost : 0); }

__device__ int raw_cut_tile(int c, int Tt, const int32_t* tf, const int32_t* wf, int U, int max_splits) {
    if (c <= 0) return 0;
    if (c >= kClusters) return Tt;
    const int W = wf[U];
    const int x = static_cast<int>(static_cast<long long>(c) * W / kClusters);
    if (x >= W) return Tt;
    int u = unit_of_page(wf, U, x);           // wf[u] <= x < wf[u + 1]
    const int tiles = tf[u + 1] - tf[u];
    const int d = x - wf[u] - kSegCost;
    const int g = tf[u] + (d <= 0 ? 0 : min(tiles, (d + 2) / 4));
    if (max_splits <= 0 || g >= Tt) return g;
    u = unit_of_page(tf, U, g);
    const int a = tf[u], P = tf[u + 1] - a;   // a <= g < tf[u + 1], so P > 0
    const int k = min(max_splits, P);
    const int j = static_cast<int>((static_cast<long long>(g - a) * k + P - 1) / P);   // ceil((g-a) k / P)
    return a + static_cast<int>(static_cast<long long>(j) * P / k);
}

// First page of global tile gt (T pages, Tt tiles in all).
__device__ int tile_to_page(int gt, int Tt, int T, const int32_t* tf, const int32_t* pf, int U) {
    if (gt >= Tt) return T;
    const int u = unit_of_page(tf, U, gt);    // tf[u] <= gt < tf[u + 1]
    return pf[u] + kTilePages * (gt - tf[u]);
}

// Cluster boundaries cuts[0 .. C] in pages: the distinct raw cuts in order,
// then T repeated, so cluster c covers pages [cuts[c], cuts[c + 1]) and every
// non-empty range comes before every empty one (a unit's ranges are always
// consecutive clusters).  All threads of the block call it; tmp holds C + 1
// ints of scratch.
__device__ void compute_cuts(int* cuts, int* tmp, const int32_t* pf, const int32_t* tf, const int32_t* wf, int U,
                             int T, int Tt, int max_splits) {
    for (int c = threadIdx.x; c <= kClusters; c += blockDim.x)
        tmp[c] = tile_to_page(raw_cut_tile(c, Tt, tf, wf, U, max_splits), Tt, T, tf, pf, U);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        constexpr int kPer = (kClusters + 1 + 31) / 32;
        int n = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int c = lane * kPer + k;
            if (c <= kClusters && (c == 0 || tmp[c] != tmp[c - 1])) ++n;
        }
        int x = n;   // inclusive warp scan of the distinct counts
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int total = __shfl_sync(0xffffffffu, x, 31);
        int pos = x - n;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int c = lane * kPer + k;
            if (c <= kClusters && (c == 0 || tmp[c] != tmp[c - 1])) cuts[pos++] = tmp[c];
        }
        for (int c = total + lane; c <= kClusters; c += 32) cuts[c] = T;
    }
    __syncthreads();
}

// Cluster whose range holds page g < T (the last cluster starting at or before g).
__device__ __forceinline__ int cluster_of_page(int g, const int* cuts) { return last_at_or_below(cuts, kClusters, g); }

// Merge metadata of unit u: {kv_len, first cluster, parts, sequence}.
template <bool kShared>
__device__ int4 unit_meta_of(int u, const int32_t* pf, const int* cuts, int kv, const UnitMap& um) {
    const int b = kShared ? 0 : unit_index(u, um.n_hb, um.B).b;
    const int a = pf[u], e = pf[u + 1];
    if (e <= a) return make_int4(0, 0, 0, b);
    const int c0 = cluster_of_page(a, cuts);
    const int c1 = cluster_of_page(e - 1, cuts);
    return make_int4(kv, c0, c1 - c0 + 1, b);
}

// One tile of a cluster's work: up to 4 consecutive pages of one unit.
struct Tile {
    int u;          // unit = (t B + b) n_hb + hb (behind the prefix units)
    int row0;       // first query row of the unit (bt n_h + 128 hb)
    int rows;       // query rows of the unit (128 but in the shared decode)
    int n_tok;      // tokens of the unit (1 but in the shared decode)
    int b;          // sequence of the unit
    int kv;         // keys of the unit (kv_len; of its last token)
    int page0;      // first page, within the unit
    int np;         // pages in this tile (1..4)
    bool first;     // first tile of a unit segment (new query, O starts from zero)
    bool last;      // last tile of a unit segment (epilogue follows)
    bool unit_end;  // the unit's last page is in this tile
    bool whole;     // the whole unit lies in this cluster's range (no partial)
};

// Page pg of the tile holds rows that not every token of the unit sees, or
// that lie behind the last key: its V rows are cleaned before they are used.
template <bool kShared>
__device__ __forceinline__ bool tail_page(const Tile& t, int pg) {
    if constexpr (kShared) return kPage * (t.page0 + pg + 1) > t.kv - (t.n_tok - 1);
    return t.unit_end && (t.kv % kPage) != 0 && pg == t.np - 1;
}

// Walks a cluster's pages [g0, g1) as tiles.  kvs[v - off] is the key count
// of unit v (a shared-memory slice of the cluster's units, or a global array
// with off = 0); unit u0 starts at global page ubeg0.  The unit's page range
// and (query row, head block, sequence) are kept up to date incrementally.
template <bool kShared>
struct TileWalker {
    const int32_t* kvs;
    int off, g, g0, g1, u, ubeg, uend, kv;
    int bt, hb, b, t, n_h, n_hb, B, T_q;
    int n_prefix, n_rows, per;   // kShared only
    __device__ void load_unit() {
        kv = kvs[u - off];
        uend = ubeg + (kv + kPage - 1) / kPage;
    }
    __device__ void step_unit() {
        ++u;
        ubeg = uend;
        load_unit();
        if (kShared && u <= n_prefix) return;   // the first sequence unit is (0, 0, 0), set by init
        if (++hb == n_hb) {
            hb = 0;
            if (++b == B) {
                b = 0;
                ++t;
            }
            if (!kShared) bt = b * T_q + t;
        }
    }
    __device__ void init(const int32_t* kvs_, int off_, int u0, int ubeg0, int g0_, int g1_, const UnitMap& um) {
        kvs = kvs_;
        off = off_;
        g = g0_;
        g0 = g0_;
        g1 = g1_;
        n_h = um.n_h;
        n_hb = um.n_hb;
        B = um.B;
        T_q = um.T_q;
        u = u0;
        ubeg = ubeg0;
        if constexpr (kShared) {
            n_prefix = um.n_prefix;
            n_rows = um.n_rows;
            per = um.tok_per_unit;
        }
        const UnitIdx x = unit_index(kShared ? max(u0 - n_prefix, 0) : u0, n_hb, B);
        b = x.b;
        t = x.t;
        hb = x.hb;
        bt = b * T_q + t;
        if (g < g1) {
            load_unit();
            while (g < g1 && uend <= g) step_unit();
        }
    }
    __device__ bool done() const { return g >= g1; }
    __device__ Tile next() {
        Tile r;
        r.u = u;
        if constexpr (kShared) {
            if (u < n_prefix) {
                r.row0 = 128 * u;
                r.rows = min(128, n_rows - r.row0);
                r.n_tok = 1;
            } else {
                r.n_tok = min(per, T_q - t * per);
                r.row0 = (b * T_q + t * per) * n_h + 128 * hb;
                r.rows = per > 1 ? r.n_tok * n_h : min(128, n_h - 128 * hb);
            }
        } else {
            r.row0 = bt * n_h + hb * 128;
            r.rows = 128;
            r.n_tok = 1;
        }
        r.b = b;
        r.kv = kv;
        r.page0 = g - ubeg;
        r.first = (g == g0) || (g == ubeg);
        r.whole = ubeg >= g0 && uend <= g1;
        const int seg_end = min(g1, uend);   // tiles start at the segment start
        r.np = min(kTilePages, seg_end - g);
        r.last = g + r.np == seg_end;
        r.unit_end = g + r.np == uend;
        g += r.np;
        while (g < g1 && uend <= g) step_unit();
        return r;
    }
};

// Block-wide exclusive scans of the units' page counts, tile counts and cut
// costs into pf, tf, wf[0 .. U] (U <= kInKernelUnits), and the units' key
// counts into kvs; every thread of the
// CTA takes part; warp_tot holds 3 x 16 ints of scratch.  Returns {T, Tt}.
template <bool kShared>
__device__ int2 schedule_scan(int* pf, int* tf, int* wf, int* kvs, int* warp_tot, const int32_t* seq_lens, int U,
                              const UnitMap& um) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (U + kThreads - 1) / kThreads;
    const int beg = min(U, tid * per), end = min(U, beg + per);
    int loc[3] = {0, 0, 0};
    for (int u = beg; u < end; ++u) {
        const int kv = unit_keys<kShared>(seq_lens, u, um);
        kvs[u] = kv;
        const int pages = (kv + kPage - 1) / kPage;
        const int tiles = (pages + kTilePages - 1) / kTilePages;
        pf[u + 1] = pages;
        tf[u + 1] = tiles;
        wf[u + 1] = unit_cost(tiles);
        loc[0] += pages;
        loc[1] += tiles;
        loc[2] += unit_cost(tiles);
    }
    int v[3] = {loc[0], loc[1], loc[2]};   // inclusive warp scans
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const int y = __shfl_up_sync(0xffffffffu, v[q], o);
            if (lane >= o) v[q] += y;
        }
    }
    if (lane == 31)
        for (int q = 0; q < 3; ++q) warp_tot[16 * q + w] = v[q];
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            int x = lane < kThreads / 32 ? warp_tot[16 * q + lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane < kThreads / 32) warp_tot[16 * q + lane] = x;   // inclusive over warps
        }
    }
    __syncthreads();
    int r[3];
    for (int q = 0; q < 3; ++q) r[q] = v[q] - loc[q] + (w > 0 ? warp_tot[16 * q + w - 1] : 0);
    for (int u = beg; u < end; ++u) {
        r[0] += pf[u + 1];
        pf[u + 1] = r[0];
        r[1] += tf[u + 1];
        tf[u + 1] = r[1];
        r[2] += wf[u + 1];
        wf[u + 1] = r[2];
    }
    if (tid == 0) pf[0] = tf[0] = wf[0] = 0;
    __syncthreads();
    return make_int2(pf[U], tf[U]);
}

// First partial row of sequence unit uo (counted behind the prefix units) in
// cluster c: the slots of the prefix units, 128 rows each, come first.
__device__ __forceinline__ size_t own_slot_row(int c, int uo, const UnitMap& um) {
    const size_t base = um.n_prefix > 0 ? static_cast<size_t>(kClusters + um.n_prefix) * 128 : 0;
    return base + (static_cast<size_t>(c) + uo) * um.own_rows;
}

// P.V operand split: CTA r supplies latent chunks 4r .. 4r+3 (columns
// [256r, 256r+256)); instruction h (N = 256) takes chunks 4r+2h, 4r+2h+1 from
// each CTA, so TMEM column 128h + j of lane half r holds latent column
// 256r + 128h + j.  V ring entry (page, h) holds exactly those two chunks.

template <bool kShared>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_decode_sm100_kernel(const __grid_constant__ Sm100Params p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t rank = ptx::cluster_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cluster = blockIdx.x >> 1;

    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    auto bar = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };
    auto leader_bar = [&](int i) { return ptx::map_to_rank(bar(i), 0); };
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSRing; ++s) {
            ptx::mbar_init(bar(BAR_SR_FULL + s), 1);
            ptx::mbar_init(bar(BAR_SR_EMPTY + s), 1);
        }
        for (int s = 0; s < kVRing; ++s) {
            ptx::mbar_init(bar(BAR_VR_FULL + s), 1);
            ptx::mbar_init(bar(BAR_VR_EMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar(BAR_S_FULL + b), 1);
            ptx::mbar_init(bar(BAR_S_FREE + b), 16);   // 8 softmax warps x 2 CTAs
        }
        for (int hf = 0; hf < 2; ++hf) {
            ptx::mbar_init(bar(BAR_P_FULL + hf), hf == 0 ? 16 : 8);   // softmax warps of both CTAs
            ptx::mbar_init(bar(BAR_P_FREE + hf), 1);
        }
        ptx::mbar_init(bar(BAR_TAIL_READY), 1);
        ptx::mbar_init(bar(BAR_TAIL_DONE), 16);
        ptx::mbar_init(bar(BAR_DRAIN), 1);
        ptx::mbar_init(bar(BAR_DRAIN_PV), 1);
        for (int g = 0; g < 2; ++g) {
            ptx::mbar_init(bar(BAR_X_FREE + g), 4);
            ptx::mbar_init(bar(BAR_X_FULL + g), 4);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&p.tm_pool);
        ptx::prefetch_tmap(&p.tm_pool_v);
        ptx::prefetch_tmap(&p.tm_qa);
        ptx::prefetch_tmap(&p.tm_qr);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // The sequence lengths and the block table are read first after the wait:
    // bring them into L2 now (a prefetch changes no data, and L2 is coherent
    // with the writes of a kernel still running, so it may precede the wait).
    // Each CTA takes every 148th 128-byte line.
    if (warp >= 4) {
        const char* lens_b = reinterpret_cast<const char*>(p.seq_lens);
        const char* tab_b = reinterpret_cast<const char*>(p.block_table);
        const long n_lens = (static_cast<long>(p.um.B) * 4 + 127) / 128;
        const long n_tab = (static_cast<long>(p.um.B) * p.um.max_blocks * 4 + 127) / 128;
        for (long k = blockIdx.x + static_cast<long>(gridDim.x) * (threadIdx.x - 128); k < n_lens + n_tab;
             k += static_cast<long>(gridDim.x) * (kThreads - 128))
            ptx::prefetch_l2_line(k < n_lens ? lens_b + 128 * k : tab_b + 128 * (k - n_lens));
    }
    // everything below reads what the kernels before this one wrote (q_abs,
    // q^R, the appended cache rows) or what an earlier decode call may still
    // read (the workspace)
    griddep_wait();

    // ---- this cluster's contiguous range of global pages [g0, g1), its first
    // unit u0 (starting at global page ubeg0) and the key counts of its units
    int32_t* kv_s = reinterpret_cast<int32_t*>(smem + kOffSlice);
    int g0 = 0, g1 = 0, u0 = 0, ubeg0 = 0;
    const int32_t* kv_base = kv_s;
    int kv_off = 0;
    if (p.in_kernel_schedule) {
        // scratch: the ring area is unused until the loads start
        int* sc = reinterpret_cast<int*>(smem + kOffSRing);          // page prefix, U + 1
        int* tfx = sc + kInKernelUnits + 1;                           // tile prefix, U + 1
        int* wfx = tfx + kInKernelUnits + 1;                          // cost prefix, U + 1
        int* ctmp = wfx + kInKernelUnits + 1;                         // cut scratch, C + 1
        int* kvx = ctmp + kClusters + 1;                              // key counts, U
        int* wtot = kvx + kInKernelUnits;                             // scan scratch, 48
        const int2 TT = schedule_scan<kShared>(sc, tfx, wfx, kvx, wtot, p.seq_lens, p.U, p.um);
        const int T = TT.x;
        int* cuts = reinterpret_cast<int*>(smem + kOffCuts);
        compute_cuts(cuts, ctmp, sc, tfx, wfx, p.U, T, TT.y, p.max_splits);
        g0 = cuts[cluster];
        g1 = cuts[cluster + 1];
        if (g0 < g1) {
            u0 = unit_of_page(sc, p.U, g0);
            ubeg0 = sc[u0];
            const int u1 = unit_of_page(sc, p.U, g1 - 1);
            int32_t* dst = kv_s;
            if (u1 - u0 + 1 > kSliceCap) {   // only this CTA reads its region
                dst = p.kv_cta + static_cast<size_t>(blockIdx.x) * p.U;
                kv_base = dst;
            }
            for (int k = threadIdx.x; k <= u1 - u0; k += kThreads)
                dst[k] = kvx[u0 + k];
        }
        kv_off = u0;
        // merge metadata and length checks, spread over the grid's threads
        for (int u = blockIdx.x * kThreads + threadIdx.x; u < p.U; u += gridDim.x * kThreads) {
            const int4 m = unit_meta_of<kShared>(u, sc, cuts, kvx[u], p.um);
            p.unit_meta[u] = m;
            if (m.x == 0 && first_of_sequence<kShared>(u, p.um)) raise_status(p.status, MLA_STATUS_BAD_SEQ_LEN);
        }
    } else {
        const int4 cinfo = p.cluster_info[cluster];
        g0 = cinfo.x;
        g1 = cinfo.y;
        u0 = cinfo.z;
        const int n_units = cinfo.w - u0 + 1;   // units u0 .. cinfo.w
        if (g0 < g1) {
            ubeg0 = p.prefix[u0];
            if (n_units <= kSliceCap) {
                for (int k = threadIdx.x; k < n_units; k += kThreads) kv_s[k] = p.unit_kv[u0 + k];
                kv_off = u0;
            } else {
                kv_base = p.unit_kv;
                kv_off = 0;
            }
        }
    }
    ptx::fence_proxy_async_smem();   // the scan's reads of the ring area precede the loads into it
    __syncthreads();   // slice written; the scan scratch is free for the rings

    // Block-table entries are plain global loads.  Each producer issues them a
    // tile or two before it needs them, so that their latency overlaps the
    // ring waits of the tiles in between; an entry is validated where it is
    // used (out-of-range entries are flagged and read as block 0).
    auto load_blk = [&](const Tile& t, int pg) -> int {
        int page = t.page0 + pg;
        if constexpr (kShared) {
            const bool prefix = t.u < p.um.n_prefix;
            if (prefix || (p.um.n_prefix == 0 && page < p.um.n_shared)) return __ldg(p.shared_table + page);
            if (p.um.n_prefix > 0) page += p.um.n_shared;
        }
        return __ldg(p.block_table + static_cast<size_t>(t.b) * p.um.max_blocks + page);
    };
    auto blk_row = [&](int blk) -> int {
        if (blk < 0 || blk >= p.num_blocks) {
            raise_status(p.status, MLA_STATUS_BAD_BLOCK);
            blk = 0;
        }
        return blk * kPage;
    };
    auto walker = [&](TileWalker<kShared>& w) { w.init(kv_base, kv_off, u0, ubeg0, g0, g1, p.um); };

    if (warp < 4) {
        // Warpgroup 0 (loads and MMA issue) needs few registers: it gives them to
        // the softmax warpgroups (setmaxnreg, per warpgroup, at the top of each
        // branch so that the compiler budgets each branch on its own).
        ptx::regs_dec<kRegsIssue>();
        if (warp == 0) {
            // ------------------------------------------------------------ S stream
            // Entry c of a tile holds column chunk c (64 columns) of this CTA's two
            // pages (keys) and of its 64 query rows, one 8 KB box each; the query is
            // re-read from L2 with every tile, which leaves the shared memory to
            // the rings (the loads run at DRAM latency, so the bytes in flight set
            // the rate).  A thread's TMA copies run one after another, so ring slot
            // s is issued by its own group of lanes 4g + {0, 1, 2}, g = s mod
            // kSLaneGroups: lane j = 0, 1 loads own page j, lane 2 the query chunk.
            // The group's lane 0 in the leader CTA arms the full barrier with both
            // CTAs' bytes.  The page lanes hold the block of their page for tiles
            // i, i+1, i+2 in b0, b1, b2.
            const int grp = lane >> 2, j = lane & 3;
            const bool active = grp < kSLaneGroups && j < 3;
            const int my_pg = 2 * static_cast<int>(rank) + (j & 1);
            TileWalker<kShared> w;
            walker(w);
            TileWalker<kShared> wa = w;
            int b0 = 0, b1 = 0, b2 = 0;
            bool h0 = false, h1 = false, h2 = false;
            // (the loads are unconditional, to a valid entry, so that nothing waits
            // for them until their value is used a tile or two later)
            auto look = [&](int& b, bool& h) {
                h = false;
                if (!wa.done()) {
                    const Tile t = wa.next();
                    h = active && j < 2 && my_pg < t.np;
                    b = load_blk(t, min(my_pg, t.np - 1));
                }
            };
            look(b0, h0);
            look(b1, h1);
            look(b2, h2);
            int e = 0;
            bool ok = g0 < g1;
            while (ok && !w.done()) {
                const Tile cur = w.next();
                const int qrow = cur.row0 + 64 * static_cast<int>(rank);
                const int row = h0 ? blk_row(b0) : 0;
                const uint32_t tx = static_cast<uint32_t>(cur.np + 2) * kBox;    // both CTAs' page and query chunks
                for (int c = 0; c < kChunks; ++c, ++e) {
                    const int slot = e % kSRing;
                    bool good = true;
                    if (active && grp == slot % kSLaneGroups) {
                        good = wait_bar(bar(BAR_SR_EMPTY + slot), ((e / kSRing) & 1) ^ 1, abort_flag, p.status, tmo);
                        if (good && j == 0 && rank == 0) ptx::mbar_arrive_expect_tx(bar(BAR_SR_FULL + slot), tx);
                        const bool q_lane = j == 2;
                        const bool withheld = p.withhold_load && rank == 0 && e == 0 && j == 0;
                        if (good && (q_lane || h0) && !withheld) {
                            const void* tm = q_lane ? (c < 8 ? static_cast<const void*>(&p.tm_qa) : &p.tm_qr) : &p.tm_pool;
                            const int bx = q_lane ? (c < 8 ? 64 * c : 0) : 64 * c;
                            ptx::tma_load_2d_pair_normal(sbase + kOffSRing + slot * kSEntry + j * kBox, tm, bx,
                                                         q_lane ? qrow : row, leader_bar(BAR_SR_FULL + slot));
                        }
                    }
                    if (!__all_sync(0xffffffffu, good)) { ok = false; break; }
                }
                b0 = b1; h0 = h1;
                b1 = b2; h1 = h2;
                look(b2, h2);
            }
        } else if (warp == 3) {
            // ------------------------------------------------------------ V stream
            // Entry per page: this CTA's latent chunks 4r .. 4r+3 of the page, one
            // 3-D box, issued by lane (slot) so that consecutive copies come from
            // different threads.  Lane pg < 4 holds the block of page pg of the
            // current tile (v0) and of the next one (v1).
            const uint64_t pol_v = ptx::l2_policy_evict_first();   // last use of these lines
            TileWalker<kShared> w;
            walker(w);
            TileWalker<kShared> wa = w;
            int v0 = 0, v1 = 0;
            auto look = [&](int& v) {
                if (!wa.done()) {
                    const Tile t = wa.next();
                    v = load_blk(t, min(lane, t.np - 1));
                }
            };
            look(v0);
            look(v1);
            int e = 0;
            bool ok = g0 < g1;
            while (ok && !w.done()) {
                const Tile cur = w.next();
                for (int pg = 0; pg < cur.np && ok; ++pg, ++e) {
                    const int row = blk_row(__shfl_sync(0xffffffffu, v0, pg));
                    const int slot = e % kVRing;
                    bool good = true;
                    if (lane == slot) {
                        good = wait_bar(bar(BAR_VR_EMPTY + slot), ((e / kVRing) & 1) ^ 1, abort_flag, p.status, tmo);
                        if (good && rank == 0) ptx::mbar_arrive_expect_tx(bar(BAR_VR_FULL + slot), 2 * kVEntry);
                        if (good)
                            ptx::tma_load_3d_pair(sbase + kOffVRing + slot * kVEntry, &p.tm_pool_v, 0, row,
                                                  4 * static_cast<int>(rank), leader_bar(BAR_VR_FULL + slot), pol_v);
                    }
                    if (!__all_sync(0xffffffffu, good)) { ok = false; break; }
                }
                v0 = v1;
                look(v1);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ S = Q K^T issuer
            // S(i) occupies entries 9 i .. 9 i + 8 of the S ring (keys as B, query as A).
            // The whole warp runs the loop, one lane issues (see elect_one).
            if (rank == 0 && g0 < g1) {
                TileWalker<kShared> w;
                walker(w);
                int i = 0;
                bool ok = true;
                while (ok && !w.done()) {
                    w.next();
                    const int e0 = kChunks * i;
                    const int sb = i & 1;
                    ok = __all_sync(0xffffffffu, wait_bar(bar(BAR_S_FREE + sb), ((i >> 1) & 1) ^ 1, abort_flag, p.status, tmo));
                    if (!ok) break;
                    ptx::tc_fence_after();   // the softmax's reads of this S buffer are done
                    for (int c = 0; c < kChunks; ++c) {
                        const int e = e0 + c;
                        ok = __all_sync(0xffffffffu, wait_bar(bar(BAR_SR_FULL + e % kSRing), (e / kSRing) & 1, abort_flag,
                                                              p.status, tmo));
                        if (!ok) break;
                        if (ptx::elect_one()) {
                            const uint32_t ent = sbase + kOffSRing + (e % kSRing) * kSEntry;
                            const uint64_t b0 = ptx::smem_desc_sw128(ent, 16, 1024);
                            const uint64_t a0 = ptx::smem_desc_sw128(ent + 2 * kBox, 16, 1024);
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4) {
                                const uint64_t a = a0 + static_cast<uint64_t>((32 * k4) >> 4);
                                const uint64_t bd = b0 + static_cast<uint64_t>((32 * k4) >> 4);
                                ptx::mma_pair_ss(tmem_base + kTmemS + 128 * sb, a, bd, kIdescS, (c | k4) ? 1u : 0u);
                            }
                            ptx::mma_commit_pair(bar(BAR_SR_EMPTY + e % kSRing), 0x3);
                            if (c == kChunks - 1) ptx::mma_commit_pair(bar(BAR_S_FULL + sb), 0x3);
                        }
                        __syncwarp();
                    }
                    ++i;
                }
                if (!ok) {
                    // let every MMA this warp issued finish before the teardown frees anything
                    if (ptx::elect_one()) ptx::mma_commit_pair(bar(BAR_DRAIN), 0x1);
                    __syncwarp();
                    const uint64_t t0 = ptx::global_timer_ns();
                    while (!ptx::mbar_try_wait(bar(BAR_DRAIN), 0) && ptx::global_timer_ns() - t0 < tmo) {
                    }
                }
            }
        } else if (warp == 2) {
            if (rank == 0) {
                // -------------------------------------------------------- O += P V issuer
                // V(i) occupies the next np entries of the V ring (one per page).
                if (g0 < g1) {
                    TileWalker<kShared> w;
                    walker(w);
                    int i = 0, tails = 0, e = 0;
                    bool ok = true;
                    const uint64_t a0 = ptx::smem_desc_sw128(sbase + kOffP, 16, 1024);
                    while (ok && !w.done()) {
                        const Tile t = w.next();
                        // P is written in two halves: keys [0,128) (pages 0, 1) by the
                        // softmax warps of TMEM lanes 0-63, keys [128,256) by those of
                        // lanes 64-127; each half is released as soon as its pages'
                        // MMAs complete.
                        for (int pg = 0; pg < 4 && ok; ++pg) {
                            if (pg == 0 || pg == 2) {
                                if (pg == 2) {
                                    if (ptx::elect_one()) ptx::mma_commit_pair(bar(BAR_P_FREE + 0), 0x3);
                                    __syncwarp();
                                }
                                ok = __all_sync(0xffffffffu, wait_bar(bar(BAR_P_FULL + (pg >> 1)), i & 1, abort_flag,
                                                                      p.status, tmo));
                                if (!ok) break;
                                ptx::tc_fence_after();
                            }
                            if (pg >= t.np) continue;
                            ok = __all_sync(0xffffffffu, wait_bar(bar(BAR_VR_FULL + e % kVRing), (e / kVRing) & 1, abort_flag,
                                                                  p.status, tmo));
                            if (!ok) break;
                            if (tail_page<kShared>(t, pg)) {
                                // the page holds rows past the end: now that its V
                                // entry has landed, the softmax warps of both CTAs zero those
                                // rows (entries are consumed in ring order, so the earlier
                                // pages' slots are already free for this load)
                                if (lane < 2) ptx::mbar_arrive_cluster(ptx::map_to_rank(bar(BAR_TAIL_READY), lane));
                                __syncwarp();
                                ok = __all_sync(0xffffffffu, wait_bar<true>(bar(BAR_TAIL_DONE), tails & 1, abort_flag,
                                                                            p.status, tmo));
                                if (!ok) break;
                                ++tails;
                            }
                            if (ptx::elect_one()) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint64_t b0 = ptx::smem_desc_sw128(
                                        sbase + kOffVRing + (e % kVRing) * kVEntry + h * 2 * kBox, kBox, 1024);
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk) {
                                        const uint64_t a = a0 + static_cast<uint64_t>((pg * kBox + 32 * kk) >> 4);
                                        const uint64_t bd = b0 + static_cast<uint64_t>((2048 * kk) >> 4);
                                        ptx::mma_pair_ss(tmem_base + kTmemO + 128 * h, a, bd, kIdescPV,
                                                         (t.first && pg == 0 && kk == 0) ? 0u : 1u);
                                    }
                                }
                                ptx::mma_commit_pair(bar(BAR_VR_EMPTY + e % kVRing), 0x3);
                            }
                            __syncwarp();
                            ++e;
                        }
                        if (!ok) break;
                        if (ptx::elect_one()) ptx::mma_commit_pair(bar(BAR_P_FREE + 1), 0x3);
                        __syncwarp();
                        ++i;
                    }
                    if (!ok) {
                        if (ptx::elect_one()) ptx::mma_commit_pair(bar(BAR_DRAIN_PV), 0x1);
                        __syncwarp();
                        const uint64_t t0 = ptx::global_timer_ns();
                        while (!ptx::mbar_try_wait(bar(BAR_DRAIN_PV), 0) && ptx::global_timer_ns() - t0 < tmo) {
                        }
                    }
                }
            }
        }
    } else {
        ptx::regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax + epilogue
        // Eight warps, two per tensor-memory lane quadrant: a thread owns lane l
        // (head row m, key half hi of the S tile, latent half hi of O) and
        // column group cg (64 of the lane's 128 S columns, 128 of its 256 O
        // columns), so four threads share a head row.
        const int sw = warp - 4;                     // softmax warp 0..7
        const int wq = warp & 3;                     // tensor-memory lane quadrant
        const int cg = sw >> 2;                      // column group
        const int l = wq * 32 + lane;                // lane = (row, half)
        const bool hi = l >= 64;
        const int m = l & 63;
        const int st = sw * 32 + lane;               // 0 .. 255 over the softmax warps
        const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(wq * 32) << 16);
        float* xmax = reinterpret_cast<float*>(smem + kOffXmax);   // [cg][l]
        TileWalker<kShared> w;
        walker(w);
        int i = 0, tails = 0;
        int v_before = 0;      // V ring entries of tiles before i
        bool ok = true;
        float m_used = -INFINITY, l_part = 0.f;
        // this thread's row of the unit and the row's token in a unit of several
        const int unit_row = 64 * static_cast<int>(rank) + m;
        const int row_tok = kShared ? unit_row / p.um.n_h : 0;
        bool saw_inf = false;   // a key that later tokens share scored -inf for this row (see the epilogue)
        // The four partial values of row m (both key halves, both column groups)
        // meet through shared memory: the four warps of 32 rows (group wq & 1)
        // write, wait for each other and read; a warp writes again only when all
        // four have read, which is long past by then.
        const int xg = wq & 1;
        int x_turn = 0;
        auto exchange = [&](float v, bool sum) {
            ok = wait_bar(bar(BAR_X_FREE + xg), (x_turn & 1) ^ 1, abort_flag, p.status, tmo);
            xmax[cg * 128 + l] = v;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BAR_X_FULL + xg));
            ok = ok && wait_bar(bar(BAR_X_FULL + xg), x_turn & 1, abort_flag, p.status, tmo);
            ++x_turn;
            float a = xmax[m], b = xmax[64 + m], c = xmax[128 + m], d = xmax[192 + m];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(BAR_X_FREE + xg));
            if (kShared && sum) {   // the sums carry saw_inf of the row's threads in their signs
                const uint32_t signs = __float_as_uint(a) | __float_as_uint(b) | __float_as_uint(c) | __float_as_uint(d);
                saw_inf = (signs >> 31) != 0;
                a = fabsf(a), b = fabsf(b), c = fabsf(c), d = fabsf(d);
            }
            return sum ? a + b + c + d : fmaxf(fmaxf(a, b), fmaxf(c, d));
        };
        while (ok && !w.done()) {
            const Tile t = w.next();
            // keys of this tile that belong to this segment
            int key_end = min(t.kv, kPage * (t.page0 + t.np));
            if constexpr (kShared) key_end = min(key_end, t.kv - max(0, t.n_tok - 1 - row_tok));
            if (t.first) {
                m_used = -INFINITY;
                l_part = 0.f;
                if constexpr (kShared) saw_inf = false;
            }
            const int sb = i & 1;
            ok = wait_bar(bar(BAR_S_FULL + sb), (i >> 1) & 1, abort_flag, p.status, tmo);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            ptx::tc_fence_after();
            // this thread's 64 scores (row m, keys key0 ..)
            const uint32_t s_col = t_lane + kTmemS + 128 * sb + 64 * cg;
            const int key0 = kPage * t.page0 + (hi ? 128 : 0) + 64 * cg;
            const int nvalid = key_end - key0;   // scores of this thread that count (<= 0 .. >= 64)
            uint32_t r[2][32];
            ptx::tmem_ld32(s_col, r[0]);
            ptx::tmem_ld32(s_col + 32, r[1]);
            ptx::tmem_wait_ld();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_bar(BAR_S_FREE + sb));
            if (nvalid < 64) {   // masked scores
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (j >= nvalid) r[j >> 5][j & 31] = __float_as_uint(-INFINITY);
            }
            if (kShared && t.n_tok > 1 && kPage * (t.page0 + t.np) > t.kv - (t.n_tok - 1)) {
                // rows of the keys from t.kv - (n_tok - 1) on are cleaned below
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    saw_inf |= j < nvalid && key0 + j >= t.kv - (t.n_tok - 1) &&
                               __uint_as_float(r[j >> 5][j & 31]) == -INFINITY;
            }
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // independent chains
#pragma unroll
            for (int j = 0; j < 64; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(r[j >> 5][j & 31]));
            float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            mx = exchange(mx * p.scale_log2, false);   // the scale is positive
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            float new_m = m_used;
            bool resc = false;
            if (mx > m_used + kRescaleThreshold) {
                new_m = mx;
                resc = !t.first;
            }
            float alpha = ex2(m_used - new_m);
            // a row of the shared decode may see none of the keys so far
            if (kShared && new_m == -INFINITY) alpha = 1.f;
            m_used = new_m;

            // The weights of row m, keys key0 + [0, 64) (a masked score's is 2^-inf = 0).
            // The tensor cores take them as bf16 beside the bf16 values (off by 2^-8 of
            // each at most); their sum keeps them in float32, and with it the lse.
            float ps2[2] = {0.f, 0.f};
            const float neg_m = kShared && m_used == -INFINITY ? 0.f : -m_used;
            uint32_t pk[32];
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                const float s0 = __uint_as_float(r[j >> 5][j & 31]), s1 = __uint_as_float(r[j >> 5][(j & 31) + 1]);
                const float p0 = ex2(fmaf(s0, p.scale_log2, neg_m)), p1 = ex2(fmaf(s1, p.scale_log2, neg_m));
                ps2[(j >> 1) & 1] += p0 + p1;
                pk[j >> 1] = pack_bf16x2(p0, p1);
            }
            const float ps = ps2[0] + ps2[1];
            l_part = l_part * alpha + ps;

            // This half of the P buffer must be free (the previous tile's P.V MMAs on
            // it complete); a rescale of O needs the whole previous P.V complete, and
            // half 0's MMAs, which add to every lane of O, need the rescale of all
            // warps: those of half 1 arrive at P_FULL + 0 too.
            const int hf = hi ? 1 : 0;
            const bool any_resc = __any_sync(0xffffffffu, resc);
            ok = wait_bar(bar(BAR_P_FREE + 0), (i & 1) ^ 1, abort_flag, p.status, tmo);
            if (hi && !any_resc && ok && lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_bar(BAR_P_FULL + 0));
            if (ok && (hi || any_resc)) ok = wait_bar(bar(BAR_P_FREE + 1), (i & 1) ^ 1, abort_flag, p.status, tmo);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            ptx::tc_fence_after();
            if (any_resc) {   // (alpha is 1 where the row keeps its maximum)
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    ptx::tmem_ld32(t_lane + kTmemO + 128 * cg + 32 * q, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        o[c] = resc ? __float_as_uint(__uint_as_float(o[c]) * alpha) : o[c];
                    ptx::tmem_st32(t_lane + kTmemO + 128 * cg + 32 * q, o);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (hi && lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_bar(BAR_P_FULL + 0));
            }
            // P row m, keys key0 + [0, 64) = one 64-key block (2 hi + cg) of P:
            // K-major, 128-byte rows, 128-byte swizzle (16-byte chunk index XOR row & 7)
            {
                unsigned char* Pb = smem + kOffP + (2 * hf + cg) * kBox + m * 128;
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    *reinterpret_cast<uint4*>(Pb + ((ch ^ (m & 7)) * 16)) =
                        make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
            }
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster_own(leader_bar(BAR_P_FULL + hf));

            // V ring position of this tile's entries (one per page)
            const int v_start = v_before;
            v_before += t.np;
            for (int pg = kShared ? 0 : t.np - 1; pg < t.np; ++pg) {
                if (!tail_page<kShared>(t, pg)) continue;
                // zero the rows past the end in this CTA's V entry of the page
                // (4 chunks of 64 rows x 128 B)
                ok = wait_bar<true>(bar(BAR_TAIL_READY), tails & 1, abort_flag, p.status, tmo);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                ++tails;
                const int left = t.kv - kPage * (t.page0 + pg);   // keys from the page's first row on
                const int valid = kShared ? max(0, min(left, kPage)) : left;
                const int bad = kPage - valid;
                const int et = v_start + pg;
                unsigned char* ent = smem + kOffVRing + (et % kVRing) * kVEntry;
                for (int x = st; x < 4 * bad * 8; x += 256) {
                    const int chunk = x / (bad * 8);
                    const int rem = x - chunk * bad * 8;
                    const int row = valid + (rem >> 3), ch = rem & 7;
                    reinterpret_cast<uint4*>(ent + chunk * kBox + row * 128)[ch] = make_uint4(0, 0, 0, 0);
                }
                if constexpr (kShared) {
                    // Rows that only the unit's later tokens see: a weight of zero
                    // hides them from the earlier ones, unless they hold infinities
                    // or NaN, which are dropped here.  The tokens that do see such a
                    // row have a score that is not finite: NaN or +inf makes the
                    // weight, and so the output, NaN; -inf a weight of zero, and the
                    // epilogue puts NaN into the columns that lost an infinity.
                    const int from = max(0, left - (t.n_tok - 1)), part = valid - from;
                    for (int x = st; x < 4 * part * 8; x += 256) {
                        const int chunk = x / (part * 8);
                        const int rem = x - chunk * part * 8;
                        uint4* at = reinterpret_cast<uint4*>(ent + chunk * kBox + (from + (rem >> 3)) * 128) + (rem & 7);
                        const uint4 v = *at;
                        const uint4 c = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z),
                                                   finite_bf16x2(v.w));
                        if (c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w) *at = c;
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(leader_bar(BAR_TAIL_DONE));
            }
            if (kShared && !__all_sync(0xffffffffu, ok)) { ok = false; break; }

            if (t.last) {
                // ---- epilogue of this unit segment: wait for P.V of this tile (all
                // warps' P of this tile is in, so every read of the maxima is done)
                ok = wait_bar(bar(BAR_P_FREE + 1), i & 1, abort_flag, p.status, tmo);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                const float lsum = exchange(kShared && saw_inf ? -l_part : l_part, true);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                // A warp of half 0, which does not see every phase of the barrier
                // above, may have passed it a tile early: the exchange orders it
                // behind those of half 1.
                ptx::tc_fence_after();
                // zero: the row sees none of these keys.  A NaN (a score of NaN or +inf)
                // stays one in the lse, so that the merge cannot weigh it away.
                const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
                const float lse = lsum == 0.f ? -INFINITY : (m_used + __log2f(lsum)) * kLn2;
                const bool whole = t.whole && !(kShared && p.um.n_prefix > 0);
                const size_t grow = static_cast<size_t>(t.row0) + unit_row;
                // the first row of the unit's partial slot
                size_t slot_row = (static_cast<size_t>(cluster) + t.u) * 128;
                int warp_rows = 32;   // rows of this warp that belong to the unit
                if constexpr (kShared) {
                    warp_rows = t.rows - (unit_row - lane);
                    if (t.u >= p.um.n_prefix) slot_row = own_slot_row(cluster, t.u - p.um.n_prefix, p.um);
                }
                // This warp's 32 rows (consecutive heads) x the thread's 128
                // latent columns go out through 4 KB tiles written in the
                // 128-byte swizzled layout of a TMA store box (a thread's row of
                // 128 bytes, 16-byte chunk k at k ^ (row & 7)), each tile one
                // bulk tensor store: 4 stores of 32 fp32 columns for a partial,
                // 2 of 64 bf16 columns otherwise.  Between tiles the staging is
                // one 4 KB tile of the free P buffer per warp, reused store
                // after store; after the CTA's last tile no load or MMA touches
                // the rings any more, so every store gets its own tile there
                // and none waits for the one before.
                const bool final_tile = w.done();
                const int h = cg;   // this thread's 128 O columns
                const int col0 = 128 * h + (hi ? 256 : 0);
                const uint32_t stage_off = final_tile ? kOffSRing + sw * 16384u : kOffP + sw * 4096u;
                unsigned char* stage = smem + stage_off;
                const uint32_t stage_u = sbase + stage_off;
                const int x7 = lane & 7;
                const int row0 = whole ? static_cast<int>(grow - lane)
                                       : static_cast<int>(slot_row + unit_row - lane);
#pragma unroll 1
                for (int q = 0; q < (warp_rows > 0 ? 4 : 0); ++q) {
                    uint32_t o[32];
                    ptx::tmem_ld32(t_lane + kTmemO + 128 * h + 32 * q, o);
                    ptx::tmem_wait_ld();
                    if constexpr (kShared) {
                        // 0 inf = NaN for the cleaned infinities that this row sees
                        // (rare: read again from the cache)
                        if (saw_inf)
                            for (int key = max(0, t.kv - (t.n_tok - 1)); key < t.kv - max(0, t.n_tok - 1 - row_tok); ++key)
                                nan_where_infinite(o, p.pool + (static_cast<size_t>(blk_row(load_blk(t, key / kPage - t.page0))) +
                                                                key % kPage) * kRow + col0 + 32 * q);
                        __syncwarp();
                    }
                    if (kShared && whole && warp_rows < 32) {
                        // the store's box would reach into another unit's rows
                        uint4* dst = reinterpret_cast<uint4*>(p.out_latent + grow * kDc + col0 + 32 * q);
                        if (lane < warp_rows) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                dst[k] = make_uint4(
                                    pack_bf16x2(__uint_as_float(o[8 * k + 0]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
                        }
                        continue;
                    }
                    const int tile_k = whole ? (q >> 1) : q;   // this round's store
                    const uint32_t tile_off = final_tile ? 4096u * tile_k : 0u;
                    unsigned char* my_row = stage + tile_off + lane * 128;
                    if (!final_tile && (!whole || (q & 1) == 0)) {
                        if (lane == 0) ptx::bulk_wait_read_all();   // the previous store has read the tile
                        __syncwarp();
                    }
                    if (whole) {
                        // columns 32q .. 32q + 31 are chunks 4 (q & 1) .. + 3 of the staged 64-column row
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 wv;
                            wv.x = pack_bf16x2(__uint_as_float(o[8 * k + 0]) * inv, __uint_as_float(o[8 * k + 1]) * inv);
                            wv.y = pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv);
                            wv.z = pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv);
                            wv.w = pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv);
                            *reinterpret_cast<uint4*>(my_row + (((4 * (q & 1) + k) ^ x7) * 16)) = wv;
                        }
                        if (q & 1) {
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                ptx::tma_store_2d(&p.tm_out, stage_u + tile_off, col0 + 64 * (q >> 1), row0);
                                ptx::bulk_commit_group();
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4*>(my_row + ((k ^ x7) * 16)) =
                                make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                                            __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::tma_store_2d(&p.tm_part, stage_u + tile_off, col0 + 32 * q, row0);
                            ptx::bulk_commit_group();
                        }
                    }
                }
                if (!final_tile) {
                    if (lane == 0) ptx::bulk_wait_read_all();   // the P buffer is written again by the next tile
                    __syncwarp();
                }
                if (!hi && cg == 0 && (!kShared || lane < warp_rows)) {
                    if (whole) p.out_lse[grow] = lse;
                    else p.part_lse[slot_row + unit_row] = lse;
                }
                ptx::tc_fence_before();
            }
            ++i;
        }
    }

    // ---------------------------------------------------------------- teardown
    if (warp >= 4 && lane == 0) ptx::bulk_wait_all();   // the epilogue's stores have completed
    if (*abort_flag) {
        // give copies still in flight time to land before shared memory is released
        const uint64_t t0 = ptx::global_timer_ns();
        while (ptx::global_timer_ns() - t0 < 200000ull) {
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    // The merge kernel may start only now: launched while this grid still
    // runs, its pending blocks slowed the decode down measurably.
    griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// Work schedule for very large unit counts (U > kInKernelUnits): the exclusive
// prefixes of pages, tiles and cut costs per unit, the units' key counts, the
// merge metadata and each cluster's page range, computed by one block of 1024
// threads with the same cut rule as the decode kernel's own scan.
// ---------------------------------------------------------------------------
template <bool kShared>
__global__ void __launch_bounds__(1024)
mla_sm100_schedule_kernel(const int32_t* __restrict__ seq_lens, const UnitMap um, int max_splits, int U,
                          int32_t* __restrict__ prefix, int32_t* __restrict__ tprefix, int32_t* __restrict__ wprefix,
                          int32_t* __restrict__ kv_out, int4* __restrict__ unit_meta,
                          int4* __restrict__ cluster_info, int32_t* status) {
    __shared__ int warp_tot[3][32];
    __shared__ int carry[3];
    griddep_launch_dependents();
    griddep_wait();   // the workspace may still be read by an earlier decode call's kernels
    if (threadIdx.x == 0) carry[0] = carry[1] = carry[2] = 0;
    __syncthreads();
    int32_t* out[3] = {prefix, tprefix, wprefix};
    for (int base = 0; base < U; base += 1024) {
        const int u = base + threadIdx.x;
        int v[3] = {0, 0, 0};   // pages, tiles, cost
        if (u < U) {
            const int kv = unit_keys<kShared>(seq_lens, u, um);
            kv_out[u] = kv;
            v[0] = (kv + kPage - 1) / kPage;
            v[1] = (v[0] + kTilePages - 1) / kTilePages;
            v[2] = unit_cost(v[1]);
        }
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
        for (int q = 0; q < 3; ++q) {   // block inclusive scans
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v[q], o);
                if (lane >= o) v[q] += y;
            }
            if (lane == 31) warp_tot[q][w] = v[q];
        }
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                int t = warp_tot[q][lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, t, o);
                    if (lane >= o) t += y;
                }
                warp_tot[q][lane] = t;
            }
        }
        __syncthreads();
        int incl[3];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            incl[q] = v[q] + (w > 0 ? warp_tot[q][w - 1] : 0) + carry[q];
            if (u < U) out[q][u + 1] = incl[q];
            if (u == 0) out[q][0] = 0;
        }
        __syncthreads();
        if (threadIdx.x == 1023)
            for (int q = 0; q < 3; ++q) carry[q] = incl[q];
        __syncthreads();
    }
    const int T = carry[0], Tt = carry[1];
    __shared__ int cuts[kClusters + 1], cut_tmp[kClusters + 1];
    compute_cuts(cuts, cut_tmp, prefix, tprefix, wprefix, U, T, Tt, max_splits);
    for (int u = threadIdx.x; u < U; u += 1024) {
        const int4 m = unit_meta_of<kShared>(u, prefix, cuts, kv_out[u], um);
        unit_meta[u] = m;
        if (m.x == 0 && first_of_sequence<kShared>(u, um)) raise_status(status, MLA_STATUS_BAD_SEQ_LEN);
    }
    for (int c = threadIdx.x; c < kClusters; c += 1024) {
        const int a = cuts[c], e = cuts[c + 1];
        cluster_info[c] = a < e ? make_int4(a, e, unit_of_page(prefix, U, a), unit_of_page(prefix, U, e - 1))
                                : make_int4(0, 0, 0, 0);
    }
}

// LSE merge of the partial slots: a warp per query row, a lane per 4 x 4 latent
// columns (16-byte loads and 8-byte stores of consecutive lanes).  mla_decode:
// rows of units covered by one cluster were written by the decode kernel; the
// others' partials are the slots meta.y + u .. meta.y + u + meta.z - 1 of unit
// u.  Shared decode with prefix units: every row, from its prefix unit's slots
// and its sequence unit's.  Rows of an invalid sequence (kv_len 0) get zeros
// and lse = -inf.
//
// The partial rows were written by the decode kernel just before and are read
// from L2 (ld.global.cg).  The first slots' rows are fetched together with the
// log-sum-exps, so that a row split in two takes two dependent round trips
// (metadata, then everything else); further slots follow kSlots at a time.
// Blocks of 8 warps; mla_decode's form at most 64 registers a thread: 4 blocks
// per SM, one wave for the 4,096 rows of 32 split units; the shared decode's
// forms up to 80: 3 blocks.  (Blocks of 4 warps doubled the merge
// at prefill sizes, where most of the U x 128 rows belong to whole units and
// the time goes into scheduling blocks that exit at once; one wave of blocks
// that walk the rows was no faster.)
//
// kWarps warps per row, 512 / kWarps columns each, with 2 kWarps partials on
// their way at a time: one for many rows, four for the few rows of a small
// shared decode, which may have dozens of partials each: 16 rows behind 64,000
// shared keys 51.0 us with one warp a row, 43.8 with four (whole call); 464
// rows behind 1,024 keys 23.3 and 23.0.
template <bool kShared, int kWarps>
__global__ void __launch_bounds__(256, kShared ? 3 : 4)
mla_sm100_merge_kernel(const int4* __restrict__ unit_meta, const float* __restrict__ part_o,
                       const float* __restrict__ part_lse, uint16_t* __restrict__ out_latent,
                       float* __restrict__ out_lse, const UnitMap um, int rows) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    // row r: its sequence unit (counted behind the prefix units), its row in
    // the unit, and the output row
    struct Place {
        int uo, unit_row, out;
    };
    auto place = [&](int r) {
        if constexpr (kShared) {
            const int n = r / um.n_h, head = r - n * um.n_h;
            const int b = n / um.T_q, t = n - b * um.T_q;
            const int group = t / um.tok_per_unit;
            const bool many = um.tok_per_unit > 1;
            return Place{(group * um.B + b) * um.n_hb + (many ? 0 : head >> 7),
                         many ? (t - group * um.tok_per_unit) * um.n_h + head : head & 127, r};
        } else {
            const UnitIdx k = unit_index(r >> 7, um.n_hb, um.B);
            return Place{r >> 7, r & 127, (k.b * um.T_q + k.t) * um.n_h + k.hb * 128 + (r & 127)};
        }
    };
    constexpr int kVec = 4 / kWarps;     // 16-byte vectors of a lane
    constexpr int kSlots = 2 * kWarps;   // partials requested together
    const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = warp / kWarps, first_vec = (warp % kWarps) * kVec * 32 + lane;
    if (r >= rows) return;
    const Place at = place(r);
    const int4 own = unit_meta[um.n_prefix + at.uo];
    int4 pre = make_int4(0, 0, 0, 0);
    if (kShared && um.n_prefix > 0) pre = unit_meta[r >> 7];
    uint2* dst = reinterpret_cast<uint2*>(out_latent + static_cast<size_t>(at.out) * kDc) + first_vec;
    if (own.x == 0) {   // the sequence's length is out of range
#pragma unroll
        for (int k = 0; k < kVec; ++k) dst[32 * k] = make_uint2(0, 0);
        if (first_vec == 0) out_lse[at.out] = -INFINITY;
        return;
    }
    const int n_pre = pre.z;
    if (n_pre == 0 && own.z <= 1) return;   // written by the decode kernel
    const int parts = n_pre + own.z;          // <= 2 kClusters
    const size_t pre_row = (static_cast<size_t>(pre.y) + (r >> 7)) * 128 + (r & 127);
    const size_t own_row = (kShared ? own_slot_row(own.y, at.uo, um)
                                    : (static_cast<size_t>(own.y) + at.uo) * 128) + at.unit_row;
    const size_t own_step = kShared ? um.own_rows : 128;
    auto row_of = [&](int i) {
        return kShared && i < n_pre ? pre_row + static_cast<size_t>(i) * 128 : own_row + (i - n_pre) * own_step;
    };
    auto load_slots = [&](float4 (&v)[kSlots][kVec], int i) {   // partials i ..
#pragma unroll
        for (int w = 0; w < kSlots; ++w) {
            if (i + w >= parts) break;
            const float4* a = reinterpret_cast<const float4*>(part_o + row_of(i + w) * kDc) + first_vec;
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[w][k] = __ldcg(a + 32 * k);
        }
    };
    float4 v[kSlots][kVec];
    load_slots(v, 0);
    constexpr int kPer = ((kShared ? 2 : 1) * kClusters + 31) / 32;   // log-sum-exp of partial lane + 32 k
    float ls[kPer];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        ls[k] = lane + 32 * k < parts ? __ldcg(part_lse + row_of(lane + 32 * k)) : -INFINITY;
        mx = fmaxf(mx, ls[k]);
    }
    mx = warp_max(mx);
    auto w_of = [&](float l) { return l == -INFINITY ? 0.f : ex2((l - mx) * kLog2e); };
    float z = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) z += w_of(ls[k]);
    z = warp_sum(z);
    auto weight = [&](int i) {   // partial i's weight, from the lane that holds its log-sum-exp
        float l = ls[0];
#pragma unroll
        for (int k = 1; k < kPer; ++k) l = (i >> 5) == k ? ls[k] : l;
        return w_of(__shfl_sync(0xffffffffu, l, i & 31));
    };
    float4 acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; i += kSlots) {
        if (i > 0) load_slots(v, i);
#pragma unroll
        for (int w = 0; w < kSlots; ++w) {
            if (i + w >= parts) break;             // the same for the whole warp
            const float g = weight(i + w);   // (nothing is skipped at zero: 0 inf of a key at -inf stays NaN)
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                acc[k].x = fmaf(g, v[w][k].x, acc[k].x);
                acc[k].y = fmaf(g, v[w][k].y, acc[k].y);
                acc[k].z = fmaf(g, v[w][k].z, acc[k].z);
                acc[k].w = fmaf(g, v[w][k].w, acc[k].w);
            }
        }
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int k = 0; k < kVec; ++k)
        dst[32 * k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (first_vec == 0) out_lse[at.out] = z == 0.f ? -INFINITY : mx + logf(z);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The pool viewed as [chunk (9)][row][64 columns]: one box loads four 64-column
// chunks of the same 64 rows into consecutive 8 KB blocks.
bool make_map_chunks(CUtensorMap* m, const void* base, uint64_t rows) {
    const cuuint64_t dims[3] = {64, rows, kChunks};
    const cuuint64_t strides[2] = {kRow * 2, 128};
    const cuuint32_t box[3] = {64, 64, 4};
    return encode_tiled_cached(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t r256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Sm100Ws {
    size_t prefix, tprefix, wprefix, kv, kv_cta, meta, cinfo, part_lse, part_o, total;
};

// U units whose partial slots take part_rows rows in all
Sm100Ws sm100_ws(int U, size_t part_rows) {
    Sm100Ws w;
    w.prefix = 0;
    w.tprefix = w.prefix + r256(static_cast<size_t>(U + 1) * 4);
    w.wprefix = w.tprefix + r256(static_cast<size_t>(U + 1) * 4);
    w.kv = w.wprefix + r256(static_cast<size_t>(U + 1) * 4);
    w.kv_cta = w.kv + r256(static_cast<size_t>(U) * 4);
    w.meta = w.kv_cta + r256(static_cast<size_t>(2 * kClusters) * U * 4);
    w.cinfo = w.meta + r256(static_cast<size_t>(U) * 16);
    w.part_lse = w.cinfo + r256(static_cast<size_t>(kClusters) * 16);
    w.part_o = w.part_lse + r256(part_rows * 4);
    w.total = w.part_o + r256(part_rows * kDc * 4);
    return w;
}
Sm100Ws sm100_ws(int U) { return sm100_ws(U, static_cast<size_t>(kClusters + U) * 128); }

// The shared decode's units.
struct SharedPlan {
    UnitMap um;
    long U;
    size_t part_rows;
};

SharedPlan shared_plan(int n_h, int B, int T_q, int max_blocks, int n_shared, bool prefix_units) {
    SharedPlan s;
    s.um.n_h = n_h;
    s.um.n_hb = (n_h + 127) / 128;
    s.um.B = B;
    s.um.T_q = T_q;
    s.um.max_blocks = max_blocks;
    s.um.n_shared = n_shared;
    s.um.n_rows = B * T_q * n_h;
    int per = n_h > 64 ? 1 : 128 / n_h;
    per = per < 64 ? per : 64;
    s.um.tok_per_unit = per < T_q ? per : T_q;
    const int rows = s.um.tok_per_unit > 1 ? s.um.tok_per_unit * n_h : (n_h < 128 ? n_h : 128);
    s.um.own_rows = (rows + 31) / 32 * 32;
    s.um.n_prefix = prefix_units ? (s.um.n_rows + 127) / 128 : 0;
    const long own = static_cast<long>(B) * ((T_q + s.um.tok_per_unit - 1) / s.um.tok_per_unit) * s.um.n_hb;
    s.U = s.um.n_prefix + own;
    s.part_rows = static_cast<size_t>(kClusters + own) * s.um.own_rows +
                  (prefix_units ? static_cast<size_t>(kClusters + s.um.n_prefix) * 128 : 0);
    return s;
}

// Whether the shared pages get units of their own: where the sequences' units
// leave so many of their 128 rows empty that walking the shared pages in each
// of them costs more tiles than the extra units' epilogues and the merge of
// every row.
bool use_prefix_units(int n_h, int B, int T_q, int n_shared) {
    if (n_shared == 0) return false;
    const SharedPlan s = shared_plan(n_h, B, T_q, n_shared, n_shared, true);
    const long own = s.U - s.um.n_prefix;
    return (own - s.um.n_prefix) * ((n_shared + kTilePages - 1) / kTilePages) > s.um.n_prefix + own;
}

// Test hook state: the next launch withholds one load and uses this wait bound.
std::atomic<uint64_t> g_test_wait_limit_ns{0};

}  // namespace

bool sm100_row_shape(int d_c, int d_r) { return d_c == kDc && d_r == kDr; }

bool sm100_supports(int n_h, int d_c, int d_r) { return d_c == kDc && d_r == kDr && n_h % 128 == 0; }

size_t sm100_workspace_bytes(int n_h, int d_c, int B, int T_q) {
    if (n_h % 128 != 0 || d_c != kDc) return 0;
    return sm100_ws(B * T_q * (n_h / 128)).total;
}

int sm100_launches(int B, int T_q, int n_h) {
    const int U = B * T_q * (n_h / 128);
    return U <= kInKernelUnits ? 2 : 3;
}

size_t sm100_unit_meta_offset(int n_h, int B, int T_q) { return sm100_ws(B * T_q * (n_h / 128)).meta; }

void sm100_arm_timeout_test(uint64_t wait_limit_ns) { g_test_wait_limit_ns.store(wait_limit_ns); }

size_t sm100_shared_workspace_bytes(int n_h, int B, int T_q) {
    const SharedPlan s = shared_plan(n_h, B, T_q, 1, 1, true);
    return sm100_ws(static_cast<int>(s.U), s.part_rows).total;
}

namespace {

template <bool kShared>
cudaError_t launch_units(const DecodeParams& P, const UnitMap& um, int U, size_t part_rows, void* ws, int max_splits,
                         cudaStream_t stream) {
    const Sm100Ws w = sm100_ws(U, part_rows);
    char* base = static_cast<char*>(ws);
    Sm100Params k;
    const uint64_t pool_rows = static_cast<uint64_t>(P.num_blocks) * P.block_size;
    const uint64_t q_rows = static_cast<uint64_t>(P.n_tok) * P.n_h;
    if (!make_map_2d(&k.tm_pool, P.pool, kRow, pool_rows, kRow * 2, 64, 64) ||
        !make_map_chunks(&k.tm_pool_v, P.pool, pool_rows) ||
        !make_map_2d(&k.tm_qa, P.q_abs, kDc, q_rows, kDc * 2, 64, 64) ||
        !make_map_2d(&k.tm_qr, P.q_r, kDr, q_rows, kDr * 2, 64, 64) ||
        !make_map_2d(&k.tm_out, P.out_latent, kDc, q_rows, kDc * 2, 64, 32) ||
        !make_map_2d_f32(&k.tm_part, base + w.part_o, kDc, part_rows, kDc * 4, 32, 32))
        return cudaErrorInvalidValue;
    k.block_table = P.block_table;
    k.shared_table = P.shared_table;
    k.pool = P.pool;
    k.seq_lens = P.seq_lens;
    k.prefix = reinterpret_cast<int32_t*>(base + w.prefix);
    k.unit_kv = reinterpret_cast<int32_t*>(base + w.kv);
    k.kv_cta = reinterpret_cast<int32_t*>(base + w.kv_cta);
    k.unit_meta = reinterpret_cast<int4*>(base + w.meta);
    k.cluster_info = reinterpret_cast<const int4*>(base + w.cinfo);
    k.out_latent = P.out_latent;
    k.out_lse = P.out_lse;
    k.part_o = reinterpret_cast<float*>(base + w.part_o);
    k.part_lse = reinterpret_cast<float*>(base + w.part_lse);
    k.status = P.status;
    k.um = um;
    k.U = U;
    k.num_blocks = P.num_blocks;
    k.max_splits = max_splits;
    k.in_kernel_schedule = U <= kInKernelUnits ? 1 : 0;
    const uint64_t test_limit = g_test_wait_limit_ns.exchange(0);
    k.withhold_load = test_limit != 0 ? 1 : 0;
    k.timeout_ns = test_limit != 0 ? test_limit : 2000000000ull;
    k.scale_log2 = P.scale_log2;

    cudaError_t e;
    if (!k.in_kernel_schedule) {
        e = launch_pdl(mla_sm100_schedule_kernel<kShared>, dim3(1), dim3(1024), 0, stream, P.seq_lens, um, max_splits,
                       U, k.prefix, reinterpret_cast<int32_t*>(base + w.tprefix),
                       reinterpret_cast<int32_t*>(base + w.wprefix), k.unit_kv, k.unit_meta,
                       reinterpret_cast<int4*>(base + w.cinfo), P.status);
        if (e != cudaSuccess) return e;
    }
    static std::atomic<uint64_t> smem_set{0};
    e = allow_smem_once(mla_decode_sm100_kernel<kShared>, static_cast<int>(kSmemBytes), smem_set);
    if (e != cudaSuccess) return e;
    e = launch_pdl(mla_decode_sm100_kernel<kShared>, dim3(2 * kClusters), dim3(kThreads), kSmemBytes, stream, k);
    if (e != cudaSuccess) return e;
    const int rows = kShared ? um.n_rows : U * 128;
    // four warps a row, two rows a block, while that makes one wave of three
    // blocks an SM (1,024 rows 28.8 us with four warps a row, 26.4 with one)
    const bool few = kShared && rows <= 2 * kClusters * 3 * 2;
    return launch_pdl(few ? mla_sm100_merge_kernel<kShared, kShared ? 4 : 1> : mla_sm100_merge_kernel<kShared, 1>,
                      dim3(few ? (rows + 1) / 2 : (rows + 7) / 8), dim3(256), 0, stream,
                      static_cast<const int4*>(k.unit_meta), static_cast<const float*>(k.part_o),
                      static_cast<const float*>(k.part_lse), P.out_latent, P.out_lse, um, rows);
}

}  // namespace

cudaError_t launch_decode_sm100(const DecodeParams& P, void* ws, int max_splits, cudaStream_t stream) {
    UnitMap um = {};
    um.n_h = P.n_h;
    um.n_hb = P.n_h / 128;
    um.B = P.B;
    um.T_q = P.T_q;
    um.max_blocks = P.max_blocks;
    const int U = P.B * P.T_q * um.n_hb;
    if (U > 65535) return cudaErrorInvalidValue;
    return launch_units<false>(P, um, U, static_cast<size_t>(kClusters + U) * 128, ws, max_splits, stream);
}

cudaError_t launch_decode_shared_sm100(const DecodeParams& P, void* ws, int max_splits, cudaStream_t stream) {
    const SharedPlan s = shared_plan(P.n_h, P.B, P.T_q, P.max_blocks, P.n_shared,
                                     use_prefix_units(P.n_h, P.B, P.T_q, P.n_shared));
    return launch_units<true>(P, s.um, static_cast<int>(s.U), s.part_rows, ws, max_splits, stream);
}

}  // namespace mla
