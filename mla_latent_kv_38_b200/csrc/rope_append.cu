// Decoupled RoPE on q^R / k^R and the paged append of c^KV || k^R.
//
// "DeepSeek-V2 review" 2.3 and "Техотчёт DeepSeek-V2 (2024): MLA и экономика
// инференса", "Идея 2: отделённый RoPE": the RoPE key k^R is one vector per
// token shared by all heads and is cached after rotation; the query keeps one
// RoPE part per head.  "MLA(Multi-head Latent Attention): DeepSeek-V2
// 논문정리", "MLA 코드 구현": half-split rotate_half pairing, new tokens take
// absolute positions past_len .. T_total-1, and the cache is the latent
// concatenated with the rotated key.
//
// The latent row is a 16-byte vector copy (bit exact), or, into an e4m3 pool,
// its 64-column groups quantised to OCP FP8 E4M3 codes with a float32 scale
// each (layout and rounding in include/mla.h; the pages quote a ~6-bit cache,
// "DeepSeek-V2 review", 4.2 "Inference efficiency", and give no format).
// RoPE is float32 multiply / add with explicit round-to-nearest intrinsics so
// that no fused multiply-add changes the bits, then bf16 round to nearest even.

#include "common.cuh"
#include "kernels.h"
#include "layer.h"

namespace mla {

__device__ __forceinline__ void rope_pair(uint16_t x1b, uint16_t x2b, float c, float s,
                                          uint16_t* y1, uint16_t* y2) {
    const float x1 = bf2f(x1b), x2 = bf2f(x2b);
    const float a = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    const float b = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    *y1 = f2bf(a);
    *y2 = f2bf(b);
}

// Blocks [0, q_blocks) rotate the queries: one thread per (token, head, four
// consecutive pairs m .. m+3), with 8-byte loads of both halves of the head's
// RoPE part and 16-byte loads of the cos / sin rows.  The remaining blocks do
// the cache append, one warp per token.
// One warp quantises a latent row of d_c <= 512 values: lane l takes values
// 16 l .. 16 l + 15, four lanes make a 64-column group.  All 32 lanes take
// part in the group maxima (lanes past d_c / 16 hold zeros).
__device__ __forceinline__ void quantize_values_e4m3(const float (&x)[16], bool active, unsigned char* row,
                                                     int scale_off, int lane) {
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (!active) return;
    const float inv = amax > 0.f ? __fdiv_rn(448.f, amax) : 0.f;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a = e4m3x2_from_f32(__fmul_rn(x[4 * k], inv), __fmul_rn(x[4 * k + 1], inv));
        const uint32_t b = e4m3x2_from_f32(__fmul_rn(x[4 * k + 2], inv), __fmul_rn(x[4 * k + 3], inv));
        w[k] = a | (b << 16);
    }
    *reinterpret_cast<uint4*>(row + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 3) == 0)
        *reinterpret_cast<float*>(row + scale_off + 4 * (lane >> 2)) = amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
}

__device__ __forceinline__ void quantize_row_e4m3(const uint16_t* __restrict__ src, unsigned char* row, int d_c,
                                                  int scale_off, int lane) {
    const bool active = 16 * lane < d_c;
    float x[16];
    if (active) {
        const uint4* s4 = reinterpret_cast<const uint4*>(src + 16 * lane);
        unpack8(s4[0], x);
        unpack8(s4[1], x + 8);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = 0.f;
    }
    quantize_values_e4m3(x, active, row, scale_off, lane);
}

// The zero padding of an e4m3 row.
__device__ __forceinline__ void pad_row_e4m3(unsigned char* row, const E4m3Row& L, int d_c, int d_r, int lane) {
    for (int o = L.scale_off + 4 * (d_c / MLA_E4M3_GROUP) + lane; o < L.kr_off; o += 32) row[o] = 0;
    for (int o = L.kr_off + 2 * d_r + lane; o < L.bytes; o += 32) row[o] = 0;
}

// kE4m3: the pool holds e4m3 rows (row_bytes each, scales at scale_off, the
// bf16 key at kr_off); otherwise bf16 rows of d_c + d_r values.
template <bool kE4m3>
__global__ void __launch_bounds__(256)
rope_append_kernel(uint16_t* __restrict__ q_r, const uint16_t* __restrict__ k_r,
                   const uint16_t* __restrict__ c_kv, const int32_t* __restrict__ positions,
                   const float* __restrict__ table, int max_pos,
                   const int32_t* __restrict__ block_table, int max_blocks,
                   unsigned char* __restrict__ pool, int num_blocks, int n_tok, int T_q,
                   int n_h, int d_c, int d_r, int block_size, int q_blocks, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();   // q_r, the pool and the status word may be in use by earlier kernels
    const int h = d_r >> 1;
    if (static_cast<int>(blockIdx.x) < q_blocks) {
        // ---- query RoPE, in place
        const int quads = h >> 2;
        const long g = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
        if (g >= static_cast<long>(n_tok) * n_h * quads) return;
        const int m = static_cast<int>(g % quads) * 4;
        const long ni = g / quads;                      // token * n_h + head
        const int n = static_cast<int>(ni / n_h);
        const int p = positions[n];
        if (p < 0 || p >= max_pos || p / block_size >= max_blocks) return;   // flagged by the append
        uint16_t* q = q_r + ni * d_r;
        // (the table needs no more than a float's alignment)
        const bool vec = (reinterpret_cast<uintptr_t>(table) & 15u) == 0;
        auto four = [vec](const float* f) {
            return vec ? *reinterpret_cast<const float4*>(f) : make_float4(f[0], f[1], f[2], f[3]);
        };
        const float4 c = four(table + static_cast<size_t>(p) * d_r + m);
        const float4 sn = four(table + static_cast<size_t>(p) * d_r + h + m);
        const uint2 x1 = *reinterpret_cast<const uint2*>(q + m);
        const uint2 x2 = *reinterpret_cast<const uint2*>(q + h + m);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
        const uint32_t a_in[2] = {x1.x, x1.y}, b_in[2] = {x2.x, x2.y};
        uint32_t a_out[2], b_out[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint16_t y1[2], y2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                rope_pair(static_cast<uint16_t>(a_in[w] >> (16 * e)), static_cast<uint16_t>(b_in[w] >> (16 * e)),
                          cc[2 * w + e], ss[2 * w + e], &y1[e], &y2[e]);
            a_out[w] = y1[0] | (static_cast<uint32_t>(y1[1]) << 16);
            b_out[w] = y2[0] | (static_cast<uint32_t>(y2[1]) << 16);
        }
        *reinterpret_cast<uint2*>(q + m) = make_uint2(a_out[0], a_out[1]);
        *reinterpret_cast<uint2*>(q + h + m) = make_uint2(b_out[0], b_out[1]);
        return;
    }

    // ---- cache append, one warp per token
    const int n = (blockIdx.x - q_blocks) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (n >= n_tok) return;
    const int b = n / T_q;
    const int p = positions[n];
    if (p < 0 || p >= max_pos || p / block_size >= max_blocks) {
        if (lane == 0) raise_status(status, MLA_STATUS_BAD_POSITION);
        return;
    }
    const float* cs = table + static_cast<size_t>(p) * d_r;
    const int blk = block_table[static_cast<size_t>(b) * max_blocks + p / block_size];
    if (blk < 0 || blk >= num_blocks) {
        if (lane == 0) raise_status(status, MLA_STATUS_BAD_BLOCK);
        return;
    }
    const size_t slot = static_cast<size_t>(blk) * block_size + (p % block_size);
    uint16_t* key;   // the row's RoPE key (bf16)
    if constexpr (kE4m3) {
        const E4m3Row L = e4m3_row(d_c, d_r);
        unsigned char* row = pool + slot * L.bytes;
        quantize_row_e4m3(c_kv + static_cast<size_t>(n) * d_c, row, d_c, L.scale_off, lane);
        pad_row_e4m3(row, L, d_c, d_r, lane);
        key = reinterpret_cast<uint16_t*>(row + L.kr_off);
    } else {
        uint16_t* row = reinterpret_cast<uint16_t*>(pool) + slot * (d_c + d_r);
        // latent: bit copy in 16-byte vectors
        const uint4* src = reinterpret_cast<const uint4*>(c_kv + static_cast<size_t>(n) * d_c);
        uint4* dst = reinterpret_cast<uint4*>(row);
        for (int v = lane; v < (d_c >> 3); v += 32) dst[v] = src[v];
        key = row + d_c;
    }

    // shared RoPE key
    const uint16_t* kr = k_r + static_cast<size_t>(n) * d_r;
    for (int m = lane; m < h; m += 32) {
        rope_pair(kr[m], kr[m + h], cs[m], cs[h + m], &key[m], &key[m + h]);
    }
}

cudaError_t launch_rope_append(uint16_t* q_r, const uint16_t* k_r, const uint16_t* c_kv,
                               const int32_t* positions, const float* table, int max_pos,
                               const int32_t* block_table, int max_blocks, void* pool, bool e4m3,
                               int num_blocks, int n_tok, int T_q, int n_h, int d_c, int d_r,
                               int block_size, int32_t* status, cudaStream_t stream) {
    const int threads = 256, warps = threads / 32;
    const long q_threads = q_r != nullptr ? static_cast<long>(n_tok) * n_h * (d_r / 8) : 0;
    const long q_blocks = (q_threads + threads - 1) / threads;
    const long a_blocks = (n_tok + warps - 1) / warps;
    if (q_blocks + a_blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(q_blocks + a_blocks));
    unsigned char* p = static_cast<unsigned char*>(pool);
    if (e4m3)
        return launch_pdl(rope_append_kernel<true>, grid, dim3(threads), 0, stream, q_r, k_r, c_kv, positions, table,
                          max_pos, block_table, max_blocks, p, num_blocks, n_tok, T_q, n_h, d_c, d_r, block_size,
                          static_cast<int>(q_blocks), status);
    return launch_pdl(rope_append_kernel<false>, grid, dim3(threads), 0, stream, q_r, k_r, c_kv, positions, table,
                      max_pos, block_table, max_blocks, p, num_blocks, n_tok, T_q, n_h, d_c, d_r, block_size,
                      static_cast<int>(q_blocks), status);
}

// mla_norm_rope_append: the append from the projections' rows.  Blocks
// [0, a_blocks) append, one warp per token: a lane holds 16 latent values, the
// sum of squares is a warp reduction, and the key is rotated as above.  The
// others split query rows, q_chunks blocks per token: the token's items are
// first its heads' copies into q_c (8 values each), then its groups of four
// rotated pairs into q_r, so that a warp does one kind and both outputs are
// written in order; a thread loads its kItems items before it stores any.
// Bound by memory, every byte read once and written once: 2,036 tokens of 128
// heads take 33 us (6.2 TB/s); with the token's position looked up in front of
// its items and four blocks an SM instead of five 39 us.
struct NormAppendArgs {
    const uint16_t* q;
    const uint16_t* kv;
    const uint16_t* w_kv;
    const int32_t* positions;
    const float* table;
    const int32_t* block_table;
    unsigned char* pool;
    uint16_t* q_c;
    uint16_t* q_r;
    int32_t* status;
    long ld_kv;
    float eps;
    int max_pos, max_blocks, num_blocks, n_tok, T_q, n_h, d_c, d_h, d_r, block_size, a_blocks, q_chunks;
};

constexpr int kItems = 4;

template <bool kE4m3>
__global__ void __launch_bounds__(256, 5) norm_rope_append_kernel(const NormAppendArgs a) {
    griddep_launch_dependents();
    griddep_wait();   // the projections, the pool and the outputs may be in use by earlier kernels
    const int h = a.d_r >> 1;
    if (static_cast<int>(blockIdx.x) >= a.a_blocks) {
        const unsigned qb = blockIdx.x - a.a_blocks;
        const unsigned n = qb / a.q_chunks;
        const int p = a.positions[n];   // first used behind the loads of the items
        const unsigned per_c = a.d_h >> 3, per_r = a.d_r >> 3;           // items of one head
        const unsigned copies = a.n_h * per_c, items = copies + a.n_h * per_r;
        const unsigned first = (qb - n * a.q_chunks) * (kItems * 256) + threadIdx.x;
        const uint16_t* src = a.q + static_cast<size_t>(n) * a.n_h * (a.d_h + a.d_r);
        uint4 v[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const unsigned i = first + 256 * k;
            if (i < copies) {
                const unsigned head = i / per_c;
                v[k] = *reinterpret_cast<const uint4*>(src + head * (a.d_h + a.d_r) + 8 * (i - head * per_c));
            } else if (i < items) {
                const unsigned head = (i - copies) / per_r, m = 4 * (i - copies - head * per_r);
                const uint16_t* s = src + head * (a.d_h + a.d_r) + a.d_h + m;
                const uint2 x1 = *reinterpret_cast<const uint2*>(s);
                const uint2 x2 = *reinterpret_cast<const uint2*>(s + h);
                v[k] = make_uint4(x1.x, x1.y, x2.x, x2.y);
            }
        }
        if (p < 0 || p >= a.max_pos || p / a.block_size >= a.max_blocks) return;   // flagged by the append
        uint4* q_c = reinterpret_cast<uint4*>(a.q_c) + static_cast<size_t>(n) * copies;
        uint16_t* q_r = a.q_r + static_cast<size_t>(n) * a.n_h * a.d_r;
        const float* cs = a.table + static_cast<size_t>(p) * a.d_r;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const unsigned i = first + 256 * k;
            if (i < copies) {
                q_c[i] = v[k];
            } else if (i < items) {
                const unsigned head = (i - copies) / per_r, m = 4 * (i - copies - head * per_r);
                const float4 c = *reinterpret_cast<const float4*>(cs + m);
                const float4 sn = *reinterpret_cast<const float4*>(cs + h + m);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
                const uint32_t a_in[2] = {v[k].x, v[k].y}, b_in[2] = {v[k].z, v[k].w};
                uint32_t a_out[2], b_out[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint16_t y1[2], y2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        rope_pair(static_cast<uint16_t>(a_in[w] >> (16 * e)), static_cast<uint16_t>(b_in[w] >> (16 * e)),
                                  cc[2 * w + e], ss[2 * w + e], &y1[e], &y2[e]);
                    a_out[w] = y1[0] | (static_cast<uint32_t>(y1[1]) << 16);
                    b_out[w] = y2[0] | (static_cast<uint32_t>(y2[1]) << 16);
                }
                uint16_t* dst = q_r + head * a.d_r + m;
                *reinterpret_cast<uint2*>(dst) = make_uint2(a_out[0], a_out[1]);
                *reinterpret_cast<uint2*>(dst + h) = make_uint2(b_out[0], b_out[1]);
            }
        }
        return;
    }

    const int n = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (n >= a.n_tok) return;
    const int b = n / a.T_q;
    const int p = a.positions[n];
    if (p < 0 || p >= a.max_pos || p / a.block_size >= a.max_blocks) {
        if (lane == 0) raise_status(a.status, MLA_STATUS_BAD_POSITION);
        return;
    }
    const int blk = a.block_table[static_cast<size_t>(b) * a.max_blocks + p / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) raise_status(a.status, MLA_STATUS_BAD_BLOCK);
        return;
    }
    const size_t slot = static_cast<size_t>(blk) * a.block_size + (p % a.block_size);
    const uint16_t* src = a.kv + n * a.ld_kv;

    // 16 consecutive latent values per lane (vectors 2 lane, 2 lane + 1)
    const int nv = a.d_c >> 3;
    float x[16], w[16];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = 2 * lane + k;
        if (j < nv) {
            unpack8(reinterpret_cast<const uint4*>(src)[j], x + 8 * k);
            unpack8(reinterpret_cast<const uint4*>(a.w_kv)[j], w + 8 * k);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * k + e] = w[8 * k + e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[8 * k + e], x[8 * k + e], s);
    }
    const float rstd = rsqrtf(warp_sum(s) / static_cast<float>(a.d_c) + a.eps);
    uint32_t y[8];   // the normed latent, rounded once to bf16
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = pack_bf16x2(x[2 * k] * rstd * w[2 * k], x[2 * k + 1] * rstd * w[2 * k + 1]);
    uint16_t* key;
    if constexpr (kE4m3) {
        const E4m3Row L = e4m3_row(a.d_c, a.d_r);
        unsigned char* row = a.pool + slot * L.bytes;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[2 * k] = __uint_as_float(y[k] << 16);
            x[2 * k + 1] = __uint_as_float(y[k] & 0xFFFF0000u);
        }
        quantize_values_e4m3(x, 16 * lane < a.d_c, row, L.scale_off, lane);
        pad_row_e4m3(row, L, a.d_c, a.d_r, lane);
        key = reinterpret_cast<uint16_t*>(row + L.kr_off);
    } else {
        uint16_t* row = reinterpret_cast<uint16_t*>(a.pool) + slot * (a.d_c + a.d_r);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * lane + k < nv)
                reinterpret_cast<uint4*>(row)[2 * lane + k] =
                    make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        key = row + a.d_c;
    }
    const float* cs = a.table + static_cast<size_t>(p) * a.d_r;
    const uint16_t* kr = src + a.d_c;
    for (int m = lane; m < h; m += 32) rope_pair(kr[m], kr[m + h], cs[m], cs[h + m], &key[m], &key[m + h]);
}

cudaError_t launch_norm_rope_append(const uint16_t* q, const uint16_t* kv, long ld_kv, const uint16_t* w_kv, float eps,
                                    const int32_t* positions, const float* table, int max_pos,
                                    const int32_t* block_table, int max_blocks, void* pool, bool e4m3, int num_blocks,
                                    int n_tok, int T_q, int n_h, int d_c, int d_h, int d_r, int block_size,
                                    uint16_t* q_c, uint16_t* q_r, int32_t* status, cudaStream_t stream) {
    const int threads = 256, warps = threads / 32;
    const long q_chunks = (static_cast<long>(n_h) * ((d_h + d_r) / 8) + kItems * threads - 1) / (kItems * threads);
    const long q_blocks = q != nullptr ? n_tok * q_chunks : 0;
    const long a_blocks = (n_tok + warps - 1) / warps;
    if (q_blocks + a_blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    NormAppendArgs a;
    a.q = q, a.kv = kv, a.w_kv = w_kv, a.positions = positions, a.table = table, a.block_table = block_table;
    a.pool = static_cast<unsigned char*>(pool), a.q_c = q_c, a.q_r = q_r, a.status = status;
    a.ld_kv = ld_kv, a.eps = eps, a.max_pos = max_pos, a.max_blocks = max_blocks, a.num_blocks = num_blocks;
    a.n_tok = n_tok, a.T_q = T_q, a.n_h = n_h, a.d_c = d_c, a.d_h = d_h, a.d_r = d_r, a.block_size = block_size;
    a.a_blocks = static_cast<int>(a_blocks), a.q_chunks = static_cast<int>(q_chunks);
    const dim3 grid(static_cast<unsigned>(q_blocks + a_blocks));
    return launch_pdl(e4m3 ? norm_rope_append_kernel<true> : norm_rope_append_kernel<false>, grid, dim3(threads), 0,
                      stream, a);
}

}  // namespace mla
