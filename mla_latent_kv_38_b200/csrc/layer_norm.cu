// Row kernels of the layer around the decode: the norms and residual between
// two blocks, and the quantisation of rows to 8-bit integers.
//
// mla_block_norm, per token's row of d values (formulas in include/mla.h):
//   x = rms(u) w_post, gated;  r = residual + alpha x;  y = rms(r) w_pre
// Bound by memory: 2 d bytes for each of u, residual, r, y (and a per-token
// gate) and two to four operations a value.  A row's values stay in registers
// from the load to the last store, in float32; the sum of squares of r and the
// largest |r w_pre| (the scale of an int8 output) go through one reduction, so
// a row costs one block-wide exchange for each norm.

#include "common.cuh"
#include "kernels.h"
#include "layer.h"

namespace mla {
namespace {

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Added to a float32 of magnitude below 2^22 this rounds it to the nearest even
// integer, which then stands in the low bits: one addition in place of two
// conversions, which run at an eighth of its rate.
constexpr float kRound = 12582912.0f;   // 1.5 x 2^23

// int8 codes of v + kRound (|v| <= 127.5, so no code leaves +-127)
__device__ __forceinline__ uint2 pack_codes(const float* r) {
    auto four = [](const float* f) {
        const uint32_t lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    };
    return make_uint2(four(r), four(r + 4));
}

// Sum and maximum over the threads of one row: a warp (kWarpRow) or the block.
// Consecutive block-wide calls alternate between two halves of `red`, so one
// barrier each is enough: a half is written again only after a barrier that
// every reader of its old values has passed.
template <bool kWarpRow>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2 (*red)[32], int& turn) {
    s = warp_sum(s);
    m = warp_max(m);
    if constexpr (kWarpRow) return make_float2(s, m);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float2* r = red[turn];
    turn ^= 1;
    if (lane == 0) r[warp] = make_float2(s, m);
    __syncthreads();
    const float2 v = lane < warps ? r[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_max(v.y));
}

// The row's operands that a thread holds, as they lie in memory.
template <int V>
struct NormRow {
    uint4 u[V], gate[V], res[V];
};

// V vectors of 8 values per thread; kWarpRow: a row per warp, else per block.
// All of a row's operands are requested together, in front of the first
// reduction, and kAhead requests the block's next row there too: with the
// loads behind the reductions the kernel ran at a third of the memory rate
// (4,096 x 5,120 with a gate per token 94 us, now 36: 5.8 TB/s).  Registers for
// two blocks an SM there; three of fewer registers took 38 to 40 us.
template <int V, bool kWarpRow, bool kAhead>
__global__ void __launch_bounds__(kWarpRow ? 256 : (V <= 2 ? 640 : 512), kWarpRow ? 4 - V : 1)
block_norm_kernel(const BlockNormArgs a) {
    __shared__ float2 red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int turn = 0;
    const int nv = a.d >> 3;
    const int T = kWarpRow ? 32 : blockDim.x;
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int per = kWarpRow ? blockDim.x >> 5 : 1;
    const long step = static_cast<long>(gridDim.x) * per;
    const float inv_d = 1.f / static_cast<float>(a.d);
    auto fetch = [&](NormRow<V>& r, long row) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int j = t + k * T;
            const bool in = j < nv;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            r.u[k] = in ? reinterpret_cast<const uint4*>(a.u + row * a.ld_u)[j] : zero;
            if (a.gate != nullptr) r.gate[k] = in ? reinterpret_cast<const uint4*>(a.gate + row * a.ld_gate)[j] : zero;
            if (a.residual != nullptr)
                r.res[k] = in ? reinterpret_cast<const uint4*>(a.residual + row * a.d)[j] : zero;
        }
    };
    long row = static_cast<long>(blockIdx.x) * per + (kWarpRow ? threadIdx.x >> 5 : 0);
    NormRow<V> cur, next;
    if (row < a.n_tok) fetch(cur, row);
    for (; row < a.n_tok; row += step) {
        if (kAhead && row + step < a.n_tok) fetch(next, row + step);
        float x[V][8];
        float rstd = 1.f;
        if (a.w_post != nullptr) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                unpack8(cur.u[k], x[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(x[k][e], x[k][e], s);
            }
            rstd = rsqrtf(row_reduce<kWarpRow>(s, 0.f, red, turn).x * inv_d + a.eps);
        }
        float s = 0.f, m = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int j = t + k * T;
            if (j >= nv) continue;
            float f[8];
            unpack8(cur.u[k], x[k]);
            if (a.w_post != nullptr) {
                unpack8(reinterpret_cast<const uint4*>(a.w_post)[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] = x[k][e] * rstd * f[e];
            }
            if (a.gate != nullptr) {
                unpack8(cur.gate[k], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] *= f[e];
            }
            if (a.residual != nullptr) {
                unpack8(cur.res[k], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] = fmaf(a.alpha, x[k][e], f[e]);
            }
            if (a.residual_out != nullptr)
                reinterpret_cast<uint4*>(a.residual_out + row * a.d)[j] = pack8(x[k]);
            if (a.w_pre != nullptr) {
                unpack8(reinterpret_cast<const uint4*>(a.w_pre)[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s = fmaf(x[k][e], x[k][e], s);
                    x[k][e] *= f[e];
                    m = fmaxf(m, fabsf(x[k][e]));
                }
            }
        }
        if (a.w_pre != nullptr) {
            const float2 tot = row_reduce<kWarpRow>(s, m, red, turn);
            rstd = rsqrtf(tot.x * inv_d + a.eps);
            // the norm's factor is common to the row: the codes follow from r w_pre
            // alone, taken 2^64 times as large where 127 / max would overflow
            const bool tiny = tot.y < 0x1p-100f;
            const float inv = tot.y > 0.f ? __fdiv_rn(127.f, tiny ? tot.y * 0x1p64f : tot.y) : 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int j = t + k * T;
                if (j >= nv) continue;
                float c[8];
                if (a.out != nullptr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) c[e] = x[k][e] * rstd;
                    reinterpret_cast<uint4*>(a.out + row * a.d)[j] = pack8(c);
                }
                if (a.out8 != nullptr) {
                    if (tiny) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[k][e] *= 0x1p64f;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) c[e] = __fadd_rn(x[k][e] * inv, kRound);
                    reinterpret_cast<uint2*>(a.out8 + row * a.d)[j] = pack_codes(c);
                }
            }
            if (a.out8 != nullptr && t == 0) a.out8_scale[row] = __fdiv_rn(tot.y * rstd, 127.f);
        }
        if (kAhead) cur = next;
        else if (row + step < a.n_tok) fetch(cur, row + step);
    }
}

// Codes and scale of a bf16 row: scale = max / 127, code = round(127 x / max),
// the codes those of exact arithmetic.  A quotient of two 8-bit mantissas times
// 254 that is no integer is at least 2^-17 of itself away from one, so the
// rounded fused product x (127 / max) is right but for quotients of exactly a
// half.  Taken with a factor 2^-21 too small and one as much too large the two
// differ there, and next to there: then the codes are divided for (127 x is
// exact, and the correctly rounded quotient meets a half only where the exact
// one does).  127 x leaves float32's range from 2^121 on, so the division takes
// large rows 2^-32 times as large: what that rounds off lies 2^200 below the
// maximum.  The kernel is bound by these instructions, not by its 3 bytes a
// value: with a division each 40 us for 2,048 rows of 16,384, whose bytes take
// 15.
struct CodeFactor {
    float amax, lo, hi;   // 127 / amax, 2^-21 of it below and above; 0 for a row of zeros
};

__device__ __forceinline__ CodeFactor code_factor(float amax) {
    const float inv = amax > 0.f ? __fdiv_rn(127.f, amax) : 0.f;
    return CodeFactor{amax, inv * (1.f - 0x1p-21f), inv * (1.f + 0x1p-21f)};
}

__device__ __forceinline__ uint2 quantize8(const uint4& w, const CodeFactor& c) {
    float f[8], r[8];
    unpack8(w, f);
    uint32_t differ = c.hi > 3e38f ? 1u : 0u;   // (127 / amax overflows for the smallest rows)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r[e] = __fmaf_rn(f[e], c.lo, kRound);
        differ |= __float_as_uint(r[e]) ^ __float_as_uint(__fmaf_rn(f[e], c.hi, kRound));
    }
    if (differ) {
        const float k = c.amax > 0x1p100f ? 0x1p-32f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = __fadd_rn(c.amax > 0.f ? __fdiv_rn(127.f * (k * f[e]), k * c.amax) : 0.f, kRound);
    }
    return pack_codes(r);
}

// Largest magnitudes of eight values, two bf16 bit patterns at a time (the
// patterns of positive values are in their order).
__device__ __forceinline__ uint32_t amax8(const uint4& w, uint32_t m) {
    const uint32_t a = __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu);
    const uint32_t b = __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu);
    return __vmaxu2(m, __vmaxu2(a, b));
}
__device__ __forceinline__ float amax_of(uint32_t m) {
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

// A block per row, rows with the grid's stride: kCachedRow vectors per thread
// stay in registers between the maximum and the codes, and those of the block's
// next row are requested in front of this row's maximum; the rest of a longer
// row is read twice.
constexpr int kCachedRow = 4;

__global__ void __launch_bounds__(512, 2)
quantize_i8_kernel(const uint16_t* __restrict__ x, long ld_x, int n_rows, int d, int8_t* __restrict__ x8,
                   float* __restrict__ scale) {
    __shared__ float2 red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    int turn = 0;
    const int nv = d >> 3, T = blockDim.x, t = threadIdx.x;
    uint4 v[kCachedRow], next[kCachedRow];
    auto fetch = [&](long row) {
        const uint4* src = reinterpret_cast<const uint4*>(x + row * ld_x);
#pragma unroll
        for (int k = 0; k < kCachedRow; ++k) next[k] = t + k * T < nv ? src[t + k * T] : make_uint4(0, 0, 0, 0);
    };
    long row = blockIdx.x;
    if (row < n_rows) fetch(row);
    for (; row < n_rows; row += gridDim.x) {
#pragma unroll
        for (int k = 0; k < kCachedRow; ++k) v[k] = next[k];
        if (row + gridDim.x < n_rows) fetch(row + gridDim.x);
        const uint4* src = reinterpret_cast<const uint4*>(x + row * ld_x);
        uint2* dst = reinterpret_cast<uint2*>(x8 + row * d);
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kCachedRow; ++k) m = amax8(v[k], m);
        for (int j = t + kCachedRow * T; j < nv; j += T) m = amax8(src[j], m);
        const float amax = row_reduce<false>(0.f, amax_of(m), red, turn).y;
        const CodeFactor c = code_factor(amax);
#pragma unroll
        for (int k = 0; k < kCachedRow; ++k)
            if (t + k * T < nv) dst[t + k * T] = quantize8(v[k], c);
        for (int j = t + kCachedRow * T; j < nv; j += T) dst[j] = quantize8(src[j], c);
        if (t == 0) scale[row] = __fdiv_rn(amax, 127.f);
    }
}

template <int V, bool kWarpRow, bool kAhead>
cudaError_t launch_norm(const BlockNormArgs& a, int threads, int resident, cudaStream_t stream) {
    const int per = kWarpRow ? threads / 32 : 1;
    const long want = (static_cast<long>(a.n_tok) + per - 1) / per;
    const long most = 148L * resident;
    return launch_pdl(block_norm_kernel<V, kWarpRow, kAhead>, dim3(static_cast<unsigned>(want < most ? want : most)),
                      dim3(threads), 0, stream, a);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t stream) {
    const int nv = a.d / 8;
    // blocks that an SM holds at the kernels' registers
    if (nv <= 32) return launch_norm<1, true, true>(a, 256, 3, stream);
    if (nv <= 64) return launch_norm<2, true, true>(a, 256, 2, stream);
    const int threads = ((nv <= 1024 ? (nv + 1) / 2 : (nv + 3) / 4) + 31) / 32 * 32;
    const int fit = 65536 / (threads * 96);
    if (nv <= 1024) return launch_norm<2, false, true>(a, threads, fit > 0 ? fit : 1, stream);
    return launch_norm<4, false, false>(a, threads, 1, stream);
}

cudaError_t launch_quantize_i8(const uint16_t* x, long ld_x, int n_rows, int d, int8_t* x8, float* scale,
                               cudaStream_t stream) {
    const int nv = d / 8;
    // as many threads as the row has vectors for few rows, kCachedRow vectors a
    // thread for many, so that more rows are on their way per SM
    const int want = n_rows <= 2 * 148 ? nv : (nv + kCachedRow - 1) / kCachedRow;
    const int threads = want >= 512 ? 512 : (want + 31) / 32 * 32;
    const int fit = 1024 / threads < 32 ? 1024 / threads : 32;   // resident blocks at 64 registers
    const int most = 148 * fit;
    return launch_pdl(quantize_i8_kernel, dim3(n_rows < most ? n_rows : most), dim3(threads), 0, stream, x, ld_x, n_rows,
                      d, x8, scale);
}

}  // namespace mla
