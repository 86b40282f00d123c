// Projection in 8-bit integers with a scale per token and per output channel:
//   out[n][o] = (sum_k x8[n][k] w8[o][k]) x_scale[n] w_scale[o]
// (the integer sum is exact: |sum| <= 65,536 x 128^2 = 2^30).

#include "common.cuh"
#include "layer.h"

namespace mla {
namespace {

// 64 tokens x 64 channels per block, 4 x 4 per thread, K in steps of 64 bytes
// through shared memory, four products an instruction (dp4a).
__global__ void __launch_bounds__(256) linear_i8_kernel(const int8_t* __restrict__ x8, long ld_x,
                                                        const float* __restrict__ x_scale,
                                                        const int8_t* __restrict__ w8,
                                                        const float* __restrict__ w_scale, uint16_t* __restrict__ out,
                                                        int n_tok, int d_in, int d_out) {
    __shared__ int xs[16][64 + 1], ws[16][64 + 1];
    griddep_launch_dependents();
    griddep_wait();
    const long n0 = blockIdx.y * 64L, o0 = blockIdx.x * 64L;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < d_in; k0 += 64) {
        for (int e = threadIdx.x; e < 1024; e += 256) {
            const int r = e >> 4, k = e & 15;
            const bool in = k0 + 4 * k < d_in;
            xs[k][r] = in && n0 + r < n_tok ? *reinterpret_cast<const int*>(x8 + (n0 + r) * ld_x + k0 + 4 * k) : 0;
            ws[k][r] = in && o0 + r < d_out ? *reinterpret_cast<const int*>(w8 + (o0 + r) * d_in + k0 + 4 * k) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long n = n0 + ty + 16 * i, o = o0 + tx + 16 * j;
            if (n < n_tok && o < d_out)
                out[n * d_out + o] = f2bf(static_cast<float>(acc[i][j]) * x_scale[n] * w_scale[o]);
        }
}

}  // namespace

cudaError_t launch_linear_i8(const int8_t* x8, long ld_x, const float* x_scale, const int8_t* w8,
                             const float* w_scale, uint16_t* out, int n_tok, int d_in, int d_out, int32_t* status,
                             cudaStream_t stream) {
    (void)status;
    const dim3 grid((d_out + 63) / 64, (n_tok + 63) / 64);
    return launch_pdl(linear_i8_kernel, grid, dim3(256), 0, stream, x8, ld_x, x_scale, w8, w_scale, out, n_tok, d_in,
                      d_out);
}

}  // namespace mla
