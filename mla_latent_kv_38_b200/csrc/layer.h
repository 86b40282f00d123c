// Launchers of the layer operators around the decode (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mla {

// Arguments of mla_block_norm, as checked by the entry point.
struct BlockNormArgs {
    const uint16_t* u;
    const uint16_t* w_post;
    const uint16_t* gate;
    const uint16_t* residual;
    const uint16_t* w_pre;
    uint16_t* residual_out;
    uint16_t* out;
    int8_t* out8;
    float* out8_scale;
    long ld_u, ld_gate;
    float alpha, eps;
    int n_tok, d;
};

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t stream);

cudaError_t launch_quantize_i8(const uint16_t* x, long ld_x, int n_rows, int d, int8_t* x8, float* scale,
                               cudaStream_t stream);

cudaError_t launch_linear_i8(const int8_t* x8, long ld_x, const float* x_scale, const int8_t* w8,
                             const float* w_scale, uint16_t* out, int n_tok, int d_in, int d_out, int32_t* status,
                             cudaStream_t stream);

// What a block of the kernel that launch_linear_i8 picks holds: CTAs of a
// cluster, tensor-memory columns and dynamic shared memory.
struct LinearShape {
    int cluster, tmem_cols;
    size_t smem;
};
LinearShape linear_i8_shape(int n_tok, int d_in, int d_out);
// Test hook: the next product withholds one load and bounds its waits by wait_limit_ns.
void linear_i8_arm_timeout_test(uint64_t wait_limit_ns);

// pool: bf16 rows of d_c + d_r values, or (e4m3) rows in the layout of
// mla_e4m3_row_bytes; q, q_c and q_r may be null together
cudaError_t launch_norm_rope_append(const uint16_t* q, const uint16_t* kv, long ld_kv, const uint16_t* w_kv, float eps,
                                    const int32_t* positions, const float* table, int max_pos,
                                    const int32_t* block_table, int max_blocks, void* pool, bool e4m3, int num_blocks,
                                    int n_tok, int T_q, int n_h, int d_c, int d_h, int d_r, int block_size,
                                    uint16_t* q_c, uint16_t* q_r, int32_t* status, cudaStream_t stream);

}  // namespace mla
