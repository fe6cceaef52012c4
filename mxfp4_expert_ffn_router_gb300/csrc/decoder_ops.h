// decoder_ops.h -- internal entry points of the operators around the MoE path: RMS
// norm, the paged key-value cache and attention of one new token.
#pragma once
#include "k3moe_launch.h"

namespace k3moe {

int launch_rmsnorm(int T, int H, const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps,
                   uint16_t *residual_out, uint16_t *y, uint8_t *codes, uint8_t *scales, cudaStream_t st);
int launch_kv_write(const k3moe_kv_cache &c, int n, const uint16_t *k, const uint16_t *v, long long k_stride,
                    long long v_stride, const int32_t *slots, int32_t *status, cudaStream_t st);
int launch_kv_read(const k3moe_kv_cache &c, int n, const int32_t *slots, uint16_t *k_out, uint16_t *v_out,
                   int32_t *status, cudaStream_t st);
size_t attn_decode_workspace(const k3moe_kv_cache &c, int B, int Hq);
int launch_attn_decode(const k3moe_kv_cache &c, int B, int Hq, const uint16_t *q, long long q_stride,
                       const int32_t *table, int max_pages, const int32_t *lens, int window, float scale, uint16_t *out,
                       float *lse, void *ws, int32_t *status, cudaStream_t st);

}  // namespace k3moe
