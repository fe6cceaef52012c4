// decoder_ops.h -- internal entry points of the operators around the MoE path: RMS
// norm, the paged key-value cache and attention of one new token, or of several of a sequence.
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
int launch_kv_append(const k3moe_kv_cache &c, int n, int Hq, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                     long long q_stride, long long k_stride, long long v_stride, const int32_t *slots,
                     const int32_t *positions, const k3moe_rotation &rot, uint16_t *q_out, long long q_out_stride,
                     int32_t *status, cudaStream_t st);

// Attention of several new tokens of a sequence (masks: those of drafted tokens, or null: each sees those before it).
struct ExtendArgs {
  k3moe_kv_cache c;
  int B, rows, Hq;
  const uint16_t *q;
  long long q_stride;
  const int32_t *offsets;
  int max_new;
  const uint64_t *masks;
  int words;
  const int32_t *table;
  int max_pages;
  const int32_t *lens;
  int window, sinks;
  float scale;
  uint16_t *out;
  float *lse;
  void *ws;
  int32_t *status;
};
// The same for at most one new token a sequence, without masks (attn_sinks.cu), and where a key-value head's rows of a
// sequence are few (attn_rows.cu: rows of sequences with more than `most` of them a head are left alone); the workspace is
// that of both.
size_t attn_rows_workspace(const k3moe_kv_cache &c);
int launch_attn_sinks(const ExtendArgs &a, cudaStream_t st);
int launch_attn_rows(const ExtendArgs &a, int most, cudaStream_t st);
size_t attn_extend_workspace(const k3moe_kv_cache &c, int B, int rows, int Hq);
int launch_attn_extend(const ExtendArgs &a, cudaStream_t st);

}  // namespace k3moe
