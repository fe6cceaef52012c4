// attn_decode.cu -- attention of one new token per sequence over a paged key-value cache.
//
// For sequence b with n = seq_lens[b] cached tokens, of which those at places
// lo = max(0, n - window) (0 without a window) .. n - 1 are seen, and query head h
// of key-value head g = h / (Hq / heads):
//   s_i = scale * q . K_i,  m = max s_i,  l = sum exp(s_i - m),
//   out = sum exp(s_i - m) V_i / l,  lse = m + log l
// A row that sees nothing (or only scores of -inf) gives out = 0 and lse = -inf.
//
// One block per (b, h); four warps take every fourth token and hold running m, l and
// the weighted sum in fp32 (a lane: dim / 32 dimensions), joined in shared memory.
#include <cuda_fp16.h>

#include "k3moe_dev.cuh"
#include "k3moe_launch.h"
#include "mx8_quant.cuh"

namespace k3moe {

namespace {

constexpr int kAdWarps = 4;

template <int D, bool E4M3>
__device__ __forceinline__ void load_vec(const void *base, const uint8_t *scales, size_t vec, int lane, float (&f)[D / 32]) {
  constexpr int P = D / 32;
  if constexpr (E4M3) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + vec * D + lane * P;
    const float x = e8m0_to_f32(scales[vec]);
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      uint32_t h, unused;
      e4m3x4_to_f16x2(*reinterpret_cast<const uint16_t *>(p + i), h, unused);
      const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      f[i] = v.x * x;
      f[i + 1] = v.y * x;
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + vec * D + lane * P;
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = bf16_bits_to_f32(p[i]);
  }
}

}  // namespace

template <int D, bool E4M3>
__global__ void __launch_bounds__(kAdWarps * 32)
    attn_decode_kernel(k3moe_kv_cache c, int page_shift, int Hq, const uint16_t *__restrict__ q, long long q_stride,
                       const int32_t *__restrict__ table, int max_pages, const int32_t *__restrict__ lens, int window,
                       float scale, uint16_t *__restrict__ out, float *__restrict__ lse, int32_t *status) {
  constexpr int P = D / 32;
  __shared__ float s_m[kAdWarps], s_l[kAdWarps], s_o[kAdWarps][D];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, h = blockIdx.x, g = h / (Hq / c.heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long most = static_cast<long long>(max_pages) << page_shift;
  int n = lens[b];
  if (n < 0 || n > most) {
    if (threadIdx.x == 0) set_status(status, K3MOE_DEV_BOUNDS);
    n = n < 0 ? 0 : static_cast<int>(most);
  }
  const int lo = window > 0 && n > window ? n - window : 0;
  float qv[P], o[P], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    qv[i] = bf16_bits_to_f32(q[b * q_stride + static_cast<size_t>(h) * D + lane * P + i]);
    o[i] = 0.f;
  }
  for (int t = lo + warp; t < n; t += kAdWarps) {
    const int page = table[static_cast<size_t>(b) * max_pages + (t >> page_shift)];
    if (page < 0 || page >= c.pages) {
      if (lane == 0) set_status(status, K3MOE_DEV_BOUNDS);
      continue;
    }
    const size_t vec = ((static_cast<size_t>(page) * c.heads + g) << page_shift) + (t & ((1 << page_shift) - 1));
    float kv[P], vv[P], s = 0.f;
    load_vec<D, E4M3>(c.k, c.k_scales, vec, lane, kv);
    load_vec<D, E4M3>(c.v, c.v_scales, vec, lane, vv);
#pragma unroll
    for (int i = 0; i < P; ++i) s = fmaf(qv[i], kv[i], s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float al = expf(m - base), p = expf(s - base);
    l = fmaf(l, al, p);
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = fmaf(o[i], al, p * vv[i]);
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) s_o[warp][lane * P + i] = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float mt = s_m[0];
  for (int w = 1; w < kAdWarps; ++w) mt = fmaxf(mt, s_m[w]);
  const float base = mt == -INFINITY ? 0.f : mt;
  float lt = 0.f;
  for (int w = 0; w < kAdWarps; ++w) lt += s_l[w] * expf(s_m[w] - base);
  const size_t row = static_cast<size_t>(b) * Hq + h;
  for (int d = threadIdx.x; d < D; d += kAdWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kAdWarps; ++w) v += s_o[w][d] * expf(s_m[w] - base);
    out[row * D + d] = f32_to_bf16_rne(lt == 0.f ? 0.f : v / lt);
  }
  if (lse && threadIdx.x == 0) lse[row] = base + logf(lt);
}

size_t attn_decode_workspace(const k3moe_kv_cache &, int, int) { return 0; }

int launch_attn_decode(const k3moe_kv_cache &c, int B, int Hq, const uint16_t *q, long long q_stride,
                       const int32_t *table, int max_pages, const int32_t *lens, int window, float scale, uint16_t *out,
                       float *lse, void *, int32_t *status, cudaStream_t st) {
  int sh = 0;
  while ((1 << sh) < c.page_size) ++sh;
  const dim3 grid(Hq, B), block(kAdWarps * 32);
  const bool e = c.format == K3MOE_KV_E4M3;
  cudaError_t err = cudaErrorInvalidValue;
#define K3_AD(D_)                                                                                                   \
  if (c.dim == D_)                                                                                                  \
    err = e ? launch_pdl(attn_decode_kernel<D_, true>, grid, block, 0, st, c, sh, Hq, q, q_stride, table, max_pages, \
                         lens, window, scale, out, lse, status)                                                     \
            : launch_pdl(attn_decode_kernel<D_, false>, grid, block, 0, st, c, sh, Hq, q, q_stride, table, max_pages, \
                         lens, window, scale, out, lse, status);
  K3_AD(64) K3_AD(128) K3_AD(256)
#undef K3_AD
  return err == cudaSuccess ? 0 : -1;
}

}  // namespace k3moe
