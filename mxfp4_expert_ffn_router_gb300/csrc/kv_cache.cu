// kv_cache.cu -- the paged key-value cache: new tokens' keys and values written into
// their slots (quantised on the way, mx8_quant.cuh), and slots read back as bf16.
//
// A cache holds [pages][heads][page_size][dim] values, so that one head's tokens of a
// page are contiguous: that is what attention streams.  A slot is page * page_size +
// place.  A negative slot is padding (not written; reads as zeros); one at or past the
// end sets K3MOE_DEV_BOUNDS and is treated the same.
//
// dim / 8 neighbouring lanes hold one vector (a token's key or value of one head), 16
// bytes of bf16 each; its scale needs one maximum over those lanes.
#include <cuda_fp16.h>

#include "k3moe_dev.cuh"
#include "k3moe_launch.h"
#include "mx8_quant.cuh"

namespace k3moe {

namespace {

struct KvView {
  uint8_t *k, *v, *ks, *vs;
  int heads, page_shift, places;  // places = pages * page_size
};

KvView view_of(const k3moe_kv_cache &c) {
  int sh = 0;
  while ((1 << sh) < c.page_size) ++sh;
  return {static_cast<uint8_t *>(c.k), static_cast<uint8_t *>(c.v), c.k_scales, c.v_scales,
          c.heads, sh, c.pages * c.page_size};
}

// Index of the vector of (slot, head) in the cache.
__device__ __forceinline__ size_t vec_index(const KvView &c, int slot, int head) {
  const size_t page = static_cast<size_t>(slot >> c.page_shift);
  return (((page * c.heads + head) << c.page_shift) + (slot & ((1 << c.page_shift) - 1)));
}

}  // namespace

// Vector i of 2 n heads: token i / (2 heads), key or value (i / heads) % 2, head i % heads.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256)
    kv_write_kernel(KvView c, int n, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, long long k_stride,
                    long long v_stride, const int32_t *__restrict__ slots, int32_t *status) {
  constexpr int L = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long total = 2LL * n * c.heads;
  const long long step = static_cast<long long>(gridDim.x) * (256 / L);
  const int sub = threadIdx.x % L;
  for (long long i0 = static_cast<long long>(blockIdx.x) * (256 / L); i0 < total; i0 += step) {
    const long long i = i0 + threadIdx.x / L;
    const bool in = i < total;
    const int t = in ? static_cast<int>(i / (2 * c.heads)) : 0;
    const int r = in ? static_cast<int>(i - static_cast<long long>(t) * 2 * c.heads) : 0;
    const bool val = r >= c.heads;
    const int head = val ? r - c.heads : r;
    const int slot = in ? slots[t] : -1;
    const bool live = slot >= 0 && slot < c.places;
    if (slot >= c.places && r == 0 && sub == 0) set_status(status, K3MOE_DEV_BOUNDS);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live)
      u = *(reinterpret_cast<const uint4 *>((val ? v + t * v_stride : k + t * k_stride) + static_cast<size_t>(head) * D) +
            sub);
    const size_t o = live ? vec_index(c, slot, head) : 0;
    uint8_t *dst = val ? c.v : c.k;
    if constexpr (!E4M3) {
      if (live) *(reinterpret_cast<uint4 *>(dst + o * (2 * D)) + sub) = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float f[8];
      uint32_t m = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = __uint_as_float(w[q] << 16);
        f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        m = max(m, max((w[q] << 16) & 0x7FFFFFFFu, w[q] & 0x7FFF0000u));
      }
#pragma unroll
      for (int off = 1; off < L; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const uint32_t byte = mx8_scale_byte(m);
      if (live) {
        *(reinterpret_cast<uint2 *>(dst + o * D) + sub) = mx8_codes(f, byte);
        if (sub == 0) (val ? c.vs : c.ks)[o] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// k_out, v_out: bf16 [n][heads][D].
template <int D, bool E4M3>
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvView c, int n, const int32_t *__restrict__ slots, uint16_t *__restrict__ k_out,
                   uint16_t *__restrict__ v_out, int32_t *status) {
  constexpr int L = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long total = 2LL * n * c.heads;
  const long long step = static_cast<long long>(gridDim.x) * (256 / L);
  const int sub = threadIdx.x % L;
  for (long long i = static_cast<long long>(blockIdx.x) * (256 / L) + threadIdx.x / L; i < total; i += step) {
    const int t = static_cast<int>(i / (2 * c.heads));
    const int r = static_cast<int>(i - static_cast<long long>(t) * 2 * c.heads);
    const bool val = r >= c.heads;
    const int head = val ? r - c.heads : r;
    const int slot = slots[t];
    if (slot >= c.places && r == 0 && sub == 0) set_status(status, K3MOE_DEV_BOUNDS);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < c.places) {
      const size_t o = vec_index(c, slot, head);
      const uint8_t *src = val ? c.v : c.k;
      if constexpr (!E4M3) {
        u = *(reinterpret_cast<const uint4 *>(src + o * (2 * D)) + sub);
      } else {
        const uint2 w = *(reinterpret_cast<const uint2 *>(src + o * D) + sub);
        const float x = e8m0_to_f32((val ? c.vs : c.ks)[o]);
        uint32_t h[4], out[4];
        e4m3x4_to_f16x2(w.x, h[0], h[1]);
        e4m3x4_to_f16x2(w.y, h[2], h[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // code * X is exact in fp32, and in bf16 above 2^-124
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[q]));
          out[q] = f32_to_bf16_rne(f.x * x) | (static_cast<uint32_t>(f32_to_bf16_rne(f.y * x)) << 16);
        }
        u = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    *(reinterpret_cast<uint4 *>((val ? v_out : k_out) + (static_cast<size_t>(t) * c.heads + head) * D) + sub) = u;
  }
}

namespace {

// Blocks for `vectors` vectors of L lanes: every vector at once, up to 16 blocks an SM.
dim3 kv_grid(long long vectors, int L) {
  const long long per = 256 / L;
  long long g = (vectors + per - 1) / per;
  const long long most = static_cast<long long>(sm_count()) * 16;
  return dim3(static_cast<unsigned>(g < most ? g : most));
}

}  // namespace

int launch_kv_write(const k3moe_kv_cache &c, int n, const uint16_t *k, const uint16_t *v, long long k_stride,
                    long long v_stride, const int32_t *slots, int32_t *status, cudaStream_t st) {
  const KvView w = view_of(c);
  const dim3 grid = kv_grid(2LL * n * c.heads, c.dim / 8), block(256);
  const bool q = c.format == K3MOE_KV_E4M3;
  cudaError_t err = cudaErrorInvalidValue;
#define K3_KV(D_)                                                                                                  \
  if (c.dim == D_)                                                                                                 \
    err = q ? launch_pdl(kv_write_kernel<D_, true>, grid, block, 0, st, w, n, k, v, k_stride, v_stride, slots, status) \
            : launch_pdl(kv_write_kernel<D_, false>, grid, block, 0, st, w, n, k, v, k_stride, v_stride, slots, status);
  K3_KV(64) K3_KV(128) K3_KV(256)
#undef K3_KV
  return err == cudaSuccess ? 0 : -1;
}

int launch_kv_read(const k3moe_kv_cache &c, int n, const int32_t *slots, uint16_t *k_out, uint16_t *v_out,
                   int32_t *status, cudaStream_t st) {
  const KvView w = view_of(c);
  const dim3 grid = kv_grid(2LL * n * c.heads, c.dim / 8), block(256);
  const bool q = c.format == K3MOE_KV_E4M3;
  cudaError_t err = cudaErrorInvalidValue;
#define K3_KV(D_)                                                                                              \
  if (c.dim == D_)                                                                                             \
    err = q ? launch_pdl(kv_read_kernel<D_, true>, grid, block, 0, st, w, n, slots, k_out, v_out, status)       \
            : launch_pdl(kv_read_kernel<D_, false>, grid, block, 0, st, w, n, slots, k_out, v_out, status);
  K3_KV(64) K3_KV(128) K3_KV(256)
#undef K3_KV
  return err == cudaSuccess ? 0 : -1;
}

}  // namespace k3moe
