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
//
// Bound: the bytes, once in and once out.  Four tokens in flight a thread where there are enough
// of them: reading 16384 tokens of 8 heads of 128 (101 MB) 17.4 us, 5.8 TB/s (one in flight 22.2 us,
// eight 19.8); writing 4096 tokens (25 MB) 5.5 us, of which about 2 are the launch (6.2 with one);
// 13 tokens of 96 heads 1.9 us with one in flight, 2.1 with four.
#include <cuda_fp16.h>

#include <type_traits>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
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

// Block (x, y): TOKENS tokens from x TOKENS on, of head y (keys) or y - heads (values): neighbouring
// tokens mostly have neighbouring slots, so that a block's stores are one stretch of the
// cache.  A group of D / 8 lanes takes every (256 / L)th of the block's tokens, U in all, loading
// all of them before the first use.  U = 4 where that leaves two blocks an SM, else 1.
template <int D, int U_>
struct KvTile {
  static constexpr int L = D / 8, G = 256 / L, U = U_, TOKENS = G * U;
};

template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256)
    kv_write_kernel(KvView c, int n, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, long long k_stride,
                    long long v_stride, const int32_t *__restrict__ slots, int32_t *status) {
  using K = KvTile<D, U>;
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % K::L;
  const bool val = static_cast<int>(blockIdx.y) >= c.heads;
  const int head = val ? blockIdx.y - c.heads : blockIdx.y;
  const uint16_t *src = (val ? v : k) + static_cast<size_t>(head) * D + sub * 8;
  const long long stride = val ? v_stride : k_stride;
  uint8_t *dst = val ? c.v : c.k, *dst_scales = val ? c.vs : c.ks;
  const int t0 = blockIdx.x * K::TOKENS + threadIdx.x / K::L;
  int slot[K::U];
  uint4 u[K::U];
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    const int t = t0 + i * K::G;
    slot[i] = t < n ? __ldg(slots + t) : -1;
    u[i] = make_uint4(0, 0, 0, 0);
    if (t < n) u[i] = __ldg(reinterpret_cast<const uint4 *>(src + t * stride));
  }
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    if (slot[i] >= c.places) {
      if (blockIdx.y == 0 && sub == 0) set_status(status, K3MOE_DEV_BOUNDS);
      slot[i] = -1;
    }
    const size_t o = slot[i] >= 0 ? vec_index(c, slot[i], head) : 0;
    if constexpr (!E4M3) {
      if (slot[i] >= 0) *(reinterpret_cast<uint4 *>(dst + o * (2 * D)) + sub) = u[i];
    } else {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      float f[8];
      uint32_t m = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = __uint_as_float(w[q] << 16);
        f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        m = max(m, max((w[q] << 16) & 0x7FFFFFFFu, w[q] & 0x7FFF0000u));
      }
#pragma unroll
      for (int off = 1; off < K::L; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const uint32_t byte = mx8_scale_byte(m);
      if (slot[i] >= 0) {
        *(reinterpret_cast<uint2 *>(dst + o * D) + sub) = mx8_codes(f, byte);
        if (sub == 0) dst_scales[o] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// k_out, v_out: bf16 [n][heads][D].
template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvView c, int n, const int32_t *__restrict__ slots, uint16_t *__restrict__ k_out,
                   uint16_t *__restrict__ v_out, int32_t *status) {
  using K = KvTile<D, U>;
  using Word = std::conditional_t<E4M3, uint2, uint4>;  // eight values
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % K::L;
  const bool val = static_cast<int>(blockIdx.y) >= c.heads;
  const int head = val ? blockIdx.y - c.heads : blockIdx.y;
  const uint8_t *src = val ? c.v : c.k, *src_scales = val ? c.vs : c.ks;
  uint16_t *out = (val ? v_out : k_out) + static_cast<size_t>(head) * D;
  const int t0 = blockIdx.x * K::TOKENS + threadIdx.x / K::L;
  int slot[K::U];
  Word w[K::U];
  uint32_t byte[K::U];
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    const int t = t0 + i * K::G;
    slot[i] = t < n ? __ldg(slots + t) : -1;
  }
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    if (slot[i] >= c.places) {
      if (blockIdx.y == 0 && sub == 0) set_status(status, K3MOE_DEV_BOUNDS);
      slot[i] = -1;
    }
    w[i] = Word{};
    byte[i] = 127u;
    if (slot[i] >= 0) {
      const size_t o = vec_index(c, slot[i], head);
      w[i] = *(reinterpret_cast<const Word *>(src + o * (E4M3 ? D : 2 * D)) + sub);
      if constexpr (E4M3) byte[i] = src_scales[o];
    }
  }
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    const int t = t0 + i * K::G;
    if (t >= n) continue;
    uint4 u;
    if constexpr (E4M3) {
      const float x = e8m0_to_f32(byte[i]);
      uint32_t h[4], r[4];
      e4m3x4_to_f16x2(w[i].x, h[0], h[1]);
      e4m3x4_to_f16x2(w[i].y, h[2], h[3]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // code * X is exact in fp32, and in bf16 above 2^-124
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[q]));
        r[q] = bf16x2(f.x * x, f.y * x);
      }
      u = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      u = w[i];
    }
    *(reinterpret_cast<uint4 *>(out + static_cast<size_t>(t) * c.heads * D) + sub) = u;
  }
}

namespace {

// Calls f(dim, whether E4M3, U, grid), the first three as types' values.
template <class F>
int kv_dispatch(const k3moe_kv_cache &c, int n, F f) {
  auto with = [&](auto D, auto E, auto U) {
    using K = KvTile<decltype(D)::value, decltype(U)::value>;
    return f(D, E, U, dim3((n + K::TOKENS - 1) / K::TOKENS, 2 * c.heads)) == cudaSuccess ? 0 : -1;
  };
  auto of_dim = [&](auto D) {
    constexpr int d = decltype(D)::value, tokens = KvTile<d, 4>::TOKENS;
    const std::true_type e{};
    const std::false_type b{};
    const std::integral_constant<int, 1> one{};
    const std::integral_constant<int, 4> four{};
    const bool many = static_cast<long long>((n + tokens - 1) / tokens) * 2 * c.heads >= 2LL * sm_count();
    if (c.format == K3MOE_KV_E4M3) return many ? with(D, e, four) : with(D, e, one);
    return many ? with(D, b, four) : with(D, b, one);
  };
  if (c.dim == 64) return of_dim(std::integral_constant<int, 64>());
  if (c.dim == 128) return of_dim(std::integral_constant<int, 128>());
  if (c.dim == 256) return of_dim(std::integral_constant<int, 256>());
  return -1;
}

}  // namespace

int launch_kv_write(const k3moe_kv_cache &c, int n, const uint16_t *k, const uint16_t *v, long long k_stride,
                    long long v_stride, const int32_t *slots, int32_t *status, cudaStream_t st) {
  return kv_dispatch(c, n, [&](auto D, auto E, auto U, dim3 grid) {
    return launch_pdl(kv_write_kernel<decltype(D)::value, decltype(E)::value, decltype(U)::value>, grid, dim3(256), 0, st,
                      view_of(c), n, k, v, k_stride, v_stride, slots, status);
  });
}

int launch_kv_read(const k3moe_kv_cache &c, int n, const int32_t *slots, uint16_t *k_out, uint16_t *v_out,
                   int32_t *status, cudaStream_t st) {
  return kv_dispatch(c, n, [&](auto D, auto E, auto U, dim3 grid) {
    return launch_pdl(kv_read_kernel<decltype(D)::value, decltype(E)::value, decltype(U)::value>, grid, dim3(256), 0, st,
                      view_of(c), n, slots, k_out, v_out, status);
  });
}

}  // namespace k3moe
