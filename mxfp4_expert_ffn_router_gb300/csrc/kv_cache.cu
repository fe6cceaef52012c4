// kv_cache.cu -- the paged key-value cache: new tokens' keys and values written into
// their slots (quantised on the way, mx8_quant.cuh), and slots read back as bf16.
//
// A cache holds [pages][heads][page_size][dim] values, so that one head's tokens of a
// page are contiguous: that is what attention streams.  A slot is page * page_size +
// place.  A negative slot is padding (not written; reads as zeros); one at or past the
// end sets K3MOE_DEV_BOUNDS and is treated the same.
//
// A few neighbouring lanes hold one vector (a token's key or value of one head), 8 or 16 values
// each; its scale needs one maximum over those lanes.
//
// Inputs are read by ordinary loads: a kernel before this one, still running when this one starts, may
// have written them.
//
// Bound: the bytes, once in and once out, with several tokens in flight a thread where there are
// enough of them: reading 16384 tokens of 8 heads of 128 (101 MB) 17.4 us, 5.8 TB/s (one in flight 22.2
// us); writing 4096 tokens (25 MB) 4.5 us, of which about 2 are the launch; 13 tokens of 96 heads 1.9 us.
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
// cache.  A group of L lanes takes every (256 / L)th of the block's tokens, U in all, loading
// all of them before the first use.
template <int D, int V_, int U_>
struct KvTile {
  static constexpr int V = V_;  // values of a lane
  static constexpr int L = D / V, G = 256 / L, U = U_, TOKENS = G * U;
};
// Values of a lane and tokens in flight (1 where fewer than two blocks an SM would be left).  Quantising
// shares a maximum, so fewer lanes with 16 values each pay (4.5 against 5.5 us for 4096 tokens); reading back
// 16 a lane would store two words 32 bytes apart at a time (20.2 against 17.4 us for 16384 tokens).
template <bool E4M3>
struct KvWriteWork {
  static constexpr int V = E4M3 ? 16 : 8, MANY = 2;
};
template <bool E4M3>
struct KvReadWork {
  static constexpr int V = 8, MANY = 4;
};

template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256)
    kv_write_kernel(KvView c, int n, const uint16_t *k, const uint16_t *v, long long k_stride,
                    long long v_stride, const int32_t *slots, int32_t *status) {
  using K = KvTile<D, KvWriteWork<E4M3>::V, U>;
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % K::L;
  const bool val = static_cast<int>(blockIdx.y) >= c.heads;
  const int head = val ? blockIdx.y - c.heads : blockIdx.y;
  const uint16_t *src = (val ? v : k) + static_cast<size_t>(head) * D + sub * K::V;
  const long long stride = val ? v_stride : k_stride;
  uint8_t *dst = val ? c.v : c.k, *dst_scales = val ? c.vs : c.ks;
  const int t0 = blockIdx.x * K::TOKENS + threadIdx.x / K::L;
  int slot[K::U];
  uint4 u[K::U][K::V / 8];
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    const int t = t0 + i * K::G;
    slot[i] = t < n ? slots[t] : -1;
#pragma unroll
    for (int h = 0; h < K::V / 8; ++h) {
      u[i][h] = make_uint4(0, 0, 0, 0);
      if (t < n) u[i][h] = *(reinterpret_cast<const uint4 *>(src + t * stride) + h);
    }
  }
#pragma unroll
  for (int i = 0; i < K::U; ++i) {
    if (slot[i] >= c.places) {
      if (blockIdx.y == 0 && sub == 0) set_status(status, K3MOE_DEV_BOUNDS);
      slot[i] = -1;
    }
    const size_t o = slot[i] >= 0 ? vec_index(c, slot[i], head) : 0;
    if constexpr (!E4M3) {
      if (slot[i] >= 0) *(reinterpret_cast<uint4 *>(dst + o * (2 * D)) + sub) = u[i][0];
    } else {
      // the largest magnitude as a bf16 pattern: two at a time
      uint32_t m2 = 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(u[i][h].x & 0x7FFF7FFFu, u[i][h].y & 0x7FFF7FFFu)),
                      __vmaxu2(u[i][h].z & 0x7FFF7FFFu, u[i][h].w & 0x7FFF7FFFu));
      uint32_t m = max(m2 << 16, m2 & 0xFFFF0000u);
#pragma unroll
      for (int off = 1; off < K::L; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const uint32_t byte = mx8_scale_byte(m);
      uint2 q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {u[i][h].x, u[i][h].y, u[i][h].z, u[i][h].w};
        float f[8];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          f[2 * x] = __uint_as_float(w[x] << 16);
          f[2 * x + 1] = __uint_as_float(w[x] & 0xFFFF0000u);
        }
        q[h] = mx8_codes(f, byte);
      }
      if (slot[i] >= 0) {
        *(reinterpret_cast<uint4 *>(dst + o * D) + sub) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
        if (sub == 0) dst_scales[o] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// k_out, v_out: bf16 [n][heads][D].
template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvView c, int n, const int32_t *slots, uint16_t *k_out,
                   uint16_t *v_out, int32_t *status) {
  using K = KvTile<D, KvReadWork<E4M3>::V, U>;
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
    slot[i] = t < n ? slots[t] : -1;
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
    uint4 *to = reinterpret_cast<uint4 *>(out + static_cast<size_t>(t) * c.heads * D + sub * K::V);
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
      *to = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      *to = w[i];
    }
  }
}

namespace {

// Calls f(dim, whether E4M3, U, grid), the first three as types' values.
template <template <bool> class Work, class F>
int kv_dispatch(const k3moe_kv_cache &c, int n, F f) {
  auto of_format = [&](auto D, auto E) {
    using Wk = Work<decltype(E)::value>;
    auto with = [&](auto U) {
      constexpr int tokens = KvTile<decltype(D)::value, Wk::V, decltype(U)::value>::TOKENS;
      const long long blocks = (static_cast<long long>(n) + tokens - 1) / tokens;
      if (U > 1 && blocks * 2 * c.heads < 2LL * sm_count()) return 1;  // too few
      return f(D, E, U, dim3(static_cast<unsigned>(blocks), 2 * c.heads)) == cudaSuccess ? 0 : -1;
    };
    const int rc = with(std::integral_constant<int, Wk::MANY>());
    return rc == 1 ? with(std::integral_constant<int, 1>()) : rc;
  };
  auto of_dim = [&](auto D) {
    return c.format == K3MOE_KV_E4M3 ? of_format(D, std::true_type()) : of_format(D, std::false_type());
  };
  if (c.dim == 64) return of_dim(std::integral_constant<int, 64>());
  if (c.dim == 128) return of_dim(std::integral_constant<int, 128>());
  if (c.dim == 256) return of_dim(std::integral_constant<int, 256>());
  return -1;
}

}  // namespace

int launch_kv_write(const k3moe_kv_cache &c, int n, const uint16_t *k, const uint16_t *v, long long k_stride,
                    long long v_stride, const int32_t *slots, int32_t *status, cudaStream_t st) {
  return kv_dispatch<KvWriteWork>(c, n, [&](auto D, auto E, auto U, dim3 grid) {
    return launch_pdl(kv_write_kernel<decltype(D)::value, decltype(E)::value, decltype(U)::value>, grid, dim3(256), 0, st,
                      view_of(c), n, k, v, k_stride, v_stride, slots, status);
  });
}

int launch_kv_read(const k3moe_kv_cache &c, int n, const int32_t *slots, uint16_t *k_out, uint16_t *v_out,
                   int32_t *status, cudaStream_t st) {
  return kv_dispatch<KvReadWork>(c, n, [&](auto D, auto E, auto U, dim3 grid) {
    return launch_pdl(kv_read_kernel<decltype(D)::value, decltype(E)::value, decltype(U)::value>, grid, dim3(256), 0, st,
                      view_of(c), n, slots, k_out, v_out, status);
  });
}

}  // namespace k3moe
