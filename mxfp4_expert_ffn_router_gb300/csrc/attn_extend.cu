// attn_extend.cu -- attention of several new tokens per sequence over a paged key-value cache.
#include <cuda_fp16.h>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"

namespace k3moe {

namespace {

struct AxParams {
  const uint8_t *k, *v, *ks, *vs;
  int heads, pages, page_shift;
  int B, rows, Hq, G;
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
  int32_t *status;
};

struct Seq {
  int n, first, m, ctx;  // cached tokens, first row, new tokens, places before them (may be negative)
};

__device__ __forceinline__ Seq seq_of(const AxParams &P, int b, bool report) {
  Seq s;
  const long long most = static_cast<long long>(P.max_pages) << P.page_shift;
  const int len = P.lens[b], o0 = P.offsets[b], o1 = P.offsets[b + 1];
  bool bad = len < 0 || len > most;
  s.n = len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
  s.first = o0;
  s.m = 0;
  if (o0 < 0 || o1 < o0 || o1 > P.rows || o1 - o0 > P.max_new)
    bad = true;
  else
    s.m = o1 - o0;
  s.ctx = s.n - s.m;
  if (s.m > s.n) bad = true;
  if (bad && report) set_status(P.status, K3MOE_DEV_BOUNDS);
  return s;
}

}  // namespace

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) attn_extend_simple(const AxParams P) {
  const int b = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const Seq s = seq_of(P, b, h == 0 && blockIdx.z == 0 && threadIdx.x == 0);
  const int g = h / P.G;
  for (int i = blockIdx.z * 8 + warp; i < s.m; i += 8 * gridDim.z) {
    const size_t row = s.first + i;
    const uint16_t *q = P.q + static_cast<long long>(row) * P.q_stride + static_cast<size_t>(h) * D;
    float qv[D / 32], o[D / 32], m = -INFINITY, l = 0.f;
    for (int x = 0; x < D / 32; ++x) qv[x] = bf16_bits_to_f32(q[x * 32 + lane]), o[x] = 0.f;
    int pos = s.ctx + i;
    if (P.masks) {
      int seen = 0;
      for (int j = 0; j < s.m; ++j) seen += (P.masks[row * P.words + j / 64] >> (j % 64)) & 1;
      pos = s.ctx + max(0, seen - 1);
    }
    for (int c = 0; c < s.n; ++c) {
      bool see;
      if (P.masks && c >= s.ctx) {
        const int j = c - s.ctx;
        see = (P.masks[row * P.words + j / 64] >> (j % 64)) & 1;
      } else {
        see = (P.masks || c <= pos) && (P.window == 0 || c > static_cast<long long>(pos) - P.window || c < P.sinks);
      }
      if (!see) continue;
      const int page = P.table[static_cast<size_t>(b) * P.max_pages + (c >> P.page_shift)];
      if (page < 0 || page >= P.pages) {
        if (lane == 0) set_status(P.status, K3MOE_DEV_BOUNDS);
        continue;
      }
      const size_t vec = ((static_cast<size_t>(page) * P.heads + g) << P.page_shift) + (c & ((1 << P.page_shift) - 1));
      float kv[D / 32], vv[D / 32], dot = 0.f;
      for (int x = 0; x < D / 32; ++x) {
        if (E4M3) {
          uint32_t a, z;
          e4m3x4_to_f16x2(P.k[vec * D + x * 32 + lane], a, z);
          kv[x] = __half2float(__ushort_as_half(a & 0xFFFF)) * e8m0_to_f32(P.ks[vec]);
          e4m3x4_to_f16x2(P.v[vec * D + x * 32 + lane], a, z);
          vv[x] = __half2float(__ushort_as_half(a & 0xFFFF)) * e8m0_to_f32(P.vs[vec]);
        } else {
          kv[x] = bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(P.k)[vec * D + x * 32 + lane]);
          vv[x] = bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(P.v)[vec * D + x * 32 + lane]);
        }
        dot += qv[x] * kv[x];
      }
      for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
      const float sc = dot * P.scale, mn = fmaxf(m, sc), base = mn == -INFINITY ? 0.f : mn;
      const float f = __expf(m - base), p = expf(sc - base);
      l = l * f + p;
      for (int x = 0; x < D / 32; ++x) o[x] = o[x] * f + p * vv[x];
      m = mn;
    }
    for (int x = 0; x < D / 32; ++x)
      P.out[(row * P.Hq + h) * D + x * 32 + lane] = l == 0.f ? 0 : f32_to_bf16_rne(o[x] / l);
    if (P.lse && lane == 0) P.lse[row * P.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
  }
}

size_t attn_extend_workspace(const k3moe_kv_cache &, int, int, int) { return 0; }

int launch_attn_extend(const ExtendArgs &a, cudaStream_t st) {
  AxParams P;
  const k3moe_kv_cache &c = a.c;
  P.k = static_cast<const uint8_t *>(c.k), P.v = static_cast<const uint8_t *>(c.v), P.ks = c.k_scales, P.vs = c.v_scales;
  P.heads = c.heads, P.pages = c.pages, P.page_shift = 0;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  P.B = a.B, P.rows = a.rows, P.Hq = a.Hq, P.G = a.Hq / c.heads;
  P.q = a.q, P.q_stride = a.q_stride, P.offsets = a.offsets, P.max_new = a.max_new, P.masks = a.masks, P.words = a.words;
  P.table = a.table, P.max_pages = a.max_pages, P.lens = a.lens, P.window = a.window, P.sinks = a.sinks;
  P.scale = a.scale, P.out = a.out, P.lse = a.lse, P.status = a.status;
  const dim3 grid(a.B, a.Hq, a.max_new > 64 ? 32 : 1);
  const bool e = c.format == K3MOE_KV_E4M3;
#define K3_AX(D_)                                                                                              \
  if (c.dim == D_)                                                                                             \
    return launch_pdl(e ? attn_extend_simple<D_, true> : attn_extend_simple<D_, false>, grid, dim3(256), 0, st, P) == \
                   cudaSuccess ? 0 : -1;
  K3_AX(64) K3_AX(128) K3_AX(256)
#undef K3_AX
  return -1;
}

}  // namespace k3moe
