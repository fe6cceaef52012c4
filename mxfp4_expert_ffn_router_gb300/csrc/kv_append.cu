// kv_append.cu -- new tokens' keys and values into the slots of a paged cache with the rotation
// of their positions on the way, and the rotated queries.
//
// Pair i of a head's rotated dimensions turns by a = position * inv_freq[i]:
//   (x, y) -> scale * (x cos a - y sin a, y cos a + x sin a)
// in fp32; q is then rounded to bf16 once, and the key quantised (or rounded) once.
//
// The angle is held in turns of 2^-64: position * turns[i] in 64-bit whole numbers wraps
// where the angle does, so nothing is lost however far the position (a fp32 product is off by a
// whole turn's tenth at position 10^6).  What is left, a number in [-1/2, 1/2) turns, goes
// to fp32 with all its leading bits, and to sincospif.
//
// Eight dimensions of a pair's first half and eight of its second (or 2 x 8 neighbours) are one
// lane's, so dim / 16 lanes hold a vector and no value is exchanged but the scale's maximum.
//
// Bound by memory where there are many tokens, and by launch and two trips to it where there are few.  A block takes four
// tokens (one where that leaves SMs idle), whose sines and cosines its threads compute once for all heads; a lane has two vectors' loads
// under way (one: 39.1 us).  Measured: 4096 tokens, 64 query and 8 key-value heads of 128, E4M3 (159 MB) 36.2 us, 4.4
// TB/s, 0.65 of a copy's rate: issue 49 %, 63 registers, the rest waits for the loads of a block's one or two turns; bf16 (168 MB)
// 33.8 us, 5.0 TB/s; 777 tokens of 15 / 5 heads of 64, bf16, 3.3 us; 13 tokens of 96 / 96 heads 3 us (bf16 2.5).
#include <type_traits>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"

namespace k3moe {

namespace {

struct ApParams {
  uint8_t *k, *v, *ks, *vs;
  int heads, page_shift, places;
  int n, Hq;
  const uint16_t *q_in, *k_in, *v_in;
  long long q_stride, k_stride, v_stride;
  const int32_t *slots, *positions;
  const int64_t *turns;
  int pairs, neighbours;  // pairs = rotated dimensions / 2
  float scale;
  uint16_t *q_out;
  long long q_out_stride;
  int vectors;  // of a token that a block takes (the last block of a token: what is left)
  int32_t *status;
};

constexpr int kApThreads = 256;

}  // namespace

// Block (x, y): TOKENS tokens from x TOKENS on, and of each the vectors (queries, keys, values in
// this order) from y * vectors on.
template <int D, bool E4M3, int TOKENS>
__global__ void __launch_bounds__(kApThreads) kv_append_kernel(const ApParams P) {
  constexpr int L = D / 16, G = kApThreads / L;
  __shared__ __align__(16) float2 s_cs[TOKENS][D / 2];  // {cos, sin} of the pairs
  __shared__ int s_slot[TOKENS];
  const int tid = threadIdx.x, t0 = blockIdx.x * TOKENS;
  pdl_wait();
  pdl_trigger();
  if (tid < TOKENS) {
    const int t = t0 + tid;
    int slot = t < P.n ? P.slots[t] : -1;
    if (slot >= P.places) {
      if (blockIdx.y == 0) set_status(P.status, K3MOE_DEV_BOUNDS);
      slot = -1;
    }
    s_slot[tid] = slot;
  }
  for (int i = tid; i < TOKENS * P.pairs; i += kApThreads) {
    const int tt = i / P.pairs, pair = i - tt * P.pairs, t = t0 + tt;
    if (t >= P.n) break;
    // the angle modulo a turn, in units of 2^-64; then in units of pi
    const long long a = static_cast<long long>(static_cast<unsigned long long>(P.turns[pair]) *
                                               static_cast<unsigned long long>(static_cast<long long>(P.positions[t])));
    float sn, cs;
    sincospif(__ll2float_rn(a) * 0x1p-63f, &sn, &cs);
    s_cs[tt][pair] = make_float2(cs * P.scale, sn * P.scale);
  }
  __syncthreads();
  const int sub = tid % L, all = P.Hq + 2 * P.heads;
  const int v0 = blockIdx.y * P.vectors, nv = min(P.vectors, all - v0);
  // this lane's two runs of eight dimensions; rotated ones are a pair's two halves
  const int half = P.pairs / 8;  // words of a half
  const bool turn = sub < half;
  const int wa = turn && !P.neighbours ? sub : 2 * sub, wb = turn && !P.neighbours ? sub + half : 2 * sub + 1;
  // (a group's lanes stay together: all of a vector's, or none.)  Two vectors a turn, loaded before the first is used
  constexpr int U = 2;
  for (int base = 0; base < TOKENS * nv; base += U * G) {
    uint4 in[U][2];
    int slot[U], tt[U], vec[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int it = base + x * G + tid / L;
      tt[x] = it / nv, vec[x] = v0 + it - tt[x] * nv;
      slot[x] = it < TOKENS * nv ? s_slot[tt[x]] : -1;
      in[x][0] = in[x][1] = make_uint4(0, 0, 0, 0);
      if (slot[x] >= 0) {
        const int t = t0 + tt[x], k = vec[x] - P.Hq, v = k - P.heads;  // (k, v: of keys, of values)
        const uint16_t *src = k < 0 ? P.q_in + t * P.q_stride + static_cast<size_t>(vec[x]) * D
                              : v < 0 ? P.k_in + t * P.k_stride + static_cast<size_t>(k) * D
                                      : P.v_in + t * P.v_stride + static_cast<size_t>(v) * D;
        in[x][0] = reinterpret_cast<const uint4 *>(src)[wa], in[x][1] = reinterpret_cast<const uint4 *>(src)[wb];
      }
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const bool on = slot[x] >= 0, is_q = vec[x] < P.Hq, is_v = vec[x] >= P.Hq + P.heads;
      const int t = t0 + tt[x], head = is_q ? vec[x] : is_v ? vec[x] - P.Hq - P.heads : vec[x] - P.Hq;
      const uint32_t w[8] = {in[x][0].x, in[x][0].y, in[x][0].z, in[x][0].w, in[x][1].x, in[x][1].y, in[x][1].z, in[x][1].w};
      float f[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
      if (on && turn && !is_v) {
        const float4 *cs = reinterpret_cast<const float4 *>(&s_cs[tt[x]][8 * sub]);
        if (P.neighbours) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 c = cs[i];
            const float a = f[4 * i], y = f[4 * i + 1], z = f[4 * i + 2], u = f[4 * i + 3];
            f[4 * i] = a * c.x - y * c.y, f[4 * i + 1] = y * c.x + a * c.y;
            f[4 * i + 2] = z * c.z - u * c.w, f[4 * i + 3] = u * c.z + z * c.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 c = cs[i];
            const float a = f[2 * i], y = f[2 * i + 8], z = f[2 * i + 1], u = f[2 * i + 9];
            f[2 * i] = a * c.x - y * c.y, f[2 * i + 8] = y * c.x + a * c.y;
            f[2 * i + 1] = z * c.z - u * c.w, f[2 * i + 9] = u * c.z + z * c.w;
          }
        }
      }
      uint32_t byte = 0;
      if constexpr (E4M3) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int off = 1; off < L; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        byte = mx8_scale_byte(m);
      }
      if (!on) continue;
      const size_t at = ((static_cast<size_t>(slot[x] >> P.page_shift) * P.heads + head) << P.page_shift) +
                        (slot[x] & ((1 << P.page_shift) - 1));
      if (E4M3 && !is_q) {
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = f[i], hi[i] = f[8 + i];
        uint2 *dst = reinterpret_cast<uint2 *>((is_v ? P.v : P.k) + at * D);
        dst[wa] = mx8_codes(lo, byte);
        dst[wb] = mx8_codes(hi, byte);
        if (sub == 0) (is_v ? P.vs : P.ks)[at] = static_cast<uint8_t>(byte);
      } else {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = bf16x2(f[2 * i], f[2 * i + 1]);
        uint4 *dst = is_q ? reinterpret_cast<uint4 *>(P.q_out + t * P.q_out_stride + static_cast<size_t>(head) * D)
                          : reinterpret_cast<uint4 *>((is_v ? P.v : P.k) + at * (2 * D));
        dst[wa] = make_uint4(r[0], r[1], r[2], r[3]);
        dst[wb] = make_uint4(r[4], r[5], r[6], r[7]);
      }
    }
  }
}

int launch_kv_append(const k3moe_kv_cache &c, int n, int Hq, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                     long long q_stride, long long k_stride, long long v_stride, const int32_t *slots,
                     const int32_t *positions, const k3moe_rotation &rot, uint16_t *q_out, long long q_out_stride,
                     int32_t *status, cudaStream_t st) {
  ApParams P;
  P.k = static_cast<uint8_t *>(c.k), P.v = static_cast<uint8_t *>(c.v), P.ks = c.k_scales, P.vs = c.v_scales;
  P.heads = c.heads, P.page_shift = 0, P.places = c.pages * c.page_size;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  P.n = n, P.Hq = Hq, P.q_in = q, P.k_in = k, P.v_in = v;
  P.q_stride = q_stride, P.k_stride = k_stride, P.v_stride = v_stride;
  P.slots = slots, P.positions = positions, P.turns = rot.turns, P.pairs = rot.dim / 2, P.neighbours = rot.neighbours;
  P.scale = rot.scale, P.q_out = q_out, P.q_out_stride = q_out_stride, P.status = status;
  const int all = Hq + 2 * c.heads;
  auto of = [&](auto D, auto E) {
    constexpr int G = kApThreads / (decltype(D)::value / 16);
    auto with = [&](auto T) {
      const int blocks = (n + T - 1) / T;
      // as many blocks as two an SM want, in whole rounds of a block's groups
      const int want = max(1, min((2 * sm_count() + blocks - 1) / blocks, (all * T + G - 1) / G));
      P.vectors = (all + want - 1) / want;
      const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((all + P.vectors - 1) / P.vectors));
      return launch_pdl(kv_append_kernel<decltype(D)::value, decltype(E)::value, decltype(T)::value>, grid,
                        dim3(kApThreads), 0, st, P) == cudaSuccess
                 ? 0
                 : -1;
    };
    return n >= 4 * sm_count() ? with(std::integral_constant<int, 4>()) : with(std::integral_constant<int, 1>());
  };
  auto of_dim = [&](auto D) {
    return c.format == K3MOE_KV_E4M3 ? of(D, std::true_type()) : of(D, std::false_type());
  };
  if (c.dim == 64) return of_dim(std::integral_constant<int, 64>());
  if (c.dim == 128) return of_dim(std::integral_constant<int, 128>());
  if (c.dim == 256) return of_dim(std::integral_constant<int, 256>());
  return -1;
}

}  // namespace k3moe
