// rmsnorm.cu -- root-mean-square norm of rows, with the residual's addition before
// it and an 8-bit output beside or instead of the bf16 one.
//
//   a[t] = x[t] + residual[t]                          (fp32, exact sum rounded once)
//   y[t] = a[t] * rsqrt(mean(a[t]^2) + eps) * weight   (fp32)
//   residual_out = bf16(a),  y = bf16(y),  codes / scales = y per 32 values (mx8_quant.cuh)
//
// The norm is of the fp32 sum, not of the bf16 value that residual_out keeps: the sum is
// in registers anyway, and rounding it first would only lose bits.  The mean is a fixed
// tree: a thread's values in order, a butterfly over the warp, a tree over the warps.
//
// Bound: the rows' bytes, 9 of them a value with every output.  A block has one row in registers,
// read once; four blocks an SM (32 registers a thread, many rows) overlap one row's reduction with the others'
// loads: 4096 rows of 7168 with both outputs (265 MB) 42.1 us, 6.3 TB/s of 6.8 measured for a copy,
// against 46.2 us at 38 registers (three blocks) and 48 us for a persistent block that loads its next
// row early.  All arrays are indexed by chunks of 8 values from one index, with an index for each at
// 32 registers 16 bytes spill: 43.4 us (4096 rows of 4096 28.5, now 25.2).  One row: 2.3 us, the launch and two trips to memory.
#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"

namespace k3moe {

namespace {

__device__ __forceinline__ void bf16x8_to_f32(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    v[2 * m] = __uint_as_float(w[m] << 16);
    v[2 * m + 1] = __uint_as_float(w[m] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32x8_to_bf16(const float (&v)[8]) {
  return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

constexpr int kWarpRows = 8;  // rows of a block where a warp takes one

}  // namespace

// One block per row, or (WARP) one warp: a thread holds CH chunks of 8 values, tid + i * nth of its row.
// FEW: at most 4 / CH rows an SM.
template <int CH, bool WARP, bool FEW>
__global__ void __launch_bounds__(512, FEW ? 1 : CH <= 2 ? 4 : 2)
    rmsnorm_kernel(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps, int T,
                   int H, uint16_t *residual_out, uint16_t *y, uint8_t *codes, uint8_t *scales) {
  __shared__ __align__(16) float part[16];
  pdl_wait();
  pdl_trigger();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nth = WARP ? 32 : blockDim.x, nch = H / 8;
  const long long r_at = WARP ? static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && r_at >= T) return;
  const size_t row = static_cast<size_t>(r_at) * nch;  // chunks
  float a[CH][8];
  float sum = 0.f;
  // Few rows: the weights are loaded beside x, at 37 to 76 registers a thread (37 rows of 7168, all outputs, 2.6 us
  // against 3.1, 300 3.6 against 5.0, but 600 9.3 against 8.7).  Many: only brought near (4096 rows of 16384 108.1 us,
  // 110.1 without)
  constexpr bool kEarly = FEW || WARP;
  uint4 wr[kEarly ? CH : 1];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nth;
    if (c < nch) {
      const uint4 *const wp = reinterpret_cast<const uint4 *>(weight) + c;
      if constexpr (kEarly)
        wr[i] = *wp;
      else
        asm volatile("prefetch.global.L1 [%0];" ::"l"(wp));
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nth;
    if (c < nch) {
      bf16x8_to_f32(reinterpret_cast<const uint4 *>(x)[row + c], a[i]);
      if (residual) {
        float r[8];
        bf16x8_to_f32(reinterpret_cast<const uint4 *>(residual)[row + c], r);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[i][q] += r[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum = fmaf(a[i][q], a[i][q], sum);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  float total = sum;
  if constexpr (!WARP) {
    if (tid < 16 && tid >= nth / 32) part[tid] = 0.f;
    if ((tid & 31) == 0) part[tid >> 5] = sum;
    __syncthreads();
    float4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = reinterpret_cast<const float4 *>(part)[i];
    total = (((s[0].x + s[0].y) + (s[0].z + s[0].w)) + ((s[1].x + s[1].y) + (s[1].z + s[1].w))) +
            (((s[2].x + s[2].y) + (s[2].z + s[2].w)) + ((s[3].x + s[3].y) + (s[3].z + s[3].w)));
  }
  // m^-1/2 with one Newton step on rsqrtf, 1 - m inv^2 taken from exact products
  const float m = total / static_cast<float>(H) + eps;
  float inv = rsqrtf(m);
  if (m > 0.f && m < INFINITY) {
    const float p = m * inv, r = fmaf(-p, inv, 1.f) - fmaf(m, inv, -p) * inv;
    inv = fmaf(0.5f * inv, r, inv);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nth;
    // the four lanes of a 32-value group are in or out together (H % 32 == 0)
    const unsigned in = __ballot_sync(0xFFFFFFFFu, c < nch);
    if (c < nch) {
      if (residual_out) reinterpret_cast<uint4 *>(residual_out)[row + c] = f32x8_to_bf16(a[i]);
      float w[8];
      if constexpr (kEarly)
        bf16x8_to_f32(wr[i], w);
      else
        bf16x8_to_f32(*(reinterpret_cast<const uint4 *>(weight) + c), w);
#pragma unroll
      for (int q = 0; q < 8; ++q) a[i][q] = a[i][q] * inv * w[q];
      if (y) reinterpret_cast<uint4 *>(y)[row + c] = f32x8_to_bf16(a[i]);
      if (codes) {
        uint32_t m = 0u;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(a[i][q]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(in, m, 1));
        m = max(m, __shfl_xor_sync(in, m, 2));
        const uint32_t byte = mx8_scale_byte(m);
        reinterpret_cast<uint2 *>(codes)[row + c] = mx8_codes(a[i], byte);
        if ((c & 3) == 0) scales[(row + c) >> 2] = static_cast<uint8_t>(byte);
      }
    }
  }
}

int launch_rmsnorm(int T, int H, const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps,
                   uint16_t *residual_out, uint16_t *y, uint8_t *codes, uint8_t *scales, cudaStream_t st) {
  const int nch = H / 8;  // at most 2048
  cudaError_t err;
#define K3_RN(CH_, WARP_, FEW_, GRID_, BLOCK_)                                                                             \
  err = launch_pdl(rmsnorm_kernel<CH_, WARP_, FEW_>, dim3(GRID_), dim3(BLOCK_), 0, st, x, residual, weight, eps, T, H, \
                   residual_out, y, codes, scales)
#define K3_RN_ROW(CH_)                                        \
  if (T <= 4 / CH_ * sm_count())                              \
    K3_RN(CH_, false, true, T, ((nch + CH_ - 1) / CH_ + 31) / 32 * 32); \
  else                                                        \
    K3_RN(CH_, false, false, T, ((nch + CH_ - 1) / CH_ + 31) / 32 * 32)
  if (nch <= 32) {  // a row is one chunk a lane: 4096 rows of 256 2.5 us, one block each 4.8
    K3_RN(1, true, false, (static_cast<unsigned>(T) + kWarpRows - 1) / kWarpRows, 32 * kWarpRows);
  } else if (nch <= 512) {
    K3_RN_ROW(1);
  } else if (nch <= 1024) {
    K3_RN_ROW(2);
  } else {
    K3_RN_ROW(4);
  }
#undef K3_RN_ROW
#undef K3_RN
  return err == cudaSuccess ? 0 : -1;
}

}  // namespace k3moe
