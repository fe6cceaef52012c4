// attn_decode.cu -- attention of one new token per sequence over a paged key-value cache.
//
// For sequence b with n = seq_lens[b] cached tokens, of which those at places
// lo = max(0, n - window) (0 without a window) .. n - 1 are seen, and query head h
// of key-value head g = h / (Hq / heads):
//   s_i = scale * q . K_i,  m = max s_i,  l = sum exp(s_i - m),
//   out = sum exp(s_i - m) V_i / l,  lse = m + log l
// A row that sees nothing (or only scores of -inf) gives out = 0 and lse = -inf.
//
// Bound: the cache is read once (2 dim bytes a token and head in E4M3) and each byte meets
// only the 1 to 16 query heads that share it, so the time is the cache's bytes over the
// HBM rate.  All the rest serves to keep those loads in flight.
//
//  * Work.  An item is (sequence, key-value head, up to 8 NT of the query heads that
//    share it); a unit is 64 of its tokens.  All items' units form one line, cut into
//    equal pieces, one per block: blocks end together however uneven the lengths are,
//    and one long sequence fills the GPU.  Lengths are read on the device, so a captured
//    graph follows them.  A piece covers the end of one item, some whole items and the
//    start of another; only the cut ones leave partial sums in the workspace, at
//    most two a block, which attn_join_kernel adds in order.  When every item
//    is short (kDirectUnits), a block takes one item and nothing is cut or joined.
//  * Loads.  Each of the four warps streams every fourth run of 16 tokens through a ring
//    of its own in shared memory with 16-byte cp.async (stages - 1 runs ahead, across items),
//    so no warp waits for another except where an item ends.  Runs never straddle a page
//    (pages hold a multiple of 16 places); the next run's page number is loaded a step
//    ahead.  Places not seen are filled with zeros by the copy, so that nothing they hold
//    (NaN, infinities) reaches a product.
//  * Products.  mma.sync m16n8k16 (f16 or bf16, fp32 sums): with at most 16 query heads
//    sharing a key the products are a small part of the time even at this instruction's
//    rate, and its operands come straight from registers, where E4M3 codes are converted.
//    S = Q K^T has the query heads as rows; O^T = V^T P^T has dimensions as rows
//    and 8 query heads as columns, so that S's registers are P^T's.  The order of
//    dimensions and tokens inside a product is free as long as both operands agree, and
//    is chosen so that a lane's share of K and V is whole 16-byte words.
//  * E4M3 (f16 products).  Codes are exact in f16; a query row is scaled by a power of two
//    to a maximum in [2^14, 2^15), exact but for values below 2^-28 of it.  K's scale
//    multiplies the score.  V's scale 2^e joins the weight: w_i = exp2(s_i + e_i - m')
//    with its own running maximum m' of s_i + e_i, times 2^14, rounded to f16 (11 bits
//    down to 2^-28 of the largest, so that a token with a large score and a tiny value
//    costs the others nothing), while l sums exp2(s_i - m) in fp32 with m = max s_i.
//  * bf16.  Q, K and V enter as they are; the weights are rounded to bf16, as V is.
#include <cuda_fp16.h>

#include "k3moe_dev.cuh"
#include "k3moe_launch.h"
#include "mx8_quant.cuh"
#include "tc_sm103.cuh"

namespace k3moe {

namespace {

constexpr int kAdWarps = 4;
constexpr int kAdThreads = kAdWarps * 32;
constexpr int kRun = 16;                 // tokens of a warp's step
constexpr int kUnit = kRun * kAdWarps;   // tokens of a block's step
constexpr int kDirectUnits = 8;          // items of at most this many units are never cut
constexpr int kMinUnits = 4;             // smallest piece of a block, in units
constexpr int kAdMostBlocks = 152 * 4;   // pieces (bounds the workspace and the join)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// d += a b, m16n8k16, f16 (H) or bf16 operands.
template <bool H>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (H)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool H>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (H)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale byte -> exponent as a float (NaN for 255).
__device__ __forceinline__ float e8m0_exp(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(0x4B000000u | b) - 8388735.0f;
}

struct AdParams {
  const uint8_t *k, *v, *ks, *vs;
  int heads, pages, page_shift;
  int B, Hq, G, groups;  // G query heads per key-value head, in `groups` items
  const uint16_t *q;
  long long q_stride;
  const int32_t *table;
  int max_pages;
  const int32_t *lens;
  int window;
  float scale;
  uint16_t *out;
  float *lse;
  int4 *meta;    // [blocks]: {parts, first slot, item's first query head, sequence} of a cut item that starts here
  float4 *stat;  // [2 blocks][8 NT]: {m', m, l, -}
  float4 *part;  // [2 blocks][accumulator quads][32 lanes]
  int32_t *status;
};

// The tokens of one sequence that are seen, and the place its units count from.
struct Seen {
  int n, lo, t0, units;
};
__device__ __forceinline__ Seen seen_of(const AdParams &P, int b, bool report) {
  Seen s;
  const long long most = static_cast<long long>(P.max_pages) << P.page_shift;
  const int len = P.lens[b];
  s.n = len;
  if (len < 0 || len > most) {
    if (report) set_status(P.status, K3MOE_DEV_BOUNDS);
    s.n = len < 0 ? 0 : static_cast<int>(most);
  }
  s.lo = P.window > 0 && s.n > P.window ? s.n - P.window : 0;
  s.t0 = s.lo & ~(kRun - 1);
  s.units = static_cast<int>((static_cast<unsigned>(s.n - s.t0) + (kUnit - 1)) / kUnit);
  return s;
}

// Walks a block's piece of the line of units.
struct Cursor {
  int b, it, u;  // sequence, item of it, unit of that
  Seen s;
  __device__ __forceinline__ void next(const AdParams &P, int items) {
    if (++u < s.units) return;
    u = 0;
    if (++it < items) return;
    it = 0;
    do {
      if (++b >= P.B) {  // past the last unit of all
        s.units = 0;
        return;
      }
      s = seen_of(P, b, false);
    } while (s.units == 0);
  }
};

template <int D, bool E4M3, int NT>
struct AdShape {
  static constexpr int ESZ = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;            // bytes of a cached vector
  static constexpr int C = ROWB / 16;             // 16-byte words of it
  static constexpr int KB = kRun * ROWB;          // bytes of a run's keys
  static constexpr int STAGE = 2 * KB + (E4M3 ? 32 : 0);
  static constexpr int MM = D / 16;               // products (16 dimensions each) of a run and 8 query heads
  static constexpr int QUADS = MM * NT;           // accumulator quads per lane
  // stages and blocks per SM: about 100 KB of loads in flight per SM
  static constexpr int STAGES = ROWB <= 64 ? 4 : 3;
  static constexpr int BLOCKS = ROWB <= 128 ? 3 : ROWB <= 256 ? 2 : 1;
  static constexpr int MERGE = kAdWarps * 4 * 32 * 16;  // four quads of each warp
  static constexpr int SMEM = kAdWarps * STAGES * STAGE + MERGE;
};

}  // namespace

template <int D, bool E4M3, int NT, bool DIRECT>
__global__ void __launch_bounds__(kAdThreads, (AdShape<D, E4M3, NT>::BLOCKS))
    attn_decode_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT>;
  constexpr int C = S::C, MM = S::MM, ST = S::STAGES, NQ = 8 * NT;
  constexpr int KL = C / 4;             // words of a key a lane reads
  constexpr int SP = E4M3 ? 4 : 2;      // products of 16 dimensions per such word
  constexpr int VL = C >= 8 ? C / 8 : 1;  // words of a value a lane reads
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_fac[kAdWarps][NQ], s_m[kAdWarps][NQ], s_l[kAdWarps][NQ];
  __shared__ float s_fin[NQ];
  __shared__ long long s_scan[kAdWarps];
  __shared__ int s_start[4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int items = P.heads * P.groups;
  pdl_wait();
  pdl_trigger();

  // ---- this block's piece
  Cursor cur;
  int steps;
  long long f0 = 0, share = 0;
  if constexpr (DIRECT) {
    cur.b = blockIdx.x / items;
    cur.it = blockIdx.x - cur.b * items;
    cur.u = 0;
    cur.s = seen_of(P, cur.b, tid == 0);
    steps = cur.s.units;
    if (steps == 0) {  // sees nothing
      const int h0 = (cur.it / P.groups) * P.G + (cur.it % P.groups) * NQ;
      const int rows = min(NQ, P.G - (cur.it % P.groups) * NQ);
      const size_t row = static_cast<size_t>(cur.b) * P.Hq + h0;
      for (int i = tid; i < rows * D / 8; i += kAdThreads)
        reinterpret_cast<uint4 *>(P.out + row * D)[i] = make_uint4(0, 0, 0, 0);
      if (P.lse && tid < rows) P.lse[row + tid] = -INFINITY;
      return;
    }
  } else {
    // thread t counts the units of sequences [t per, t per + per); a scan finds the piece
    const int per = (P.B + kAdThreads - 1) / kAdThreads;
    const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += seen_of(P, b, blockIdx.x == 0).units;
    mine *= items;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kAdWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    share = max(static_cast<long long>(kMinUnits), (total + gridDim.x - 1) / gridDim.x);
    f0 = static_cast<long long>(blockIdx.x) * share;
    const long long first = before + incl - mine;  // of this thread's sequences
    steps = static_cast<int>(max(0LL, min(share, total - f0)));
    if (steps > 0 && f0 >= first && f0 < first + mine) {
      long long at = first;
      int b = b0;
      Seen s;
      for (;; ++b) {
        s = seen_of(P, b, false);
        const long long here = static_cast<long long>(s.units) * items;
        if (f0 < at + here) break;
        at += here;
      }
      const long long r = f0 - at;
      s_start[0] = b;
      s_start[1] = static_cast<int>(r / s.units);
      s_start[2] = static_cast<int>(r % s.units);
    }
    if (tid == 0) P.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    // rows that see nothing
    for (int b = blockIdx.x; b < P.B; b += gridDim.x)
      if (seen_of(P, b, false).units == 0) {
        for (size_t i = tid; i < static_cast<size_t>(P.Hq) * D / 8; i += kAdThreads)
          reinterpret_cast<uint4 *>(P.out + static_cast<size_t>(b) * P.Hq * D)[i] = make_uint4(0, 0, 0, 0);
        if (P.lse)
          for (int i = tid; i < P.Hq; i += kAdThreads) P.lse[static_cast<size_t>(b) * P.Hq + i] = -INFINITY;
      }
    __syncthreads();
    if (steps == 0) return;
    cur.b = s_start[0];
    cur.it = s_start[1];
    cur.u = s_start[2];
    cur.s = seen_of(P, cur.b, false);
  }

  // ---- loads: run `warp` of the unit at `pre` into stage st
  const uint32_t ring = su32(smem) + warp * (ST * S::STAGE);
  Cursor pre = cur;
  uint32_t bad = 0;  // stages whose page number lies outside the cache
  int page = -1;
  auto next_page = [&]() {
    const int tok = pre.s.t0 + pre.u * kUnit + warp * kRun;
    page = -1;
    if (pre.s.units && tok < pre.s.n) page = __ldg(P.table + static_cast<size_t>(pre.b) * P.max_pages + (tok >> P.page_shift));
  };
  auto issue = [&](int st) {
    const int tok = pre.s.t0 + pre.u * kUnit + warp * kRun;
    bad &= ~(1u << st);
    if (tok < pre.s.n) {
      if (page < 0 || page >= P.pages) {
        bad |= 1u << st;
        if (lane == 0) set_status(P.status, K3MOE_DEV_BOUNDS);
      } else {
        const size_t vec = ((static_cast<size_t>(page) * P.heads + pre.it / P.groups) << P.page_shift) +
                           (tok & ((1 << P.page_shift) - 1));
        const uint8_t *kp = P.k + vec * S::ROWB, *vp = P.v + vec * S::ROWB;
        const uint32_t dst = ring + st * S::STAGE;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
          const int w = lane + 32 * i, r = w / C, x = w % C;
          const bool on = tok + r >= pre.s.lo && tok + r < pre.s.n;
          cp16(dst + r * S::ROWB + ((C >= 8 ? x ^ (4 * (r & 1)) : x) << 4), kp + w * 16, on);
          cp16(dst + S::KB + r * S::ROWB + ((C >= 8 ? x ^ (2 * ((r >> 2) & 3)) : x) << 4), vp + w * 16, on);
        }
        if (E4M3 && lane < 2) cp16(dst + 2 * S::KB + 16 * lane, (lane ? P.vs : P.ks) + vec, true);
      }
    }
    cp_commit();
    pre.next(P, items);
    next_page();
  };
  next_page();
  int ahead = 0;
  for (; ahead < ST - 1; ++ahead) {
    if (ahead < steps)
      issue(ahead);
    else
      cp_commit();
  }

  uint32_t qf[D / 16][2 * NT];
  float sq[NT];  // scale of a raw score, in powers of two
  float o[NT][MM][4], mrun[NT], m_l[NT], l[NT];
  auto start_item = [&]() {
    const int gi = cur.it % P.groups;
    const int h0 = (cur.it / P.groups) * P.G + gi * NQ, rows = min(NQ, P.G - gi * NQ);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = g + 8 * t;
      const uint16_t *qp = P.q + cur.b * P.q_stride + static_cast<size_t>(h0 + r) * D;
      uint2 raw[D / 16];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < KL; ++i)
#pragma unroll
        for (int w = 0; w < SP; ++w) {
          const int d = (c + 4 * i) * (16 / S::ESZ) + 4 * w;
          const uint2 u = r < rows ? __ldg(reinterpret_cast<const uint2 *>(qp + d)) : make_uint2(0, 0);
          raw[i * SP + w] = u;
          mx = max(mx, max(max((u.x << 16) & 0x7FFFFFFFu, u.x & 0x7FFF0000u),
                           max((u.y << 16) & 0x7FFFFFFFu, u.y & 0x7FFF0000u)));
        }
      float up = 1.f;
      if constexpr (E4M3) {
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        // 2^(14 - floor(log2 max)), as far as fp32 has it
        const int e = mx == 0 ? 0 : max(-126, min(127, 14 + 127 - static_cast<int>(mx >> 23)));
        up = exp2i(e);
        sq[t] = P.scale * kLog2e * mx_pow2(-e);
      } else {
        sq[t] = P.scale * kLog2e;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if constexpr (E4M3) {
          qf[i][t] = pack2<true>(__uint_as_float(raw[i].x << 16) * up, __uint_as_float(raw[i].x & 0xFFFF0000u) * up);
          qf[i][NT + t] = pack2<true>(__uint_as_float(raw[i].y << 16) * up, __uint_as_float(raw[i].y & 0xFFFF0000u) * up);
        } else {
          qf[i][t] = raw[i].x;
          qf[i][NT + t] = raw[i].y;
        }
      }
      mrun[t] = m_l[t] = -INFINITY;
      l[t] = 0.f;
#pragma unroll
      for (int m = 0; m < MM; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][m][x] = 0.f;
    }
  };

  int item_u0 = cur.u;  // first unit of the item in this piece
  bool first_item = true;
  int stage = 0;
  start_item();
  for (int step = 0; step < steps; ++step) {
    __syncwarp();  // every lane is done with the stage that is loaded next
    if (ahead < steps)
      issue(stage == 0 ? ST - 1 : stage - 1);
    else
      cp_commit();
    ++ahead;
    cp_wait<ST - 1>();
    __syncwarp();
    const int tok = cur.s.t0 + cur.u * kUnit + warp * kRun;
    if (tok < cur.s.n && !((bad >> stage) & 1u)) {
      const uint32_t kb = ring + stage * S::STAGE, vb = kb + S::KB;
      // S: columns 2c, 2c+1 of product j are tokens 4c + 2j, 4c + 2j + 1
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int kr = 4 * (g >> 1) + (g & 1);
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int x = c + 4 * i;
        uint4 kw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          kw[j] = lds128(kb + (kr + 2 * j) * S::ROWB + ((C >= 8 ? x ^ (4 * (g & 1)) : x) << 4));
#pragma unroll
        for (int w = 0; w < SP; ++w) {
          const int qi = i * SP + w;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t kk[4] = {kw[j].x, kw[j].y, kw[j].z, kw[j].w};
            uint32_t b0, b1;
            if constexpr (E4M3)
              e4m3x4_to_f16x2(kk[w], b0, b1);
            else
              b0 = kk[2 * w], b1 = kk[2 * w + 1];
            if constexpr (NT == 1)
              mma16<E4M3>(s[j], qf[qi][0], 0u, qf[qi][1], 0u, b0, b1);
            else
              mma16<E4M3>(s[j], qf[qi][0], qf[qi][1], qf[qi][2], qf[qi][3], b0, b1);
          }
        }
      }
      // weights of tokens 4c .. 4c+3, in powers of two
      float kx[4], ve[4];
      if constexpr (E4M3) {
        const uint32_t kw = lds32(vb + S::KB + 4 * c), vw = lds32(vb + S::KB + 16 + 4 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          kx[j] = e8m0_to_f32((kw >> (8 * j)) & 255u);
          ve[j] = e8m0_exp((vw >> (8 * j)) & 255u);
        }
      }
      const bool whole = tok >= cur.s.lo && tok + kRun <= cur.s.n;
      float sc[NT][4], top[NT];
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[t][j] = s[j >> 1][2 * t + (j & 1)] * (E4M3 ? sq[t] * kx[j] : sq[t]);
          if (!whole && (tok + 4 * c + j < cur.s.lo || tok + 4 * c + j >= cur.s.n)) {
            sc[t][j] = -INFINITY;
            if (E4M3) ve[j] = 0.f;
          }
        }
        if constexpr (E4M3) {  // l and its maximum, of this lane's tokens alone
          const float mn = fmaxf(m_l[t], fmaxf(fmaxf(sc[t][0], sc[t][1]), fmaxf(sc[t][2], sc[t][3])));
          const float base = mn == -INFINITY ? 0.f : mn;
          l[t] = l[t] * ex2(m_l[t] - base) + ((ex2(sc[t][0] - base) + ex2(sc[t][1] - base)) +
                                              (ex2(sc[t][2] - base) + ex2(sc[t][3] - base)));
          m_l[t] = mn;
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[t][j] += ve[j];
        }
        top[t] = fmaxf(fmaxf(sc[t][0], sc[t][1]), fmaxf(sc[t][2], sc[t][3]));
        grows |= top[t] > mrun[t];
      }
      if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          top[t] = fmaxf(top[t], __shfl_xor_sync(0xFFFFFFFFu, top[t], 1));
          top[t] = fmaxf(top[t], __shfl_xor_sync(0xFFFFFFFFu, top[t], 2));
          const float mn = fmaxf(mrun[t], top[t]);
          const float al = mn > mrun[t] ? ex2(mrun[t] - mn) : 1.f;
          mrun[t] = mn;
          if (!E4M3) l[t] *= al;
          const float a0 = __shfl_sync(0xFFFFFFFFu, al, 8 * c), a1 = __shfl_sync(0xFFFFFFFFu, al, 8 * c + 4);
#pragma unroll
          for (int m = 0; m < MM; ++m) {
            o[t][m][0] *= a0;
            o[t][m][1] *= a1;
            o[t][m][2] *= a0;
            o[t][m][3] *= a1;
          }
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float base = (mrun[t] == -INFINITY ? 0.f : mrun[t]) - (E4M3 ? 14.f : 0.f);
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = ex2(sc[t][j] - base);
        if (!E4M3) l[t] += (p[0] + p[1]) + (p[2] + p[3]);
        pf[t][0] = pack2<E4M3>(p[0], p[1]);
        pf[t][1] = pack2<E4M3>(p[2], p[3]);
      }
      // O^T: rows g and g + 8 of product m are this lane's dimensions 2m and 2m + 1
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        uint32_t vw[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t row = vb + (4 * c + j) * S::ROWB;
          if constexpr (C >= 8) {
            const uint4 u = lds128(row + (((g + 8 * i) ^ (2 * c)) << 4));
            vw[j][0] = u.x, vw[j][1] = u.y, vw[j][2] = u.z, vw[j][3] = u.w;
          } else {
            const uint2 u = lds64(row + g * 8);
            vw[j][0] = u.x, vw[j][1] = u.y, vw[j][2] = vw[j][3] = 0u;
          }
        }
        constexpr int W = C >= 8 ? 4 : 2;  // 32-bit words a lane holds of a token
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if constexpr (E4M3) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2(__byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140), a0, a1);
              e4m3x4_to_f16x2(__byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16<true>(o[t][(i * W + w) * 2 + hf], a0, a1, a2, a3, pf[t][0], pf[t][1]);
            }
          } else {
            const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
            const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410), a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16<false>(o[t][i * W + w], a0, a1, a2, a3, pf[t][0], pf[t][1]);
          }
        }
      }
    }
    stage = stage + 1 == ST ? 0 : stage + 1;

    const bool last = step + 1 == steps;
    if (cur.u + 1 < cur.s.units && !last) {
      ++cur.u;
      continue;
    }
    // ---- the item ends here (or is cut here): join the warps
    const bool cut = item_u0 > 0 || cur.u + 1 < cur.s.units;
    const int gi = cur.it % P.groups;
    const int h0 = (cur.it / P.groups) * P.G + gi * NQ, rows = min(NQ, P.G - gi * NQ);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float m = E4M3 ? m_l[t] : mrun[t];
      float mm = m;
      mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 1));
      mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 2));
      float lt = mm == -INFINITY ? l[t] : l[t] * ex2(m - mm);
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 1);
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 2);
      if (c == 0) {
        s_fac[warp][g + 8 * t] = mrun[t];
        s_m[warp][g + 8 * t] = mm;
        s_l[warp][g + 8 * t] = lt;
      }
    }
    __syncthreads();
    if (tid < NQ) {
      float mp = -INFINITY, mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < kAdWarps; ++w) {
        mp = fmaxf(mp, s_fac[w][tid]);
        mt = fmaxf(mt, s_m[w][tid]);
      }
#pragma unroll
      for (int w = 0; w < kAdWarps; ++w) {
        lt += mt == -INFINITY ? s_l[w][tid] : s_l[w][tid] * ex2(s_m[w][tid] - mt);
        s_fac[w][tid] = mp == -INFINITY ? 1.f : ex2(s_fac[w][tid] - mp);
      }
      if (cut) {
        const int slot = 2 * blockIdx.x + (first_item ? 0 : 1);
        P.stat[static_cast<size_t>(slot) * NQ + tid] = make_float4(mp, mt, lt, 0.f);
      } else {
        // out = O' 2^(m' - m - 14) / l
        const float fin = (mp == -INFINITY ? 1.f : exp2f(mp - mt - (E4M3 ? 14.f : 0.f))) / lt;
        s_fin[tid] = lt == 0.f ? 0.f : fin;
        if (P.lse && tid < rows)
          P.lse[static_cast<size_t>(cur.b) * P.Hq + h0 + tid] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
      }
    }
    __syncthreads();
    float4 *buf = reinterpret_cast<float4 *>(smem + kAdWarps * ST * S::STAGE);
#pragma unroll
    for (int rd = 0; rd < S::QUADS / 4; ++rd) {
      if (rd) __syncthreads();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = (rd * 4 + x) / MM, m = (rd * 4 + x) % MM;
        const float f0w = s_fac[warp][8 * t + 2 * c], f1w = s_fac[warp][8 * t + 2 * c + 1];
        buf[(warp * 4 + x) * 32 + lane] = make_float4(o[t][m][0] * f0w, o[t][m][1] * f1w, o[t][m][2] * f0w, o[t][m][3] * f1w);
      }
      __syncthreads();
      const int quad = rd * 4 + warp, t = quad / MM, m = quad % MM;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAdWarps; ++w) {
        const float4 u = buf[(w * 4 + warp) * 32 + lane];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      if (cut) {
        const int slot = 2 * blockIdx.x + (first_item ? 0 : 1);
        P.part[(static_cast<size_t>(slot) * S::QUADS + quad) * 32 + lane] = v;
      } else {
        const int r0 = 8 * t + 2 * c;
        const float x0 = s_fin[r0], x1 = s_fin[r0 + 1];
        constexpr int PER = 16 / S::ESZ;  // dimensions of a 16-byte word
        const int dl = 2 * m;             // of the lane's dimensions
        const int d = C >= 8 ? (g + 8 * (dl / PER)) * PER + dl % PER : g * 8 + dl;
        uint16_t *op = P.out + (static_cast<size_t>(cur.b) * P.Hq + h0 + r0) * D + d;
        // a row without weight is 0 (its sums are 0, or its scale is)
        if (r0 < rows) *reinterpret_cast<uint32_t *>(op) = pack2<false>(x0 == 0.f ? 0.f : v.x * x0, x0 == 0.f ? 0.f : v.z * x0);
        if (r0 + 1 < rows)
          *reinterpret_cast<uint32_t *>(op + D) = pack2<false>(x1 == 0.f ? 0.f : v.y * x1, x1 == 0.f ? 0.f : v.w * x1);
      }
    }
    if constexpr (!DIRECT) {
      if (tid == 0 && item_u0 == 0 && cur.u + 1 < cur.s.units) {
        // a cut item that starts here: the blocks whose pieces it covers
        const long long end = f0 + step + (cur.s.units - cur.u) - 1;  // its last unit on the line
        P.meta[blockIdx.x] = make_int4(static_cast<int>(end / share) - static_cast<int>(blockIdx.x) + 1,
                                       2 * static_cast<int>(blockIdx.x) + (first_item ? 0 : 1), cur.it, cur.b);
      }
    }
    first_item = false;
    if (last) break;
    cur.next(P, items);
    item_u0 = 0;
    __syncthreads();
    start_item();
  }
  cp_wait<0>();
}

// Adds the partial sums of the items that were cut, in the order of their pieces: block
// i joins the item that starts in block i's piece and goes on, if there is one.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(512) attn_join_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT>;
  constexpr int NQ = 8 * NT, QUADS = S::QUADS, MM = S::MM, C = S::C;
  constexpr int SPLIT = QUADS >= 16 ? 1 : 16 / QUADS;  // warps that share a quad's parts
  extern __shared__ float fac[];                       // [parts][NQ]
  __shared__ float s_fin[NQ];
  __shared__ float4 s_sum[16][32];
  pdl_wait();
  pdl_trigger();
  const int4 me = P.meta[blockIdx.x];
  const int parts = me.x;
  if (parts < 2) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int gi = me.z % P.groups, h0 = (me.z / P.groups) * P.G + gi * NQ, rows = min(NQ, P.G - gi * NQ);
  // part i is the first slot of block blockIdx.x + i, except part 0
  auto slot = [&](int i) { return i == 0 ? me.y : 2 * (static_cast<int>(blockIdx.x) + i); };
  if (warp < NQ) {
    for (int r = warp; r < NQ; r += 16) {
      float mp = -INFINITY, mt = -INFINITY;
      for (int i = lane; i < parts; i += 32) {
        const float4 s = P.stat[static_cast<size_t>(slot(i)) * NQ + r];
        mp = fmaxf(mp, s.x);
        mt = fmaxf(mt, s.y);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        mp = fmaxf(mp, __shfl_xor_sync(0xFFFFFFFFu, mp, off));
        mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, off));
      }
      float lt = 0.f;
      for (int i = lane; i < parts; i += 32) {
        const float4 s = P.stat[static_cast<size_t>(slot(i)) * NQ + r];
        lt += mt == -INFINITY ? s.z : s.z * ex2(s.y - mt);
        fac[i * NQ + r] = mp == -INFINITY ? 1.f : ex2(s.x - mp);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, off);
      if (lane == 0) {
        const float fin = (mp == -INFINITY ? 1.f : exp2f(mp - mt - (E4M3 ? 14.f : 0.f))) / lt;
        s_fin[r] = lt == 0.f ? 0.f : fin;
        if (P.lse && r < rows)
          P.lse[static_cast<size_t>(me.w) * P.Hq + h0 + r] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
      }
    }
  }
  __syncthreads();
  for (int q0 = 0; q0 < QUADS; q0 += 16 / SPLIT) {
    const int quad = q0 + warp / SPLIT, sub = warp % SPLIT, t = quad / MM, m = quad % MM;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = sub; i < parts; i += SPLIT) {
      const float4 u = P.part[(static_cast<size_t>(slot(i)) * QUADS + quad) * 32 + lane];
      const float a0 = fac[i * NQ + 8 * t + 2 * c], a1 = fac[i * NQ + 8 * t + 2 * c + 1];
      v.x = fmaf(u.x, a0, v.x);
      v.y = fmaf(u.y, a1, v.y);
      v.z = fmaf(u.z, a0, v.z);
      v.w = fmaf(u.w, a1, v.w);
    }
    if constexpr (SPLIT > 1) {
      s_sum[warp][lane] = v;
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int x = 1; x < SPLIT; ++x) {
          const float4 u = s_sum[warp + x][lane];
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
      }
    }
    if (sub == 0) {
      const int r0 = 8 * t + 2 * c;
      const float x0 = s_fin[r0], x1 = s_fin[r0 + 1];
      constexpr int PER = 16 / S::ESZ;
      const int dl = 2 * m, d = C >= 8 ? (g + 8 * (dl / PER)) * PER + dl % PER : g * 8 + dl;
      uint16_t *op = P.out + (static_cast<size_t>(me.w) * P.Hq + h0 + r0) * D + d;
      if (r0 < rows) *reinterpret_cast<uint32_t *>(op) = pack2<false>(x0 == 0.f ? 0.f : v.x * x0, x0 == 0.f ? 0.f : v.z * x0);
      if (r0 + 1 < rows)
        *reinterpret_cast<uint32_t *>(op + D) = pack2<false>(x1 == 0.f ? 0.f : v.y * x1, x1 == 0.f ? 0.f : v.w * x1);
    }
  }
}

namespace {

struct AdPlan {
  int NT, groups, quads, blocks;
  size_t meta, stat, part, bytes;
};

AdPlan plan_of(const k3moe_kv_cache &c, int Hq) {
  AdPlan p;
  const int G = Hq / c.heads;
  p.NT = G <= 8 ? 1 : 2;
  p.groups = (G + 8 * p.NT - 1) / (8 * p.NT);
  p.quads = c.dim / 16 * p.NT;
  const size_t slots = 2 * static_cast<size_t>(kAdMostBlocks);
  p.meta = 0;
  p.stat = (kAdMostBlocks * sizeof(int4) + 255) / 256 * 256;
  p.part = p.stat + slots * 8 * p.NT * sizeof(float4);
  p.bytes = p.part + slots * p.quads * 32 * sizeof(float4);
  return p;
}

template <int D, bool E4M3, int NT>
int launch_attn(AdParams &P, cudaStream_t st) {
  using S = AdShape<D, E4M3, NT>;
  const long long items = static_cast<long long>(P.B) * P.heads * P.groups;
  const int visible = P.max_pages << P.page_shift;  // most tokens an item can have
  const int tokens = P.window > 0 && P.window < visible ? P.window + kRun - 1 : visible;
  const int units = (tokens + kUnit - 1) / kUnit;
  static bool attr = false;
  if (!attr) {
    if (cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM) != cudaSuccess ||
        cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM) != cudaSuccess)
      return -1;
    attr = true;
  }
  if (units <= kDirectUnits && items < (1LL << 31))
    return launch_pdl(attn_decode_kernel<D, E4M3, NT, true>, dim3(static_cast<unsigned>(items)), dim3(kAdThreads), S::SMEM,
                      st, P) == cudaSuccess
               ? 0
               : -1;
  long long blocks = static_cast<long long>(sm_count()) * S::BLOCKS;
  if (blocks > kAdMostBlocks) blocks = kAdMostBlocks;
  const long long most = (items * units + kMinUnits - 1) / kMinUnits;
  if (blocks > most) blocks = most;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (launch_pdl(attn_decode_kernel<D, E4M3, NT, false>, grid, dim3(kAdThreads), S::SMEM, st, P) != cudaSuccess) return -1;
  return launch_pdl(attn_join_kernel<D, E4M3, NT>, grid, dim3(512), blocks * 8 * NT * sizeof(float), st, P) == cudaSuccess
             ? 0
             : -1;
}

}  // namespace

size_t attn_decode_workspace(const k3moe_kv_cache &c, int, int Hq) { return plan_of(c, Hq).bytes; }

int launch_attn_decode(const k3moe_kv_cache &c, int B, int Hq, const uint16_t *q, long long q_stride,
                       const int32_t *table, int max_pages, const int32_t *lens, int window, float scale, uint16_t *out,
                       float *lse, void *ws, int32_t *status, cudaStream_t st) {
  const AdPlan p = plan_of(c, Hq);
  AdParams P;
  P.k = static_cast<const uint8_t *>(c.k), P.v = static_cast<const uint8_t *>(c.v), P.ks = c.k_scales, P.vs = c.v_scales;
  P.heads = c.heads, P.pages = c.pages, P.page_shift = 0;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  P.B = B, P.Hq = Hq, P.G = Hq / c.heads, P.groups = p.groups;
  P.q = q, P.q_stride = q_stride, P.table = table, P.max_pages = max_pages, P.lens = lens;
  P.window = window, P.scale = scale, P.out = out, P.lse = lse;
  uint8_t *w = static_cast<uint8_t *>(ws);
  P.meta = reinterpret_cast<int4 *>(w + p.meta), P.stat = reinterpret_cast<float4 *>(w + p.stat);
  P.part = reinterpret_cast<float4 *>(w + p.part), P.status = status;
  const bool e = c.format == K3MOE_KV_E4M3;
#define K3_AD(D_)                                                                                          \
  if (c.dim == D_)                                                                                         \
    return p.NT == 1 ? (e ? launch_attn<D_, true, 1>(P, st) : launch_attn<D_, false, 1>(P, st))             \
                     : (e ? launch_attn<D_, true, 2>(P, st) : launch_attn<D_, false, 2>(P, st));
  K3_AD(64) K3_AD(128) K3_AD(256)
#undef K3_AD
  return -1;
}

}  // namespace k3moe
