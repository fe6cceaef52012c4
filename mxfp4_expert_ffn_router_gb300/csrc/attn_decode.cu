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
//    share it); a unit is 64 or 128 of its tokens.  All items' units form one line, cut into
//    equal pieces, one per block: blocks end together however uneven the lengths are,
//    and one long sequence fills the GPU.  Lengths are read on the device, so a captured
//    graph follows them.  A piece covers the end of one item, some whole items and the
//    start of another; only the cut ones leave partial sums in the workspace, at
//    most two a block, which attn_join_kernel adds in order.  When every item
//    is short (kDirectTokens), a block takes one item and nothing is cut or joined.
//  * Loads.  Each of the four warps streams every fourth run of 16 or 32 tokens through a ring
//    of its own in shared memory with 16-byte cp.async (stages - 1 runs ahead, across items),
//    so no warp waits for another except where an item ends.  16 tokens from a multiple of
//    16 on never straddle a page (pages hold a multiple of 16 places); the next run's page
//    numbers are loaded a step ahead.  Places not seen are filled with zeros by the copy, so that nothing they hold
//    (NaN, infinities) reaches a product.
//  * Products.  mma.sync m16n8k16 (f16 or bf16, fp32 sums): with at most 16 query heads
//    sharing a key the products are a small part of the time even at this instruction's
//    rate, and its operands come straight from registers, where E4M3 codes are converted.
//    S = Q K^T has the query heads as rows; O^T = V^T P^T has dimensions as rows
//    and 8 query heads as columns, so that S's registers are P^T's.  The order of
//    dimensions and tokens inside a product is free as long as both operands agree, and
//    is chosen so that a lane's share of K and V is whole 16-byte words.
//  * E4M3.  Codes are converted to f16 (exact; the E4M3 form of this instruction does the
//    same within, on both operands and for every product: measured slower).  A query row is
//    scaled by a power of two to a maximum in [2^14, 2^15), exact but for values below 2^-28
//    of it.  K's scale multiplies the score.  V's scale 2^e joins the weight: w_i = exp2(s_i + e_i - m')
//    with its own running maximum m' of s_i + e_i, times 2^14, rounded to f16 (11 bits
//    down to 2^-28 of the largest, so that a token with a large score and a tiny value
//    costs the others nothing), while l sums exp2(s_i - m) in fp32 with m = max s_i.
//  * bf16.  Q, K and V enter as they are; the weights are rounded to bf16, as V is.
#include <cuda_fp16.h>

#include <type_traits>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"
#include "tc_sm103.cuh"

namespace k3moe {

namespace {

#ifndef KRR
#define KRR (ROWB <= 64 ? 4 : ROWB <= 128 ? 2 : 1)
#endif
#ifndef KST
#define KST 3
#endif
#ifndef KQS
#define KQS 32
#endif
#ifndef KBL
#define KBL (ROWB <= 256 && W == 4 ? 2 : 1)
#endif
constexpr int kRun = 16;                 // tokens of a product
#ifndef KDT
#define KDT 1024
#endif
#ifndef KDW
#define KDW 2048
#endif
constexpr int kDirectTokens = KDT, kWideTokens = KDW;       // items of at most this many tokens are never cut
constexpr int kMinTokens = 256;          // smallest piece of a block
#ifndef KWU
#define KWU 4
#define KWI 6
#endif
constexpr int kUnitLen = KWU, kItemLen = KWI;  // length on the line of a unit, and of an item beside its units
constexpr int kJoinParts = 8;            // parts of an item that one warp joins
constexpr int kAdMostBlocks = 152 * 12;  // pieces (bounds the workspace)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zeros(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
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

// The same from zero: d = a b.
template <bool H>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  if constexpr (H)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Not 0 where a byte of w is 255.
__device__ __forceinline__ uint32_t byte_255(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;
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
  int4 *meta;    // [2 blocks]: {first slot, parts, item, sequence} of the cut items of a piece: one that began
                 // before it, one that begins in it and goes on (parts 0: none)
  float4 *stat;  // [2 blocks][8 NT]: {m', m, l, -}
  float4 *part;  // [2 blocks][accumulator quads][32 lanes]
  int32_t *status;
};

// a / b for a, b >= 0: mostly both fit 32 bits, where a division costs a fifth.
__device__ __forceinline__ long long div_small(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// The tokens of one sequence that are seen, lo .. n - 1, and the place its units count from.
struct Seen {
  int n, lo, t0;
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
  return s;
}
template <int UNIT>
__device__ __forceinline__ int units_of(const Seen &s) {
  return static_cast<int>((static_cast<unsigned>(s.n - s.t0) + (UNIT - 1)) / UNIT);
}

// A block's piece [from, to) of the line, and where one warp is in it.  An item that begins at
// `begin` lies on the line as kItemLen, then kUnitLen for each of its units; a unit belongs
// to the piece in which it begins.
template <int UNIT>
struct Walk {
  int b, head, group;    // sequence, key-value head, which of its items
  int n, lo, t0;
  unsigned tok, stop;    // the warp's next run begins at tok; the piece holds the item's runs below stop
  long long begin;       // of the item
  bool more;             // whether a run is left
  __device__ __forceinline__ int units() const { return units_of<UNIT>({n, lo, t0}); }
  // The item's first unit at or past place x of the line.
  __device__ __forceinline__ int unit_at(long long x) const {
    const long long u = (x - begin - kItemLen + kUnitLen - 1) / kUnitLen;
    return u < 0 ? 0 : u > units() ? units() : static_cast<int>(u);
  }
  // Begins the item at `begin`, from its first unit in [from, to) on; first: the warp's place in a unit.
  __device__ __forceinline__ void enter(long long from, long long to, int first) {
    tok = static_cast<unsigned>(t0) + static_cast<unsigned>(unit_at(from)) * UNIT + first;
    stop = static_cast<unsigned>(t0) + static_cast<unsigned>(unit_at(to)) * UNIT + first;
  }
  __device__ __forceinline__ void set(const Seen &s) { n = s.n, lo = s.lo, t0 = s.t0; }
  __device__ __forceinline__ void next_item(const AdParams &P, long long from, long long to, int first) {
    begin += static_cast<long long>(units()) * kUnitLen + kItemLen;
    more = begin + kItemLen < to;
    if (!more) return;
    if (++group == P.groups) {
      group = 0;
      if (++head == P.heads) {
        head = 0;
        Seen s;
        do {
          if (++b >= P.B) {  // past the last unit of all
            more = false;
            return;
          }
          s = seen_of(P, b, false);
        } while (s.n <= s.t0);
        set(s);
      }
    }
    enter(from, to, first);
  }
};

template <int D, bool E4M3, int NT, int W>
struct AdShape {
  static constexpr int ESZ = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;            // bytes of a cached vector
  static constexpr int C = ROWB / 16;             // 16-byte words of it
  static constexpr int KB = kRun * ROWB;          // bytes of 16 tokens' keys
  static constexpr int MM = D / 16;               // products (16 dimensions each) of 16 tokens and 8 query heads
  static constexpr int QUADS = MM * NT;           // accumulator quads per lane
  // A warp's step is RR times 16 tokens: 4 to 16 KB, so that what a step costs besides its bytes counts little
  static constexpr int RR = KRR;
  static constexpr int RUN = RR * kRun;
  static constexpr int UNIT = RUN * W;            // tokens of a block's step
  static constexpr int SUB = 2 * KB;              // keys and values of 16 tokens; a multiple of 128: words swizzle by xor
  static constexpr int SCALES = E4M3 ? 32 : 0;    // scale bytes of 16 tokens, after all stages
  // stages and blocks per SM: about 100 KB of loads in flight per SM
  static constexpr int STAGES = KST;
  static constexpr int BLOCKS = KBL;
  // quads that the warps exchange at once where an item ends, each in the stage it has just used
  static constexpr int QR = RR * SUB / 512 < QUADS ? RR * SUB / 512 : QUADS;
  // query fragments: in registers, or from 32 of them on in shared memory (the same for all warps)
  static constexpr int QREGS = D / 16 * 2 * NT;
  static constexpr int QSMEM = QREGS >= KQS ? QREGS * 32 * 4 : 0;
  static constexpr int SMEM = W * STAGES * RR * (SUB + SCALES) + QSMEM + 128;
};

// First of the two neighbouring dimensions that a lane of group g holds of product m.
template <int D, bool E4M3>
__device__ __forceinline__ int quad_dim(int m, int g) {
  constexpr int PER = E4M3 ? 16 : 8;  // dimensions of a 16-byte word
  const int dl = 2 * m;               // of the lane's dimensions
  return D / PER >= 8 ? (g + 8 * (dl / PER)) * PER + dl % PER : g * 8 + dl;
}

// Two neighbouring dimensions of a row, times f (0: a row without weight, whatever the sums are).
__device__ __forceinline__ void store_row2(uint16_t *p, float f, float a, float b, bool on) {
  if (on) *reinterpret_cast<uint32_t *>(p) = f == 0.f ? 0u : pack2<false>(a * f, b * f);
}

}  // namespace

template <int D, bool E4M3, int NT, int W, bool DIRECT>
__global__ void __launch_bounds__(W * 32, (AdShape<D, E4M3, NT, W>::BLOCKS))
    attn_decode_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT, W>;
  constexpr int THREADS = W * 32;
  constexpr int C = S::C, MM = S::MM, ST = S::STAGES, RR = S::RR, UNIT = S::UNIT, NQ = 8 * NT;
  constexpr int KL = C / 4;             // words of a key a lane reads
  constexpr int SP = E4M3 ? 4 : 2;      // products of 16 dimensions per such word
  constexpr int VL = C >= 8 ? C / 8 : 1;  // words of a value a lane reads
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((128u - (su32(smem_raw) & 127u)) & 127u);
  __shared__ __align__(16) float s_mp[NQ][W], s_m[NQ][W], s_l[NQ][W];
  __shared__ long long s_scan[W];
  __shared__ long long s_begin;
  __shared__ int s_start[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int items = P.heads * P.groups, first = warp * S::RUN;
  // hints only: nothing of these is read before the wait
  if (tid < (P.B + 31) / 32) prefetch_l2(P.lens + 32 * tid);
  pdl_wait();
  pdl_trigger();

  auto zero_rows = [&]() {  // of the sequences that see nothing; every block takes its share
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      const Seen s = seen_of(P, b, false);
      if (s.n > s.t0) continue;
      for (size_t i = tid; i < static_cast<size_t>(P.Hq) * D / 8; i += THREADS)
        reinterpret_cast<uint4 *>(P.out + static_cast<size_t>(b) * P.Hq * D)[i] = make_uint4(0, 0, 0, 0);
      if (P.lse)
        for (int i = tid; i < P.Hq; i += THREADS) P.lse[static_cast<size_t>(b) * P.Hq + i] = -INFINITY;
    }
  };

  // ---- this block's piece
  Walk<UNIT> cur;
  long long from = 0, to = 1LL << 62, share = 0;
  if constexpr (DIRECT) {
    cur.b = blockIdx.x / items;
    const int item = blockIdx.x - cur.b * items;
    cur.head = item / P.groups;
    cur.group = item - cur.head * P.groups;
    cur.set(seen_of(P, cur.b, tid == 0));
    cur.begin = 0;
    cur.more = true;
    cur.enter(from, to, first);
    if (cur.n <= cur.t0) {  // sees nothing
      const int h0 = cur.head * P.G + cur.group * NQ;
      const int rows = min(NQ, P.G - cur.group * NQ);
      const size_t row = static_cast<size_t>(cur.b) * P.Hq + h0;
      for (int i = tid; i < rows * D / 8; i += THREADS)
        reinterpret_cast<uint4 *>(P.out + row * D)[i] = make_uint4(0, 0, 0, 0);
      if (P.lse && tid < rows) P.lse[row + tid] = -INFINITY;
      return;
    }
  } else {
    // thread t measures sequences [t per, t per + per); a scan finds the piece
    const int per = (P.B + THREADS - 1) / THREADS;
    const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
    auto length = [&](int b, bool report) {  // of an item of sequence b on the line
      const int u = units_of<UNIT>(seen_of(P, b, report));
      return u ? static_cast<long long>(u) * kUnitLen + kItemLen : 0LL;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += length(b, blockIdx.x == 0);
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
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    share = max(static_cast<long long>(kMinTokens / UNIT * kUnitLen), div_small(total + gridDim.x - 1, gridDim.x));
    from = static_cast<long long>(blockIdx.x) * share;
    to = min(total, from + share);
    const long long ahead = before + incl - mine;  // of this thread's sequences
    if (from < to && from >= ahead && from < ahead + mine) {
      long long at = ahead, len;
      int b = b0;
      for (;; ++b) {
        len = length(b, false);
        if (from < at + len * items) break;
        at += len * items;
      }
      const int item = static_cast<int>(div_small(from - at, len));
      s_begin = at + item * len;
      s_start[0] = b;
      s_start[1] = item;
    }
    if (tid < 2) P.meta[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (from >= to) {
      zero_rows();
      return;
    }
    cur.b = s_start[0];
    cur.head = s_start[1] / P.groups;
    cur.group = s_start[1] - cur.head * P.groups;
    cur.set(seen_of(P, cur.b, false));
    cur.begin = s_begin;
    cur.more = true;
    cur.enter(from, to, first);
    if (cur.tok >= cur.stop) cur.next_item(P, from, to, first);  // the piece begins behind the item's last unit
    if (!cur.more || cur.tok >= cur.stop) {                      // or ends before its first
      zero_rows();
      return;
    }
  }

  // ---- loads: the run at `pre` into stage st.  Lane l copies words l, l + 32, .. of 16 tokens' keys
  // and values: row lr + i RI, word lx.  Word w of key row r lies at w ^ 4 (r & 1), of value row r at
  // w ^ 2 (r / 4): the reads of fragments below then meet all banks evenly.
  constexpr int RI = C >= 32 ? 1 : 32 / C;  // rows between a lane's words
  const uint32_t ring = su32(smem) + warp * (ST * RR * S::SUB);
  const uint32_t sring = su32(smem) + W * ST * RR * S::SUB + warp * (ST * RR * S::SCALES);
  const int lr = lane / C, lx = lane % C;
  const uint32_t kdst = lr * S::ROWB + ((C == 8 || C == 16 ? lx ^ (4 * (lr & 1)) : lx) << 4);
  const uint32_t vdst = S::KB + lr * S::ROWB + (lx << 4);
  const uint8_t *const klane = P.k + lane * 16, *const vlane = P.v + lane * 16;
  const unsigned place = (1u << P.page_shift) - 1u, page_vecs = static_cast<unsigned>(P.heads) << P.page_shift;
  Walk<UNIT> pre = cur;
  uint32_t bad = 0;    // bit st RR + r: a page number outside the cache
  int page[RR];
  auto pages = [&]() {  // of the run at `pre`
    const int32_t *row = P.table + static_cast<size_t>(pre.b) * P.max_pages;
#pragma unroll
    for (int r = 0; r < RR; ++r) {
      const unsigned tok = pre.tok + r * kRun;
      page[r] = tok < static_cast<unsigned>(pre.n) ? __ldg(row + (tok >> P.page_shift)) : -1;
    }
  };
  auto issue = [&](int st) {
    if (pre.more) {
#pragma unroll
      for (int r = 0; r < RR; ++r) {
        const unsigned tok = pre.tok + r * kRun;
        const int tile = st * RR + r;
        if (tok < static_cast<unsigned>(pre.n)) {
          if (static_cast<unsigned>(page[r]) >= static_cast<unsigned>(P.pages)) {
            bad |= 1u << tile;
            if (lane == 0) set_status(P.status, K3MOE_DEV_BOUNDS);
          } else {
            if (bad) bad &= ~(1u << tile);
            const size_t vec = static_cast<size_t>(static_cast<unsigned>(page[r])) * page_vecs +
                               ((static_cast<unsigned>(pre.head) << P.page_shift) + (tok & place));
            const uint8_t *kp = klane + vec * S::ROWB, *vp = vlane + vec * S::ROWB;
            const uint32_t kd = ring + tile * S::SUB + kdst, vd = ring + tile * S::SUB + vdst;
            const bool whole = tok >= static_cast<unsigned>(pre.lo) && tok + kRun <= static_cast<unsigned>(pre.n);
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
              // the part of the swizzles that varies with i
              const uint32_t ki = C == 32 ? (i & 1) << 6 : 0, vi = C >= 8 ? ((i * RI) >> 2) << 5 : 0;
              if (whole) {
                cp16(((kd ^ ki) + i * RI * S::ROWB), kp + i * 512);
                cp16(((vd ^ vi) + i * RI * S::ROWB), vp + i * 512);
              } else {
                const unsigned at = tok + lr + i * RI;
                const bool on = at >= static_cast<unsigned>(pre.lo) && at < static_cast<unsigned>(pre.n);
                cp16_or_zeros((kd ^ ki) + i * RI * S::ROWB, kp + i * 512, on);
                cp16_or_zeros((vd ^ vi) + i * RI * S::ROWB, vp + i * 512, on);
              }
            }
            if (E4M3 && lane < 2) cp16(sring + tile * S::SCALES + 16 * lane, (lane ? P.vs : P.ks) + vec);
          }
        }
      }
      pre.tok += UNIT;
      if (pre.tok >= pre.stop) {
        if (DIRECT)
          pre.more = false;
        else
          pre.next_item(P, from, to, first);
      }
      if (pre.more) pages();
    }
    cp_commit();
  };
  pages();
#pragma unroll
  for (int st = 0; st < ST - 1; ++st) issue(st);

  constexpr int QN = D / 16, QW = 2 * NT;  // products along the dimensions, registers of the query rows in each
  constexpr bool QS = S::QSMEM > 0;
  uint32_t qf[QS ? 1 : QN][QW];
  uint4 *const q_sm = reinterpret_cast<uint4 *>(smem + W * ST * RR * (S::SUB + S::SCALES));
  uint2 raw[D / 16][NT];
  float sq[NT];  // scale of a raw score, in powers of two
  float o[NT][MM][4], mrun[NT], m_l[NT], l[NT];
  auto load_q = [&](const Walk<UNIT> &at) {
    const int h0 = at.head * P.G + at.group * NQ, rows = min(NQ, P.G - at.group * NQ);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = g + 8 * t;
      const uint16_t *qp = P.q + at.b * P.q_stride + static_cast<size_t>(h0 + r) * D + c * (16 / S::ESZ);
#pragma unroll
      for (int i = 0; i < KL; ++i)
#pragma unroll
        for (int w = 0; w < SP; ++w)
          raw[i * SP + w][t] =
              r < rows ? __ldg(reinterpret_cast<const uint2 *>(qp + i * (64 / S::ESZ) + 4 * w)) : make_uint2(0, 0);
    }
  };
  auto start_item = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float up = 1.f;
      sq[t] = P.scale * kLog2e;
      if constexpr (E4M3) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < QN; ++i) {
          const uint2 u = raw[i][t];
          mx = max(mx, max(max((u.x << 16) & 0x7FFFFFFFu, u.x & 0x7FFF0000u),
                           max((u.y << 16) & 0x7FFFFFFFu, u.y & 0x7FFF0000u)));
        }
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        // 2^(14 - floor(log2 max)), as far as fp32 has it
        const int e = mx == 0 ? 0 : max(-126, min(127, 14 + 127 - static_cast<int>(mx >> 23)));
        up = exp2i(e);
        sq[t] *= mx_pow2(-e);
      }
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        uint2 u = raw[i][t];
        if constexpr (E4M3)
          u = make_uint2(pack2<true>(__uint_as_float(u.x << 16) * up, __uint_as_float(u.x & 0xFFFF0000u) * up),
                         pack2<true>(__uint_as_float(u.y << 16) * up, __uint_as_float(u.y & 0xFFFF0000u) * up));
        if constexpr (QS) {  // (every warp writes the same)
          uint32_t *const to_sm = reinterpret_cast<uint32_t *>(&q_sm[(NT == 1 ? i / 2 : i) * 32 + lane]);
          to_sm[NT == 1 ? 2 * (i & 1) : t] = u.x;
          to_sm[NT == 1 ? 2 * (i & 1) + 1 : NT + t] = u.y;
        } else {
          qf[i][t] = u.x;
          qf[i][NT + t] = u.y;
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

  constexpr bool kEarlyQ = D / 16 * NT <= 8;  // as far as there are registers for it
  bool first_item = true;
  int stage = 0, after = ST - 1;  // the stage in use, and the one that is loaded next
  load_q(cur);
  start_item();
  if (QS) __syncthreads();
  for (;;) {
    __syncwarp();  // every lane is done with the stage that is loaded next
    issue(after);
    after = after + 1 == ST ? 0 : after + 1;
    cp_wait<ST - 1>();
    __syncwarp();
    if (cur.tok < static_cast<unsigned>(cur.n)) {
      const uint32_t base0 = ring + stage * (RR * S::SUB), sbase = sring + stage * (RR * S::SCALES);
      const bool whole = cur.tok >= static_cast<unsigned>(cur.lo) &&
                         cur.tok + S::RUN <= static_cast<unsigned>(cur.n) && bad == 0u;
      // S: columns 2c, 2c+1 of product j of 16 tokens are tokens 4c + 2j, 4c + 2j + 1.  Where a step
      // has 16 tokens there are two partial sums each, so that a product does not wait for the one before it
      constexpr int CH = RR == 1 ? 2 : 1;
      float s[RR][CH][2][4];
      const uint32_t kofs = (4 * (g >> 1) + (g & 1)) * S::ROWB + (c << 4) + (C >= 8 ? (g & 1) << 6 : 0);
#pragma unroll
      for (int i = 0; i < KL; ++i) {
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          uint4 kw[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kw[j] = lds128(((base0 + r * S::SUB + kofs) ^ ((i & 1) << 6)) + (i >> 1) * 128 + 2 * j * S::ROWB);
#pragma unroll
          for (int w = 0; w < SP; ++w) {
            const int qi = i * SP + w;
            uint32_t a[QW];
            if constexpr (QS) {
              if constexpr (NT == 1)
                *reinterpret_cast<uint2 *>(a) = reinterpret_cast<const uint2 *>(&q_sm[(qi / 2) * 32 + lane])[qi & 1];
              else
                *reinterpret_cast<uint4 *>(a) = q_sm[qi * 32 + lane];
            } else {
#pragma unroll
              for (int x = 0; x < QW; ++x) a[x] = qf[qi][x];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t kk[4] = {kw[j].x, kw[j].y, kw[j].z, kw[j].w};
              uint32_t b0, b1;
              if constexpr (E4M3)
                e4m3x4_to_f16x2(kk[w], b0, b1);
              else
                b0 = kk[2 * w], b1 = kk[2 * w + 1];
              float(&d)[4] = s[r][qi & (CH - 1)][j];
              const uint32_t a1 = NT == 1 ? 0u : a[1], a2 = NT == 1 ? a[1] : a[QW - 2], a3 = NT == 1 ? 0u : a[QW - 1];
              if (qi < CH)
                mma16_first<E4M3>(d, a[0], a1, a2, a3, b0, b1);
              else
                mma16<E4M3>(d, a[0], a1, a2, a3, b0, b1);
            }
          }
        }
      }
      // weights of tokens 4c .. 4c+3 of each 16, in powers of two
      float sc[NT][4 * RR], ve[4 * RR];
      if constexpr (E4M3) {
        float kx[4 * RR];
        uint32_t kw[RR], vw[RR], odd = 0;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          kw[r] = lds32(sbase + r * S::SCALES + 4 * c);
          vw[r] = lds32(sbase + r * S::SCALES + 16 + 4 * c);
          odd |= byte_255(kw[r]) | byte_255(vw[r]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // byte j << 23 (0 stands for 2^-127), and byte j - 127
            kx[4 * r + j] = fmaxf(__uint_as_float(__byte_perm(kw[r], 0u, 0x0444 | (j << 12)) >> 1),
                                  __uint_as_float(0x00400000u));
            ve[4 * r + j] = __uint_as_float(__byte_perm(vw[r], 0x4B000000u, 0x7440 | j)) - 8388735.0f;
          }
        }
        if (odd) {  // NaN
#pragma unroll
          for (int j = 0; j < 4 * RR; ++j) {
            if (((kw[j >> 2] >> (8 * (j & 3))) & 255u) == 255u) kx[j] = __uint_as_float(0x7FC00000u);
            if (((vw[j >> 2] >> (8 * (j & 3))) & 255u) == 255u) ve[j] = __uint_as_float(0x7FC00000u);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4 * RR; ++j) sc[t][j] = sq[t] * kx[j];
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4 * RR; ++j) sc[t][j] = sq[t];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4 * RR; ++j) {
          const int h = (j >> 1) & 1, x = j & 1;
          float raw_s = s[j >> 2][0][h][2 * t + x];
          if constexpr (CH == 2) raw_s += s[j >> 2][CH - 1][h][2 * t + x];
          sc[t][j] *= raw_s;
        }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 4 * RR; ++j) {
          const unsigned tok = cur.tok + (j >> 2) * kRun + 4 * c + (j & 3);
          if (tok < static_cast<unsigned>(cur.lo) || tok >= static_cast<unsigned>(cur.n) ||
              ((bad >> (stage * RR + (j >> 2))) & 1u)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][j] = -INFINITY;
            if (E4M3) ve[j] = 0.f;
          }
        }
      }
      float top[NT];
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (E4M3) {  // l and its maximum, of this lane's tokens alone
          float mn = m_l[t], add = 0.f;
#pragma unroll
          for (int j = 0; j < 4 * RR; ++j) mn = fmaxf(mn, sc[t][j]);
          const float base = mn == -INFINITY ? 0.f : mn;
#pragma unroll
          for (int j = 0; j < 4 * RR; j += 2) add += ex2(sc[t][j] - base) + ex2(sc[t][j + 1] - base);
          l[t] = l[t] * ex2(m_l[t] - base) + add;
          m_l[t] = mn;
#pragma unroll
          for (int j = 0; j < 4 * RR; ++j) sc[t][j] += ve[j];
        }
        top[t] = sc[t][0];
#pragma unroll
        for (int j = 1; j < 4 * RR; ++j) top[t] = fmaxf(top[t], sc[t][j]);
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
      uint32_t pf[RR][NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float base = (mrun[t] == -INFINITY ? 0.f : mrun[t]) - (E4M3 ? 14.f : 0.f);
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = ex2(sc[t][4 * r + j] - base);
          if (!E4M3) l[t] += (p[0] + p[1]) + (p[2] + p[3]);
          pf[r][t][0] = pack2<E4M3>(p[0], p[1]);
          pf[r][t][1] = pack2<E4M3>(p[2], p[3]);
        }
      }
      // O^T: rows g and g + 8 of product m are this lane's dimensions 2m and 2m + 1.  16 tokens that are
      // not seen at all (past the end, or of a bad page) were not loaded and are left out
#pragma unroll
      for (int r = 0; r < RR; ++r) {
        if (r > 0 && cur.tok + r * kRun >= static_cast<unsigned>(cur.n)) break;
        if (bad && ((bad >> (stage * RR + r)) & 1u)) continue;
        const uint32_t vb = base0 + r * S::SUB + S::KB + 4 * c * S::ROWB + (C >= 8 ? (g ^ (2 * c)) << 4 : g * 8);
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          uint32_t vw[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (C >= 8) {
              const uint4 u = lds128(vb + j * S::ROWB + i * 128);
              vw[j][0] = u.x, vw[j][1] = u.y, vw[j][2] = u.z, vw[j][3] = u.w;
            } else {
              const uint2 u = lds64(vb + j * S::ROWB);
              vw[j][0] = u.x, vw[j][1] = u.y, vw[j][2] = vw[j][3] = 0u;
            }
          }
            constexpr int VW = C >= 8 ? 4 : 2;  // 32-bit words a lane holds of a token
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            if constexpr (E4M3) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2(__byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140), a0, a1);
                e4m3x4_to_f16x2(__byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma16<true>(o[t][(i * VW + w) * 2 + hf], a0, a1, a2, a3, pf[r][t][0], pf[r][t][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
              const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410), a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16<false>(o[t][i * VW + w], a0, a1, a2, a3, pf[r][t][0], pf[r][t][1]);
            }
          }
        }
      }
    }
    const int used = stage;
    stage = stage + 1 == ST ? 0 : stage + 1;
    cur.tok += UNIT;
    if (cur.tok < cur.stop) continue;

    // ---- the item ends here (or is cut here): join the warps
    const Walk<UNIT> done = cur;
    const bool began_before = !DIRECT && done.unit_at(from) > 0, cut = began_before || (!DIRECT && done.unit_at(to) < done.units());
    const int h0 = done.head * P.G + done.group * NQ, rows = min(NQ, P.G - done.group * NQ);
    if (DIRECT)
      cur.more = false;
    else
      cur.next_item(P, from, to, first);
    if (kEarlyQ && cur.more) load_q(cur);  // arrives while the warps join
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float m = E4M3 ? m_l[t] : mrun[t];
      float mm = m;
      mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 1));
      mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 2));
      float lt = mm == -INFINITY ? l[t] : l[t] * ex2(m - mm);
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 1);
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 2);
      if (c == 0) {
        s_mp[g + 8 * t][warp] = mrun[t];
        s_m[g + 8 * t][warp] = mm;
        s_l[g + 8 * t][warp] = lt;
      }
    }
    // quad x of warp w: in the stage that the warp has just used, and loads again only after this
    float4 *buf = reinterpret_cast<float4 *>(smem + used * (RR * S::SUB));
    constexpr int NEXT = ST * RR * S::SUB / 16;  // from one warp's stages to the next's
    const int slot = 2 * blockIdx.x + (first_item ? 0 : 1);
    float fin[2], fac[2][W];
    int t_of = -1;
    __syncwarp();
#pragma unroll
    for (int q0 = 0; q0 < S::QUADS; q0 += S::QR) {
#pragma unroll
      for (int x = 0; x < S::QR; ++x) {
        const int t = (q0 + x) / MM, m = (q0 + x) % MM;
        buf[warp * NEXT + x * 32 + lane] = make_float4(o[t][m][0], o[t][m][1], o[t][m][2], o[t][m][3]);
      }
      __syncthreads();
      // this warp's share of the quads, summed over the warps at their common maximum
#pragma unroll
      for (int x0 = 0; x0 < S::QR; x0 += W) {
        const int x = x0 + warp, quad = q0 + x, t = quad / MM, m = quad % MM;
        if (S::QR % W && x >= S::QR) continue;
        if (t != t_of) {
          t_of = t;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * t + 2 * c + e;
            float mp = -INFINITY, mt = -INFINITY, lt = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) mp = fmaxf(mp, s_mp[r][w]), mt = fmaxf(mt, s_m[r][w]);
            const float mb = mt == -INFINITY ? 0.f : mt, pb = mp == -INFINITY ? 0.f : mp;
#pragma unroll
            for (int w = 0; w < W; ++w) {
              lt = fmaf(s_l[r][w], ex2(s_m[r][w] - mb), lt);
              fac[e][w] = ex2(s_mp[r][w] - pb);
            }
            // out = O' 2^(m' - m - 14) / l; a row without weight is 0
            fin[e] = lt == 0.f ? 0.f : __fdividef(exp2f(pb - mb - (E4M3 ? 14.f : 0.f)), lt);
            if (m == 0 && g == 0) {
              if (cut)
                P.stat[static_cast<size_t>(slot) * NQ + r] = make_float4(mp, mt, lt, 0.f);
              else if (P.lse && r < rows)
                P.lse[static_cast<size_t>(done.b) * P.Hq + h0 + r] = lt == 0.f ? -INFINITY : (mb + log2f(lt)) * kLn2;
            }
          }
        }
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 u = buf[w * NEXT + x * 32 + lane];
          v.x = fmaf(u.x, fac[0][w], v.x);
          v.y = fmaf(u.y, fac[1][w], v.y);
          v.z = fmaf(u.z, fac[0][w], v.z);
          v.w = fmaf(u.w, fac[1][w], v.w);
        }
        if (cut) {
          P.part[(static_cast<size_t>(slot) * S::QUADS + quad) * 32 + lane] = v;
        } else {
          const int r0 = 8 * t + 2 * c;
          uint16_t *op = P.out + (static_cast<size_t>(done.b) * P.Hq + h0 + r0) * D + quad_dim<D, E4M3>(m, g);
          store_row2(op, fin[0], v.x, v.z, r0 < rows);
          store_row2(op + D, fin[1], v.y, v.w, r0 + 1 < rows);
        }
      }
      __syncthreads();
    }
    if constexpr (!DIRECT) {
      if (tid == 0 && cut) {  // the blocks whose pieces the item covers
        const long long unit0 = done.begin + kItemLen;
        const int b0 = static_cast<int>(div_small(unit0, share));
        P.meta[2 * blockIdx.x + (began_before ? 0 : 1)] = make_int4(
            // not the first item of its block if the one before has a unit there
            2 * b0 + (done.begin - kUnitLen >= b0 * share ? 1 : 0),
            static_cast<int>(div_small(unit0 + static_cast<long long>(done.units() - 1) * kUnitLen, share)) - b0 + 1,
            done.head * P.groups + done.group, done.b);
      }
    }
    if (!cur.more) break;
    first_item = false;
    if (!kEarlyQ) load_q(cur);
    start_item();
    if (QS) __syncthreads();
  }
  cp_wait<0>();
  if constexpr (!DIRECT) zero_rows();
}

// Adds the partial sums of the items that were cut, in the order of their pieces.  The
// blocks are those of the kernel before; each takes its share of the accumulator quads
// of the (at most two) cut items that it holds a piece of, so that an item of many pieces
// is joined by many blocks.  A warp adds up to kJoinParts parts of a quad, their
// statistics and sums loaded together; where there are more, warps share a quad.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(256) attn_join_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT, 4>;
  constexpr int NQ = 8 * NT, QUADS = S::QUADS, MM = S::MM;
  __shared__ float4 s_sum[8][32], s_stat[8][2][4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();
  const int4 both[2] = {P.meta[2 * blockIdx.x], P.meta[2 * blockIdx.x + 1]};
  // quads of each item that are this block's: mine, mine + parts, ..; warps that share one
  int count[2], split[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int parts = both[e].y, mine = static_cast<int>(blockIdx.x) - (both[e].x >> 1);
    count[e] = parts > 1 && mine < QUADS ? (QUADS - 1 - mine) / parts + 1 : 0;
    split[e] = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;
  }
  // a quad's warps lie in one round of eight: splits are powers of two, and the second item's
  // tasks start at a multiple of its split
  const int tasks0 = count[0] * split[0], from1 = (tasks0 + split[1] - 1) / split[1] * split[1];
  const int tasks = count[1] ? from1 + count[1] * split[1] : tasks0;
  for (int base = 0; base < tasks; base += 8) {
    int task = base + warp;
    const int e = task < tasks0 ? 0 : 1;
    if (e) task -= from1;
    const int sp = split[e], sub = task & (sp - 1), q = task / sp;
    const bool in = task >= 0 && q < count[e];
    const int4 me = both[e];
    const int parts = me.y, b0 = me.x >> 1, quad = static_cast<int>(blockIdx.x) - b0 + q * parts;
    const int t = quad / MM, m = quad - t * MM, r0 = 8 * t + 2 * c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mp[2], mt[2], lt[2];
    // the sum of N parts (statistics s of this lane's two rows, sums u), all at once
    auto add = [&](const auto &s, const auto &u, auto N) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float np = -INFINITY, nt = -INFINITY;
#pragma unroll
        for (int i = 0; i < N.value; ++i) np = fmaxf(np, s[i][x].x), nt = fmaxf(nt, s[i][x].y);
        const float pb = np == -INFINITY ? 0.f : np, mb = nt == -INFINITY ? 0.f : nt;
        float a = 0.f, b = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < N.value; ++i) {
          const float f = ex2(s[i][x].x - pb);
          a = fmaf(x ? u[i].y : u[i].x, f, a);
          b = fmaf(x ? u[i].w : u[i].z, f, b);
          sum = fmaf(s[i][x].z, ex2(s[i][x].y - mb), sum);
        }
        (x ? v.y : v.x) = a;
        (x ? v.w : v.z) = b;
        mp[x] = np, mt[x] = nt, lt[x] = sum;
      }
    };
    const float4 none = make_float4(-INFINITY, -INFINITY, 0.f, 0.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
    mp[0] = mp[1] = mt[0] = mt[1] = -INFINITY;
    lt[0] = lt[1] = 0.f;
    if (in) {
      // part i lies in the first slot of block b0 + i, part 0 in me.x; this warp adds a run of them
      const int i0 = parts * sub / sp, i1 = parts * (sub + 1) / sp;
      for (int i = i0; i < i1; i += kJoinParts) {
        float4 s[kJoinParts + 1][2], u[kJoinParts + 1];
#pragma unroll
        for (int x = 0; x < kJoinParts; ++x) {
          const bool on = i + x < i1;
          const size_t slot = static_cast<size_t>(i + x == 0 ? me.x : 2 * (b0 + i + x));
          s[x][0] = on ? P.stat[slot * NQ + r0] : none;
          s[x][1] = on ? P.stat[slot * NQ + r0 + 1] : none;
          u[x] = on ? P.part[(slot * QUADS + quad) * 32 + lane] : zero;
        }
        s[kJoinParts][0] = make_float4(mp[0], mt[0], lt[0], 0.f);
        s[kJoinParts][1] = make_float4(mp[1], mt[1], lt[1], 0.f);
        u[kJoinParts] = v;
        add(s, u, std::integral_constant<int, kJoinParts + 1>());
      }
    }
    if (max(split[0], split[1]) > 1) {  // (uniform: the block's)
      s_sum[warp][lane] = v;
      if (g == 0) {
        s_stat[warp][0][c] = make_float4(mp[0], mt[0], lt[0], 0.f);
        s_stat[warp][1][c] = make_float4(mp[1], mt[1], lt[1], 0.f);
      }
      __syncthreads();
      if (in && sub == 0 && sp > 1) {
        float4 s[8][2], u[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int w = min(warp + x, 7);
          s[x][0] = x < sp ? s_stat[w][0][c] : none;
          s[x][1] = x < sp ? s_stat[w][1][c] : none;
          u[x] = x < sp ? s_sum[w][lane] : zero;
        }
        add(s, u, std::integral_constant<int, 8>());
      }
      __syncthreads();
    }
    if (in && sub == 0) {
      const int head = me.z / P.groups, group = me.z - head * P.groups;
      const int h0 = head * P.G + group * NQ, rows = min(NQ, P.G - group * NQ);
      float fin[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mb = mt[x] == -INFINITY ? 0.f : mt[x], pb = mp[x] == -INFINITY ? 0.f : mp[x];
        fin[x] = lt[x] == 0.f ? 0.f : exp2f(pb - mb - (E4M3 ? 14.f : 0.f)) / lt[x];
        if (P.lse && m == 0 && g == 0 && r0 + x < rows)
          P.lse[static_cast<size_t>(me.w) * P.Hq + h0 + r0 + x] = lt[x] == 0.f ? -INFINITY : (mb + log2f(lt[x])) * kLn2;
      }
      uint16_t *op = P.out + (static_cast<size_t>(me.w) * P.Hq + h0 + r0) * D + quad_dim<D, E4M3>(m, g);
      store_row2(op, fin[0], v.x, v.z, r0 < rows);
      store_row2(op + D, fin[1], v.y, v.w, r0 + 1 < rows);
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
  p.stat = slots * sizeof(int4);
  p.part = p.stat + slots * 8 * p.NT * sizeof(float4);
  p.bytes = p.part + slots * p.quads * 32 * sizeof(float4);
  return p;
}

template <int D, bool E4M3, int NT, int W, bool DIRECT>
cudaError_t start(const AdParams &P, long long blocks, cudaStream_t st) {
  using S = AdShape<D, E4M3, NT, W>;
  static bool attr = false;
  if (!attr) {
    const cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, NT, W, DIRECT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    attr = true;
  }
  return launch_pdl(attn_decode_kernel<D, E4M3, NT, W, DIRECT>, dim3(static_cast<unsigned>(blocks)), dim3(W * 32), S::SMEM,
                    st, P);
}

template <int D, bool E4M3, int NT>
int launch_attn(const AdParams &P, cudaStream_t st) {
  using S = AdShape<D, E4M3, NT, 4>;
  const long long items = static_cast<long long>(P.B) * P.heads * P.groups;
  const int visible = P.max_pages << P.page_shift;  // most tokens an item can have
  const int tokens = P.window > 0 && P.window < visible ? P.window + kRun - 1 : visible;
  if constexpr (S::ROWB <= 256) {  // (beyond, the stages of eight warps do not fit)
    if (items <= sm_count() && tokens <= kWideTokens)
      return start<D, E4M3, NT, 8, true>(P, items, st) == cudaSuccess ? 0 : -1;
  }
  if (tokens <= kDirectTokens && items < (1LL << 31)) return start<D, E4M3, NT, 4, true>(P, items, st) == cudaSuccess ? 0 : -1;
  long long blocks = static_cast<long long>(sm_count()) * S::BLOCKS;
  if (blocks > kAdMostBlocks) blocks = kAdMostBlocks;
  const long long most = (items * ((tokens + S::UNIT - 1) / S::UNIT * S::UNIT) + kMinTokens - 1) / kMinTokens;
  if (blocks > most) blocks = most;
  if (start<D, E4M3, NT, 4, false>(P, blocks, st) != cudaSuccess) return -1;
  return launch_pdl(attn_join_kernel<D, E4M3, NT>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, P) == cudaSuccess
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
