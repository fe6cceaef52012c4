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
//    share it); a unit is 64 to 256 of its tokens (8 warps: twice that).  All items' units form one line, cut into
//    equal pieces, one per block: blocks end together however uneven the lengths are,
//    and one long sequence fills the GPU.  An item's end costs a block about as much as 1.5 or 3 units
//    (fitted to the blocks' end times), so it takes that much of the line: 64 sequences of 256 to 16384
//    tokens took 124.6 us with a weight of 0.25 and 110.9 us with 1.5; 64 of 125 to 8000 tokens with 16 query heads
//    a key 88.4 us with 1.5 and 74.2 with 3.  Lengths are read on the
//    device, so a captured graph follows them.  A piece covers the end of one item, some
//    whole items and the start of another; only the cut ones leave partial sums in the
//    workspace, at most two a block, which attn_join_kernel adds in order.
//  * Short ones.  The line costs 7 to 10 us whatever the work.  The host does not know the lengths, only the most
//    that the table's width (and the window) allows: a sequence of 37 tokens takes 3.2 us in a table of 64
//    places, 4.0 in one of up to 2048 and 6.9, on the line, in a wider one (96 heads, E4M3).  Where no item can see more than
//    kDirectTokens, a block takes one item and nothing is cut or joined (256 sequences of 900 tokens:
//    80.9 us against 95.5).  Where items are short and more than such blocks fit the GPU at once, a block is
//    one warp, eight to an SM: most of the time is starting and ending items, which then overlap, and no
//    warps are joined.  kOneWarp is where that stops paying (64 query and 8 key-value heads of 128, E4M3,
//    128 sequences of 60 tokens: 11.0 us with four warps, 9.4 with one; 250: 20.2 and 18.2, but 100 of up to
//    250 with 96 heads 15.6 and 17.8; 256 of 1000: 87.6 and 111.3, since a warp has two steps in flight at
//    most).  At rows of 512 bytes, where an SM holds one block of four warps, it pays twice as long (80
//    sequences of 250 tokens, 64 heads on 8 of 256 in bf16: 39.9 and 30.7).  Where there are no more items
//    than SMs, blocks of eight warps (rows of 512 bytes: four) take an item each, or a cluster of 2, 4 or 8 of
//    them shares it evenly and joins its sums through
//    distributed shared memory, up to kPartBytes of keys a block (E4M3, 8 heads: 4000 tokens of one
//    sequence 7.4 us against 11.0 on the line, 16000 14.9 against 15.2, 40000 27.9 against 23.3; 8
//    sequences of 3000 14.4 against 18.1; 2 of 2000, 32 heads on 4 of 256 in bf16, 9.0 against 13.0; one of
//    200, 64 on 8 of 256, 5.9 in clusters of 4 and 7.1 without).
//  * More than 8 query heads a key.  16 of them share an item (NT = 2), so that the cache is read once.  Where
//    the call is so short that a warp's own chain of instructions is what takes the time, each 8 take an
//    item of their own and read the keys again through L2: 128 heads on 8, E4M3, one sequence of 60 tokens
//    5.2 against 3.6 us, of 1000 8.6 and 6.6; 25 sequences of 250 8.8 and 7.2.  That holds as long as the
//    twice as many items run at once; past kDirectTokens only if their clusters are no smaller (64 heads on 4 of
//    256, bf16, 4000 tokens: 16.8 and 12.4; 30 sequences of 3000, 16 heads on one of 64, bf16: 8.7 and 10.0), and
//    where 16 heads' items would each have an SM but 8 heads' would not, up to kSplitTokens (15 sequences of
//    250, 128 heads on 8 of 128: 7.6 and 6.9, of 1000 13.1 and 15.7).
//  * Loads.  Each warp streams every fourth (eighth) run of 16 RR tokens through a ring
//    of its own in shared memory with 16-byte cp.async (stages - 1 runs ahead, across items),
//    so no warp waits for another except where an item ends.  16 tokens from a multiple of
//    16 on never straddle a page (pages hold a multiple of 16 places); the next run's page
//    numbers are loaded a step ahead.  Places not seen are filled with zeros by the copy, so
//    that nothing they hold (NaN, infinities) reaches a product.  Where an item ends the
//    warps exchange their sums through the stages they have just used.
//  * Products.  mma.sync m16n8k16 (f16 or bf16, fp32 sums): with at most 16 query heads
//    sharing a key the products are a small part of the time even at this instruction's
//    rate (1024 multiply-adds a clock and SM, measured), and its operands come straight
//    from registers, where E4M3 codes are converted.  S^T = K Q^T has 16 tokens as rows and
//    8 query heads as columns, O^T = V^T P^T 16 dimensions and the same columns, so that a
//    lane scales the sums of the heads whose maxima it holds; movmatrix turns S^T's registers
//    into P^T's.  The order of dimensions and tokens inside a product is free as long as both
//    operands agree, and is chosen so that a lane's share of K and V is whole 16-byte words.
//  * E4M3.  Codes are converted to f16 (exact; the E4M3 form of mma.sync does the same within,
//    for both operands of every product: 100 instructions for 16 tokens' scores).  A query
//    row is scaled by a power of two to a maximum in [2^14, 2^15), exact but for values below
//    2^-28 of it.  K's scale multiplies the score.  V's scale 2^e joins the weight: w_i =
//    exp2(s_i + e_i - m') with its own running maximum m' of s_i + e_i, times 2^14, rounded to
//    f16 (11 bits down to 2^-28 of the largest, so that a token with a large score and a tiny
//    value costs the others nothing), while l sums exp2(s_i - m) in fp32 with m = max s_i.
//  * bf16.  Q, K and V enter as they are.  Both operands of a product are of one type, and bf16's 8 bits are too few for
//    a weight (the output's error grew from 0.00166 to 0.00188 of its size): it enters as two bf16 numbers, rounded
//    and what the rounding left, in a product each, 16 bits together.  That costs 0 to 1 % where the cache's bytes
//    are the time, and 1 to 4 % of a short call (96 heads, 1.51 GB: 232.4 and 234.0 us; window of 1000: 6.7 and 6.9).
//    E4M3's f16 weights stay in one part: their 11 bits add less than 1 % to the error of the output's own rounding.
//
// Measured (GB300, of 6787 GB/s copy; one GPU and the next differ by 2 %): 32 sequences of 63 to 4001 tokens, 96
// heads of 128, bf16 (1.51 GB): 232 us, 6.5 TB/s; 64 sequences of 256 to 16384 tokens, 64 query and 8 key-value
// heads, E4M3 (668 MB): 111 us, 6.0 TB/s; one of 131072 tokens (271 MB): 51 us, of which 8 are the start, the
// last blocks and the join; 37 tokens of 96 heads: 3.2 us.
#include <cuda_fp16.h>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"
#include "per_device.h"
#include "tc_sm103.cuh"

namespace k3moe {

namespace {

constexpr int kRun = 16;                 // tokens of a product
constexpr int kDirectTokens = 1024;      // items that see at most this many are never cut
constexpr int kSplitTokens = 256;        // (see "More than 8 query heads" above)
constexpr long long kPartBytes = 256 << 10;  // most bytes of keys that one of eight-warp blocks takes
constexpr int kMinTokens = 256;          // smallest piece of a block
constexpr int kUnitLen = 4;              // length of a unit on the line
constexpr int kJoinWarps = 8, kJoinParts = 4;  // warps of a joining block, parts that one adds at once
constexpr int kAdMostBlocks = 152 * 2;   // pieces (bounds the workspace)
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

// An 8 x 8 matrix of 16-bit values, row g in lanes 4g .. 4g + 3 (two values each), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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
template <int RUN>
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
  s.t0 = s.lo & ~(RUN - 1);
  return s;
}
template <int UNIT>
__device__ __forceinline__ int units_of(const Seen &s) {
  return static_cast<int>((static_cast<unsigned>(s.n - s.t0) + (UNIT - 1)) / UNIT);
}

// A block's piece [from, to) of the line, and where one warp is in it.  An item that begins at
// `begin` lies on the line as ITEM_LEN, then kUnitLen for each of its units; a unit belongs
// to the piece in which it begins.
template <int RUN, int UNIT, int ITEM_LEN>
struct Walk {
  int b, head, group;    // sequence, key-value head, which of its items
  int n, lo, t0;
  unsigned tok, stop;    // the warp's next run begins at tok; the piece holds the item's runs below stop
  long long begin;       // of the item
  bool more;             // whether a run is left
  __device__ __forceinline__ int units() const { return units_of<UNIT>({n, lo, t0}); }
  // The item's first unit at or past place x of the line.
  __device__ __forceinline__ int unit_at(long long x) const {
    const long long u = (x - begin - ITEM_LEN + kUnitLen - 1) / kUnitLen;
    return u < 0 ? 0 : u > units() ? units() : static_cast<int>(u);
  }
  // Begins the item at `begin`, from its first unit in [from, to) on; first: the warp's place in a unit.
  __device__ __forceinline__ void enter(long long from, long long to, int first) {
    tok = static_cast<unsigned>(t0) + static_cast<unsigned>(unit_at(from)) * UNIT + first;
    stop = static_cast<unsigned>(t0) + static_cast<unsigned>(unit_at(to)) * UNIT + first;
  }
  __device__ __forceinline__ void set(const Seen &s) { n = s.n, lo = s.lo, t0 = s.t0; }
  __device__ __forceinline__ void next_item(const AdParams &P, long long from, long long to, int first) {
    begin += static_cast<long long>(units()) * kUnitLen + ITEM_LEN;
    more = begin + ITEM_LEN < to;
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
          s = seen_of<RUN>(P, b, false);
        } while (s.n <= s.t0);
        set(s);
      }
    }
    enter(from, to, first);
  }
};

// Warps of a block where there are few items (rows of 512 bytes: the stages of eight do not fit)
template <int D, bool E4M3>
constexpr int kFewWarps = D * (E4M3 ? 1 : 2) <= 256 ? 8 : 4;

template <int D, bool E4M3, int NT, int W, bool DIRECT>
struct AdShape {
  static constexpr int ESZ = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;            // bytes of a cached vector
  static constexpr int C = ROWB / 16;             // 16-byte words of it
  static constexpr int KB = kRun * ROWB;          // bytes of 16 tokens' keys
  static constexpr int MM = D / 16;               // products (16 dimensions each) of 16 tokens and 8 query heads
  static constexpr int QUADS = MM * NT;           // accumulator quads per lane
  // What an item's end costs, on the line: 1.5 units, or 3 where there is more to join
  static constexpr int ITEM_LEN = QUADS <= 8 ? 6 : 12;
  // A warp's step is RR times 16 tokens: 8 KB (16 KB at rows of 512 bytes), so that what a step costs besides its
  // bytes counts little
  static constexpr int RR = ROWB <= 64 ? 4 : ROWB <= 128 ? 2 : 1;
  static constexpr int RUN = RR * kRun;
  static constexpr int UNIT = RUN * W;            // tokens of a block's step
  static constexpr int SUB = 2 * KB;              // keys and values of 16 tokens; a multiple of 128: words swizzle by xor
  static constexpr int SCALES = E4M3 ? 32 : 0;    // scale bytes of 16 tokens, after all stages
  // Stages and blocks per SM: 8 warps (three blocks: 12; rows of 512 bytes: 4) with 64 to 128 KB of loads in flight per
  // SM.  Blocks of one item each spend more of their time starting and ending, which a third block covers (256
  // sequences of 1000 tokens, 128 heads on 8, E4M3: 122.8 us with two, 104.3 with three); on the line it costs more in
  // spilled registers and shorter rings than it brings (32 of 8000, 128 heads on 8, bf16: 172 and 178)
  static constexpr bool THREE = DIRECT && W == 4 && ROWB <= 256 && (NT == 1 || D <= 128);
  static constexpr int STAGES = THREE || W == 1 ? 2 : 3;
  static constexpr int BLOCKS = W == 1 ? (ROWB <= 256 ? 8 : 4) : THREE ? 3 : ROWB <= 256 && W == 4 ? 2 : 1;
  // quads that the warps exchange at once where an item ends, each in the stage it has just used
  static constexpr int QR = RR * SUB / 512 < QUADS ? RR * SUB / 512 : QUADS;
  // query fragments: in registers, or from 32 of them on in shared memory (the same for all warps)
  static constexpr int QREGS = D / 16 * 2 * NT;
  static constexpr int QSMEM = QREGS >= 32 ? QREGS * 32 * 4 : 0;
  // what a cluster's blocks show one another: their sums and statistics
  static constexpr bool CLUSTER = DIRECT && W == kFewWarps<D, E4M3>;
  static constexpr int SHOWN = CLUSTER ? QUADS * 512 + 8 * NT * 16 : 0;
  static constexpr int SMEM = W * STAGES * RR * (SUB + SCALES) + QSMEM + SHOWN + 128;
};

// First of the two neighbouring dimensions that a lane of group g holds of product m.
template <int D, bool E4M3>
__device__ __forceinline__ int quad_dim(int m, int g) {
  constexpr int PER = E4M3 ? 16 : 8;  // dimensions of a 16-byte word
  const int dl = 2 * m;               // of the lane's dimensions
  return D / PER >= 8 ? (g + 8 * (dl / PER)) * PER + dl % PER : g * 8 + dl;
}

// Two neighbouring dimensions of a row, times f and up; zeros for a row without weight, whatever the sums are.
__device__ __forceinline__ void store_row2(uint16_t *p, float f, float up, float a, float b, bool weight, bool on) {
  if (on) *reinterpret_cast<uint32_t *>(p) = weight ? pack2<false>(a * f * up, b * f * up) : 0u;
}

// Adds N parts of a quad: statistics s (m', m, l) of this lane's two rows, sums u at m'.
template <int N>
__device__ __forceinline__ void add_parts(const float4 (&s)[N][2], const float4 (&u)[N], float4 &v, float (&mp)[2],
                                          float (&mt)[2], float (&lt)[2]) {
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float np = -INFINITY, nt = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) np = fmaxf(np, s[i][x].x), nt = fmaxf(nt, s[i][x].y);
    const float pb = np == -INFINITY ? 0.f : np, mb = nt == -INFINITY ? 0.f : nt;
    float a = 0.f, b = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float f = ex2(s[i][x].x - pb);
      a = fmaf(x ? u[i].y : u[i].x, f, a);
      b = fmaf(x ? u[i].w : u[i].z, f, b);
      sum = fmaf(s[i][x].z, ex2(s[i][x].y - mb), sum);
    }
    (x ? v.y : v.x) = a;
    (x ? v.w : v.z) = b;
    mp[x] = np, mt[x] = nt, lt[x] = sum;
  }
}

// Writes a quad of rows that are complete: out = (O' 2^-14 / l) 2^(m' - m), and with the first quad lse.  m' - m is -127
// to 127, as V's scales are, so that one factor of both would leave fp32's normal numbers where V is tiny (but for
// the rounding of sums past 2^24, which must not make it infinite).
template <int D, bool E4M3>
__device__ __forceinline__ void store_quad(const AdParams &P, int b, int h0, int rows, int t, int m, const float4 &v,
                                           const float (&mp)[2], const float (&mt)[2], const float (&lt)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, r0 = 8 * t + 2 * (lane & 3);
  float fin[2], up[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    // (no m' beside an m: every value is NaN, and so are the sums)
    const float mb = mt[x] == -INFINITY ? 0.f : mt[x], pb = mp[x] == -INFINITY ? mb : mp[x];
    fin[x] = __fdividef(E4M3 ? 0x1p-14f : 1.f, lt[x]);
    up[x] = E4M3 ? exp2f(fminf(pb - mb, 127.f)) : 1.f;
    if (P.lse && m == 0 && g == 0 && r0 + x < rows)
      P.lse[static_cast<size_t>(b) * P.Hq + h0 + r0 + x] = lt[x] == 0.f ? -INFINITY : (mb + log2f(lt[x])) * kLn2;
  }
  uint16_t *op = P.out + (static_cast<size_t>(b) * P.Hq + h0 + r0) * D + quad_dim<D, E4M3>(m, g);
  store_row2(op, fin[0], up[0], v.x, v.z, lt[0] != 0.f, r0 < rows);
  store_row2(op + D, fin[1], up[1], v.y, v.w, lt[1] != 0.f, r0 + 1 < rows);
}

// ---- thread-block clusters
__device__ __forceinline__ int cluster_size() {
  int n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Sixteen bytes at shared address a of the cluster's block `rank`.
__device__ __forceinline__ float4 lds_of(uint32_t a, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(a), "r"(rank)
      : "memory");
  return v;
}

}  // namespace

template <int D, bool E4M3, int NT, int W, bool DIRECT>
__global__ void __launch_bounds__(W * 32, (AdShape<D, E4M3, NT, W, DIRECT>::BLOCKS))
    attn_decode_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT, W, DIRECT>;
  constexpr int THREADS = W * 32;
  constexpr int C = S::C, MM = S::MM, ST = S::STAGES, RR = S::RR, RUN = S::RUN, UNIT = S::UNIT, NQ = 8 * NT;
  constexpr int KL = C / 4;             // words of a key a lane reads
  constexpr int SP = E4M3 ? 4 : 2;      // products of 16 dimensions per such word
  constexpr int VL = C >= 8 ? C / 8 : 1;  // words of a value a lane reads
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((128u - (su32(smem_raw) & 127u)) & 127u);
  __shared__ __align__(16) float s_mp[NQ][W], s_m[NQ][W], s_l[NQ][W];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int items = P.heads * P.groups, first = warp * RUN;
  // hints only: nothing of these is read before the wait
  if (tid < (P.B + 31) / 32) prefetch_l2(P.lens + 32 * tid);
  pdl_wait();
  pdl_trigger();

  auto zero_rows = [&]() {  // of the sequences that see nothing; every block takes its share
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      const Seen s = seen_of<RUN>(P, b, false);
      if (s.n > s.t0) continue;
      for (size_t i = tid; i < static_cast<size_t>(P.Hq) * D / 8; i += THREADS)
        reinterpret_cast<uint4 *>(P.out + static_cast<size_t>(b) * P.Hq * D)[i] = make_uint4(0, 0, 0, 0);
      if (P.lse)
        for (int i = tid; i < P.Hq; i += THREADS) P.lse[static_cast<size_t>(b) * P.Hq + i] = -INFINITY;
    }
  };

  // ---- this block's piece
  Walk<RUN, UNIT, S::ITEM_LEN> cur;
  int part = 0, parts = 1;  // of an item that a cluster's blocks share
  long long from = 0, to = 1LL << 62, share = 0;
  if constexpr (DIRECT) {
    if constexpr (S::CLUSTER) parts = cluster_size(), part = cluster_rank();
    const int block = blockIdx.x / parts;
    cur.b = block / items;
    const int item = block - cur.b * items;
    cur.head = item / P.groups;
    cur.group = item - cur.head * P.groups;
    cur.set(seen_of<RUN>(P, cur.b, tid == 0));
    cur.begin = 0;
    cur.more = true;
    if (cur.n <= cur.t0) {  // sees nothing
      if (part) return;
      const int h0 = cur.head * P.G + cur.group * NQ;
      const int rows = min(NQ, P.G - cur.group * NQ);
      const size_t row = static_cast<size_t>(cur.b) * P.Hq + h0;
      for (int i = tid; i < rows * D / 8; i += THREADS)
        reinterpret_cast<uint4 *>(P.out + row * D)[i] = make_uint4(0, 0, 0, 0);
      if (P.lse && tid < rows) P.lse[row + tid] = -INFINITY;
      return;
    }
    const unsigned units = cur.units(), base = static_cast<unsigned>(cur.t0) + first;
    cur.tok = base + units * part / parts * UNIT;
    cur.stop = base + units * (part + 1) / parts * UNIT;
    cur.more = cur.tok < cur.stop;  // (a part may be left without a unit)
  } else {
    // every warp for itself: lane l measures sequences [l per, l per + per); a scan finds the piece
    const int per = (P.B + 31) / 32;
    const int b0 = min(P.B, lane * per), b1 = min(P.B, b0 + per);
    auto length = [&](int b, bool report) {  // of an item of sequence b on the line
      const int u = units_of<UNIT>(seen_of<RUN>(P, b, report));
      return u ? static_cast<long long>(u) * kUnitLen + S::ITEM_LEN : 0LL;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += length(b, blockIdx.x == 0 && warp == 0);
    mine *= items;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    const long long total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    share = max(static_cast<long long>(kMinTokens / UNIT * kUnitLen), div_small(total + gridDim.x - 1, gridDim.x));
    from = static_cast<long long>(blockIdx.x) * share;
    to = min(total, from + share);
    const bool here = from < to && from >= incl - mine && from < incl;  // in this lane's sequences
    int at_b = b0, at_item = 0;
    long long at = incl - mine;
    if (here) {
      long long len;
      for (;; ++at_b) {
        len = length(at_b, false);
        if (from < at + len * items) break;
        at += len * items;
      }
      at_item = static_cast<int>(div_small(from - at, len));
      at += at_item * len;
    }
    if (tid < 2) P.meta[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
    if (from >= to) {
      zero_rows();
      return;
    }
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
    cur.b = __shfl_sync(0xFFFFFFFFu, at_b, src);
    at_item = __shfl_sync(0xFFFFFFFFu, at_item, src);
    cur.head = at_item / P.groups;
    cur.group = at_item - cur.head * P.groups;
    cur.set(seen_of<RUN>(P, cur.b, false));
    cur.begin = __shfl_sync(0xFFFFFFFFu, at, src);
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
  Walk<RUN, UNIT, S::ITEM_LEN> pre = cur;
  uint32_t bad = 0;    // bit st RR + r: 16 tokens that were not loaded: before the window, or a page outside the cache
  // a run starts at a multiple of RUN and lies in one page if pages are no smaller
  const bool one_page = (RUN - 1u) <= place;
  int page[RR];
  const int32_t *row;  // of the table
  auto new_item = [&]() { row = P.table + static_cast<size_t>(pre.b) * P.max_pages; };
  auto pages = [&]() {  // of the run at `pre`
#pragma unroll
    for (int r = 0; r < RR; ++r) {
      const unsigned tok = pre.tok + r * kRun;
      // a run that lies in one page begins at most RUN - 1 places before the window, and needs that page.  Tiles that
      // lie in pages of their own may all be before it: those pages may have been given back, and are not looked up
      const bool seen = tok < static_cast<unsigned>(pre.n) && (one_page || tok + kRun > static_cast<unsigned>(pre.lo));
      if (r == 0 || !one_page) page[r] = seen ? row[tok >> P.page_shift] : -1;
    }
  };
  auto issue = [&](int st) {
    if (pre.more) {
      const uint32_t kd = ring + st * RR * S::SUB + kdst, vd = ring + st * RR * S::SUB + vdst;
      const uint32_t sd = sring + st * RR * S::SCALES;
      auto vec_of = [&](int page, unsigned tok) {
        return static_cast<size_t>(static_cast<unsigned>(page)) * page_vecs +
               ((static_cast<unsigned>(pre.head) << P.page_shift) + (tok & place));
      };
      if (one_page && pre.tok >= static_cast<unsigned>(pre.lo) && pre.tok + RUN <= static_cast<unsigned>(pre.n) &&
          static_cast<unsigned>(page[0]) < static_cast<unsigned>(P.pages)) {  // all of it is seen
        if (bad) bad &= ~(((1u << RR) - 1u) << (st * RR));
        const size_t vec = vec_of(page[0], pre.tok);
        const uint8_t *kp = klane + vec * S::ROWB, *vp = vlane + vec * S::ROWB;
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
          for (int i = 0; i < C / 2; ++i) {
            // the part of the swizzles that varies with i
            const uint32_t ki = C == 32 ? (i & 1) << 6 : 0, vi = C >= 8 ? ((i * RI) >> 2) << 5 : 0;
            cp16((kd ^ ki) + r * S::SUB + i * RI * S::ROWB, kp + r * S::KB + i * 512);
            cp16((vd ^ vi) + r * S::SUB + i * RI * S::ROWB, vp + r * S::KB + i * 512);
          }
        if (E4M3 && lane < 2 * RR)
          cp16(sd + (lane >> 1) * S::SCALES + 16 * (lane & 1), (lane & 1 ? P.vs : P.ks) + vec + 16 * (lane >> 1));
      } else {
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          const unsigned tok = pre.tok + r * kRun;
          const int tile = st * RR + r, pg = one_page ? page[0] : page[r];
          if (tok >= static_cast<unsigned>(pre.n)) break;
          if (tok + kRun <= static_cast<unsigned>(pre.lo)) {
            bad |= 1u << tile;
            continue;
          }
          if (static_cast<unsigned>(pg) >= static_cast<unsigned>(P.pages)) {
            bad |= 1u << tile;
            if (lane == 0) set_status(P.status, K3MOE_DEV_BOUNDS);
            continue;
          }
          bad &= ~(1u << tile);
          const size_t vec = vec_of(pg, tok);
          const uint8_t *kp = klane + vec * S::ROWB, *vp = vlane + vec * S::ROWB;
#pragma unroll
          for (int i = 0; i < C / 2; ++i) {
            const uint32_t ki = C == 32 ? (i & 1) << 6 : 0, vi = C >= 8 ? ((i * RI) >> 2) << 5 : 0;
            const unsigned at = tok + lr + i * RI;
            const bool on = at >= static_cast<unsigned>(pre.lo) && at < static_cast<unsigned>(pre.n);
            cp16_or_zeros((kd ^ ki) + r * S::SUB + i * RI * S::ROWB, kp + i * 512, on);
            cp16_or_zeros((vd ^ vi) + r * S::SUB + i * RI * S::ROWB, vp + i * 512, on);
          }
          if (E4M3 && lane < 2) cp16(sd + r * S::SCALES + 16 * lane, (lane ? P.vs : P.ks) + vec);
        }
      }
      pre.tok += UNIT;
      if (pre.tok >= pre.stop) {
        if (DIRECT) {
          pre.more = false;
        } else {
          pre.next_item(P, from, to, first);
          new_item();
        }
      }
      if (pre.more) pages();
    }
    cp_commit();
  };
  new_item();
  if (pre.more) pages();
#pragma unroll
  for (int st = 0; st < ST - 1; ++st) issue(st);

  constexpr int QN = D / 16, QW = 2 * NT;  // products along the dimensions, registers of the query rows in each
  constexpr bool QS = S::QSMEM > 0;
  uint32_t qf[QS ? 1 : QN][QW];
  uint4 *const q_sm = reinterpret_cast<uint4 *>(smem + W * ST * RR * (S::SUB + S::SCALES));
  float4 *const shown = reinterpret_cast<float4 *>(smem + W * ST * RR * (S::SUB + S::SCALES) + S::QSMEM);
  float4 *const shown_stat = shown + S::QUADS * 32;  // (CLUSTER)
  uint2 raw[D / 16][NT];
  // of query heads 8 t + 2c + x: the scale of a raw score (in powers of two), the running maxima and l
  float sq[NT][2], o[NT][MM][4], mrun[NT][2], m_l[NT][2], l[NT][2];
  auto load_q = [&](const Walk<RUN, UNIT, S::ITEM_LEN> &at) {
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
              r < rows ? *reinterpret_cast<const uint2 *>(qp + i * (64 / S::ESZ) + 4 * w) : make_uint2(0, 0);
    }
  };
  auto start_item = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float up = 1.f, mine = P.scale * kLog2e;  // of row 8 t + g
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
        mine *= mx_pow2(-e);
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
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sq[t][x] = E4M3 ? __shfl_sync(0xFFFFFFFFu, mine, 8 * c + 4 * x) : mine;
        mrun[t][x] = m_l[t][x] = -INFINITY;
        l[t][x] = 0.f;
      }
#pragma unroll
      for (int m = 0; m < MM; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][m][x] = 0.f;
    }
  };

  constexpr bool kEarlyQ = D / 16 * NT <= (E4M3 && NT == 2 ? 8 : 16);  // as far as there are registers for it
  bool first_item = true;
  int stage = 0, after = ST - 1;  // the stage in use, and the one that is loaded next
  load_q(cur);
  start_item();
  if (QS) __syncthreads();
  while (cur.more) {
    __syncwarp();  // every lane is done with the stage that is loaded next
    issue(after);
    after = after + 1 == ST ? 0 : after + 1;
    cp_wait<ST - 1>();
    __syncwarp();
    if (cur.tok < static_cast<unsigned>(cur.n)) {
      const uint32_t base0 = ring + stage * (RR * S::SUB), sbase = sring + stage * (RR * S::SCALES);
      const bool whole = cur.tok >= static_cast<unsigned>(cur.lo) &&
                         cur.tok + S::RUN <= static_cast<unsigned>(cur.n) && bad == 0u;
      // S^T: rows g and g + 8 are tokens tg and tg + 2 of the 16, tg = 4 (g / 2) + g % 2, columns 2c and
      // 2c + 1 query heads.  CH partial sums, so that a product does not wait for the one before it
      constexpr int CH = RR * NT >= 4 ? 1 : 2, T2 = 2 * RR;
      float s[RR][NT][CH][4];
      const int tg = 4 * (g >> 1) + (g & 1);
      const uint32_t kofs = tg * S::ROWB + (c << 4) + (C >= 8 ? (g & 1) << 6 : 0);
#pragma unroll
      for (int i = 0; i < KL; ++i) {
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          uint4 kw[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kw[j] = lds128(((base0 + r * S::SUB + kofs) ^ ((i & 1) << 6)) + (i >> 1) * 128 + 2 * j * S::ROWB);
          const uint32_t k0[4] = {kw[0].x, kw[0].y, kw[0].z, kw[0].w}, k1[4] = {kw[1].x, kw[1].y, kw[1].z, kw[1].w};
#pragma unroll
          for (int w = 0; w < SP; ++w) {
            const int qi = i * SP + w;
            uint32_t b[QW], a0, a1, a2, a3;
            if constexpr (QS) {
              if constexpr (NT == 1)
                *reinterpret_cast<uint2 *>(b) = reinterpret_cast<const uint2 *>(&q_sm[(qi / 2) * 32 + lane])[qi & 1];
              else
                *reinterpret_cast<uint4 *>(b) = q_sm[qi * 32 + lane];
            } else {
#pragma unroll
              for (int x = 0; x < QW; ++x) b[x] = qf[qi][x];
            }
            if constexpr (E4M3) {
              e4m3x4_to_f16x2(k0[w], a0, a2);
              e4m3x4_to_f16x2(k1[w], a1, a3);
            } else {
              a0 = k0[2 * w], a1 = k1[2 * w], a2 = k0[2 * w + 1], a3 = k1[2 * w + 1];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (qi < CH)
                mma16_first<E4M3>(s[r][t][qi], a0, a1, a2, a3, b[t], b[NT + t]);
              else
                mma16<E4M3>(s[r][t][qi & (CH - 1)], a0, a1, a2, a3, b[t], b[NT + t]);
            }
          }
        }
      }
      // weights of tokens tg and tg + 2 of each 16, in powers of two
      float kx[T2], ve[T2];
      if constexpr (E4M3) {
        uint32_t kw[RR], vw[RR], odd = 0;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          kw[r] = lds32(sbase + r * S::SCALES + 4 * (g >> 1)) >> (8 * (g & 1));
          vw[r] = lds32(sbase + r * S::SCALES + 16 + 4 * (g >> 1)) >> (8 * (g & 1));
          odd |= byte_255(kw[r]) | byte_255(vw[r]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // byte 2h << 23 (0 stands for 2^-127), and byte 2h - 127
            kx[2 * r + h] = fmaxf(__uint_as_float(__byte_perm(kw[r], 0u, 0x0444 | ((2 * h) << 12)) >> 1),
                                  __uint_as_float(0x00400000u));
            ve[2 * r + h] = __uint_as_float(__byte_perm(vw[r], 0x4B000000u, 0x7440 | (2 * h))) - 8388735.0f;
          }
        }
        if (odd) {  // NaN
#pragma unroll
          for (int j = 0; j < T2; ++j) {
            if (((kw[j >> 1] >> (16 * (j & 1))) & 255u) == 255u) kx[j] = __uint_as_float(0x7FC00000u);
            if (((vw[j >> 1] >> (16 * (j & 1))) & 255u) == 255u) ve[j] = __uint_as_float(0x7FC00000u);
          }
        }
      }
      float sc[NT][2][T2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < T2; ++j) {
            const int at = 2 * (j & 1) + x;
            float raw_s = s[j >> 1][t][0][at];
            if constexpr (CH == 2) raw_s += s[j >> 1][t][CH - 1][at];
            sc[t][x][j] = raw_s * (E4M3 ? sq[t][x] * kx[j] : sq[t][x]);
          }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < T2; ++j) {
          const unsigned tok = cur.tok + (j >> 1) * kRun + tg + 2 * (j & 1);
          if (tok < static_cast<unsigned>(cur.lo) || tok >= static_cast<unsigned>(cur.n) ||
              ((bad >> (stage * RR + (j >> 1))) & 1u)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][0][j] = sc[t][1][j] = -INFINITY;
            if (E4M3) ve[j] = 0.f;
          }
        }
      }
      float top[NT][2];
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (E4M3) {  // l and its maximum, of this lane's tokens alone
            float mn = m_l[t][x], add = 0.f;
#pragma unroll
            for (int j = 0; j < T2; ++j) mn = fmaxf(mn, sc[t][x][j]);
            const float base = mn == -INFINITY ? 0.f : mn;
#pragma unroll
            for (int j = 0; j < T2; j += 2) add += ex2(sc[t][x][j] - base) + ex2(sc[t][x][j + 1] - base);
            l[t][x] = l[t][x] * ex2(m_l[t][x] - base) + add;
            m_l[t][x] = mn;
#pragma unroll
            for (int j = 0; j < T2; ++j) sc[t][x][j] += ve[j];
          }
          top[t][x] = sc[t][x][0];
#pragma unroll
          for (int j = 1; j < T2; ++j) top[t][x] = fmaxf(top[t][x], sc[t][x][j]);
          grows |= top[t][x] > mrun[t][x];
        }
      if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float al[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xFFFFFFFFu, top[t][x], off));
            const float mn = fmaxf(mrun[t][x], top[t][x]);
            al[x] = mn > mrun[t][x] ? ex2(mrun[t][x] - mn) : 1.f;
            mrun[t][x] = mn;
            if (!E4M3) l[t][x] *= al[x];
          }
#pragma unroll
          for (int m = 0; m < MM; ++m) {
            o[t][m][0] *= al[0];
            o[t][m][1] *= al[1];
            o[t][m][2] *= al[0];
            o[t][m][3] *= al[1];
          }
        }
      }
      // P^T: eight tokens by eight query heads, turned so that a lane has two tokens of one head
      uint32_t pf[RR][NT][2], pl[E4M3 ? 1 : RR][NT][2];  // (bf16: and what the rounding left)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float base[2] = {(mrun[t][0] == -INFINITY ? 0.f : mrun[t][0]) - (E4M3 ? 14.f : 0.f),
                               (mrun[t][1] == -INFINITY ? 0.f : mrun[t][1]) - (E4M3 ? 14.f : 0.f)};
#pragma unroll
        for (int j = 0; j < T2; ++j) {
          const float p0 = ex2(sc[t][0][j] - base[0]), p1 = ex2(sc[t][1][j] - base[1]);
          if (!E4M3) l[t][0] += p0, l[t][1] += p1;
          const uint32_t hi = pack2<E4M3>(p0, p1);
          pf[j >> 1][t][j & 1] = transpose8x8(hi);
          if constexpr (!E4M3)
            pl[j >> 1][t][j & 1] =
                transpose8x8(pack2<false>(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u)));
        }
      }
      // O^T: rows g and g + 8 of product m are this lane's dimensions 2m and 2m + 1.  16 tokens that are
      // not seen at all (past the end, before the window, or of a bad page) were not loaded and are left out
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
              for (int t = 0; t < NT; ++t) {
                mma16<false>(o[t][i * VW + w], a0, a1, a2, a3, pf[r][t][0], pf[r][t][1]);
                mma16<false>(o[t][i * VW + w], a0, a1, a2, a3, pl[r][t][0], pl[r][t][1]);
              }
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
    const Walk<RUN, UNIT, S::ITEM_LEN> done = cur;
    const bool began_before = !DIRECT && done.unit_at(from) > 0, cut = began_before || (!DIRECT && done.unit_at(to) < done.units());
    const int h0 = done.head * P.G + done.group * NQ, rows = min(NQ, P.G - done.group * NQ);
    if (DIRECT)
      cur.more = false;
    else
      cur.next_item(P, from, to, first);
    if (kEarlyQ && cur.more) load_q(cur);  // arrives while the warps join
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float m = E4M3 ? m_l[t][x] : mrun[t][x];
        float mm = m;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, off));
        float lt = mm == -INFINITY ? l[t][x] : l[t][x] * ex2(m - mm);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, off);
        if (g == 0) {
          s_mp[8 * t + 2 * c + x][warp] = mrun[t][x];
          s_m[8 * t + 2 * c + x][warp] = mm;
          s_l[8 * t + 2 * c + x][warp] = lt;
        }
      }
    }
    // quad x of warp w: in the stage that the warp has just used, and loads again only after this
    float4 *buf = reinterpret_cast<float4 *>(smem + used * (RR * S::SUB));
    constexpr int NEXT = ST * RR * S::SUB / 16;  // from one warp's stages to the next's
    const int slot = 2 * blockIdx.x + (first_item ? 0 : 1);
    float fac[2][W], mp[2], mt[2], lt[2];
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
            mp[e] = mt[e] = -INFINITY;
            lt[e] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) mp[e] = fmaxf(mp[e], s_mp[r][w]), mt[e] = fmaxf(mt[e], s_m[r][w]);
            const float mb = mt[e] == -INFINITY ? 0.f : mt[e], pb = mp[e] == -INFINITY ? 0.f : mp[e];
#pragma unroll
            for (int w = 0; w < W; ++w) {
              lt[e] = fmaf(s_l[r][w], ex2(s_m[r][w] - mb), lt[e]);
              fac[e][w] = ex2(s_mp[r][w] - pb);
            }
            if (m == 0 && g == 0) {
              if (cut) P.stat[static_cast<size_t>(slot) * NQ + r] = make_float4(mp[e], mt[e], lt[e], 0.f);
              if (parts > 1) shown_stat[r] = make_float4(mp[e], mt[e], lt[e], 0.f);
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
        if (cut)
          P.part[(static_cast<size_t>(slot) * S::QUADS + quad) * 32 + lane] = v;
        else if (parts > 1)
          shown[quad * 32 + lane] = v;
        else
          store_quad<D, E4M3>(P, done.b, h0, rows, t, m, v, mp, mt, lt);
      }
      __syncthreads();
    }
    if constexpr (!DIRECT) {
      if (tid == 0 && cut) {  // the blocks whose pieces the item covers
        const long long unit0 = done.begin + S::ITEM_LEN;
        const int b0 = static_cast<int>(div_small(unit0, share));
        P.meta[2 * blockIdx.x + (began_before ? 0 : 1)] = make_int4(
            // not the first item of its block if the one before has a unit there
            2 * b0 + (done.begin - kUnitLen >= b0 * share ? 1 : 0),
            static_cast<int>(div_small(unit0 + static_cast<long long>(done.units() - 1) * kUnitLen, share)) - b0 + 1,
            done.head * P.groups + done.group, done.b);
      }
    }
    first_item = false;
    if (!cur.more) break;
    if (!kEarlyQ) load_q(cur);
    start_item();
    if (QS) __syncthreads();
  }
  cp_wait<0>();
  if constexpr (!DIRECT) zero_rows();
  if constexpr (S::CLUSTER) {
    if (parts > 1) {  // join the cluster's blocks: each takes every parts-th quad
      if (first_item) {  // (nothing came of the loop: an empty part)
        for (int i = tid; i < S::QUADS * 32; i += THREADS) shown[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tid < NQ) shown_stat[tid] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
      }
      cluster_sync();
      const int h0 = cur.head * P.G + cur.group * NQ, rows = min(NQ, P.G - cur.group * NQ);
      for (int quad = part + parts * warp; quad < S::QUADS; quad += parts * W) {
        const int t = quad / MM, m = quad - t * MM, r0 = 8 * t + 2 * c;
        float4 s[8][2], u[8], v;
        float mp[2], mt[2], lt[2];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          s[x][0] = s[x][1] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
          u[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x < parts) {
            s[x][0] = lds_of(su32(shown_stat + r0), x);
            s[x][1] = lds_of(su32(shown_stat + r0 + 1), x);
            u[x] = lds_of(su32(shown + quad * 32 + lane), x);
          }
        }
        add_parts(s, u, v, mp, mt, lt);
        store_quad<D, E4M3>(P, cur.b, h0, rows, t, m, v, mp, mt, lt);
      }
      cluster_sync();  // the others have read this block's
    }
  }
}

// Adds the partial sums of the items that were cut, in the order of their pieces.  The
// blocks are those of the kernel before; each takes its share of the accumulator quads
// of the (at most two) cut items that it holds a piece of, so that an item of many pieces
// is joined by many blocks.  A warp adds up to kJoinParts parts of a quad, their
// statistics and sums loaded together; where there are more, warps share a quad.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const AdParams P) {
  using S = AdShape<D, E4M3, NT, 4, false>;
  constexpr int NQ = 8 * NT, QUADS = S::QUADS, MM = S::MM;
  __shared__ float4 s_sum[kJoinWarps][32], s_stat[kJoinWarps][2][4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();
  const int4 m0 = P.meta[2 * blockIdx.x], m1 = P.meta[2 * blockIdx.x + 1];
  // quads of an item that are this block's: mine, mine + parts, ..; warps that share one
  auto count_of = [&](const int4 &m) {
    const int parts = m.y, mine = static_cast<int>(blockIdx.x) - (m.x >> 1);
    return parts > 1 && mine < QUADS ? (QUADS - 1 - mine) / parts + 1 : 0;
  };
  auto split_of = [&](const int4 &m) {
    int s = 1;
#pragma unroll
    for (int w = 1; w < kJoinWarps; w *= 2) s = m.y > w * kJoinParts ? 2 * w : s;
    return s;
  };
  const int n0 = count_of(m0), n1 = count_of(m1), sp0 = split_of(m0), sp1 = split_of(m1);
  // a quad's warps lie in one round of all warps: splits are powers of two, and the second item's
  // tasks start at a multiple of its split
  const int tasks0 = n0 * sp0, from1 = (tasks0 + sp1 - 1) / sp1 * sp1;
  const int tasks = n1 ? from1 + n1 * sp1 : tasks0;
  for (int base = 0; base < tasks; base += kJoinWarps) {
    const bool e = base + warp >= tasks0;
    const int task = base + warp - (e ? from1 : 0);
    const int sp = e ? sp1 : sp0, sub = task & (sp - 1), q = task / sp;
    const bool in = task >= 0 && q < (e ? n1 : n0);
    const int4 me = make_int4(e ? m1.x : m0.x, e ? m1.y : m0.y, e ? m1.z : m0.z, e ? m1.w : m0.w);
    const int parts = me.y, b0 = me.x >> 1, quad = static_cast<int>(blockIdx.x) - b0 + q * parts;
    const int t = quad / MM, m = quad - t * MM, r0 = 8 * t + 2 * c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mp[2], mt[2], lt[2];
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
        add_parts(s, u, v, mp, mt, lt);
      }
    }
    if (max(sp0, sp1) > 1) {  // (uniform: the block's)
      s_sum[warp][lane] = v;
      if (g == 0) {
        s_stat[warp][0][c] = make_float4(mp[0], mt[0], lt[0], 0.f);
        s_stat[warp][1][c] = make_float4(mp[1], mt[1], lt[1], 0.f);
      }
      __syncthreads();
      if (in && sub == 0 && sp > 1) {
        for (int i = 1; i < sp; i += kJoinParts) {
          float4 s[kJoinParts + 1][2], u[kJoinParts + 1];
#pragma unroll
          for (int x = 0; x < kJoinParts; ++x) {
            const bool on = i + x < sp;
            const int w = on ? warp + i + x : warp;
            s[x][0] = on ? s_stat[w][0][c] : none;
            s[x][1] = on ? s_stat[w][1][c] : none;
            u[x] = on ? s_sum[w][lane] : zero;
          }
          s[kJoinParts][0] = make_float4(mp[0], mt[0], lt[0], 0.f);
          s[kJoinParts][1] = make_float4(mp[1], mt[1], lt[1], 0.f);
          u[kJoinParts] = v;
          add_parts(s, u, v, mp, mt, lt);
        }
      }
      __syncthreads();
    }
    if (in && sub == 0) {
      const int head = me.z / P.groups, group = me.z - head * P.groups;
      const int h0 = head * P.G + group * NQ, rows = min(NQ, P.G - group * NQ);
      store_quad<D, E4M3>(P, me.w, h0, rows, t, m, v, mp, mt, lt);
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

int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// A launch of `blocks` blocks in clusters of `cluster`; 0 blocks: only how many clusters fit the GPU at once.
template <int D, bool E4M3, int NT, int W, bool DIRECT>
cudaError_t start(const AdParams &P, long long blocks, int cluster, cudaStream_t st, int *fit = nullptr) {
  using S = AdShape<D, E4M3, NT, W, DIRECT>;
  static PerDevice raised;  // whether the kernel's limit of shared memory is
  cudaError_t err = cudaSuccess;
  raised.get(current_device(), [&] {
    err = cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, NT, W, DIRECT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               S::SMEM);
    return err == cudaSuccess ? 1 : -1;
  });
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks ? blocks : cluster));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (!blocks) {
    cfg.attrs = attrs + 1;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(fit, attn_decode_kernel<D, E4M3, NT, W, DIRECT>, &cfg);
  }
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, E4M3, NT, W, DIRECT>, P);
}

// Clusters of `parts` (2, 4 or 8) eight-warp blocks that run at once: not all SMs, since a cluster
// lies within one group of 16 to 20 of them (128 blocks in clusters of 8 took two rounds, 16.3 us, where
// 64 in clusters of 4 took 10.2).
template <int D, bool E4M3, int NT>
int clusters_at_once(const AdParams &P, int parts) {
  static PerDevice known[9];
  return max(0, known[parts].get(current_device(), [&] {
    int n = 0;
    if (start<D, E4M3, NT, kFewWarps<D, E4M3>, true>(P, 0, parts, nullptr, &n) == cudaSuccess) return n;
    cudaGetLastError();  // leave no error behind
    return -1;
  }));
}

// Items of at most 8 NT query heads, and the most tokens that one can see.
long long items_of(const AdParams &P) { return static_cast<long long>(P.B) * P.heads * P.groups; }
long long tokens_of(const AdParams &P) {
  const long long visible = static_cast<long long>(P.max_pages) << P.page_shift;
  return P.window > 0 && P.window < visible ? P.window : visible;
}

// No more items than SMs: how many blocks share one, 0 where there are more or they are too long for that.
template <int D, bool E4M3, int NT>
int few_parts(const AdParams &P) {
  using S = AdShape<D, E4M3, NT, 4, false>;
  const long long items = items_of(P), tokens = tokens_of(P);
  if (items > sm_count()) return 0;
  int parts = 1;
  constexpr long long kStep = S::RUN * kFewWarps<D, E4M3>;  // tokens that a block takes at once
  if (tokens > 2 * kStep)  // (one more step costs less than a cluster's join up to here)
    while (parts < 8 && tokens > kStep * parts && items <= clusters_at_once<D, E4M3, NT>(P, 2 * parts)) parts *= 2;
  return tokens * S::ROWB <= kPartBytes * parts ? parts : 0;
}

template <int D, bool E4M3, int NT>
int launch_few(const AdParams &P, int parts, cudaStream_t st) {
  using S = AdShape<D, E4M3, NT, 4, false>;
  const long long items = items_of(P);
  const cudaError_t e = tokens_of(P) <= S::UNIT ? start<D, E4M3, NT, 4, true>(P, items, 1, st)
                                                : start<D, E4M3, NT, kFewWarps<D, E4M3>, true>(P, items * parts, parts, st);
  return e == cudaSuccess ? 0 : -1;
}

template <int D, bool E4M3, int NT>
int launch_attn(const AdParams &P, cudaStream_t st) {
  using S = AdShape<D, E4M3, NT, 4, false>;
  const long long items = items_of(P), tokens = tokens_of(P);
  const int parts = few_parts<D, E4M3, NT>(P);
  if constexpr (NT == 2) {
    AdParams Q = P;
    Q.groups = (P.G + 7) / 8;
    const int split = few_parts<D, E4M3, 1>(Q);
    if (split && (split >= parts || tokens <= kDirectTokens)) return launch_few<D, E4M3, 1>(Q, split, st);
    if (tokens <= (parts ? kSplitTokens : kDirectTokens) &&
        items_of(Q) <= static_cast<long long>(sm_count()) * AdShape<D, E4M3, 1, 4, true>::BLOCKS)
      return start<D, E4M3, 1, 4, true>(Q, items_of(Q), 1, st) == cudaSuccess ? 0 : -1;
  }
  if (parts) return launch_few<D, E4M3, NT>(P, parts, st);
  constexpr int kOneWarp = S::ROWB > 256 ? 256 : 128;  // most tokens of a warp's item
  if (tokens <= kOneWarp && items < (1LL << 31) &&
      items > static_cast<long long>(sm_count()) * AdShape<D, E4M3, NT, 4, true>::BLOCKS)
    return start<D, E4M3, NT, 1, true>(P, items, 1, st) == cudaSuccess ? 0 : -1;
  if (tokens <= kDirectTokens && items < (1LL << 31))
    return start<D, E4M3, NT, 4, true>(P, items, 1, st) == cudaSuccess ? 0 : -1;
  long long blocks = static_cast<long long>(sm_count()) * S::BLOCKS;
  if (blocks > kAdMostBlocks) blocks = kAdMostBlocks;
  const long long most = (items * ((tokens + S::RUN + S::UNIT - 2) / S::UNIT * S::UNIT) + kMinTokens - 1) / kMinTokens;
  if (blocks > most) blocks = most;
  if (start<D, E4M3, NT, 4, false>(P, blocks, 1, st) != cudaSuccess) return -1;
  return launch_pdl(attn_join_kernel<D, E4M3, NT>, dim3(static_cast<unsigned>(blocks)), dim3(kJoinWarps * 32), 0, st, P) == cudaSuccess
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
