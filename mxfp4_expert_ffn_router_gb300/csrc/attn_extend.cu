// attn_extend.cu -- attention of several new tokens per sequence over a paged key-value cache.
//
// A row (a new token's query head) sees places c of its sequence: all up to its own, within a window and the first `sinks`, or
// the context and the drafted tokens that its mask names.  With a running reference m and sum l of the weights:
//   s_c = scale q . K_c ;  w_c = 2^((s_c - m) log2 e) ;  l = sum w_c ;  out = (sum w_c V_c) / l ;  lse = m + ln l
// The reference is that of the row's first tile; it moves, and the sums with it, only when a weight would pass 2^8, which
// seldom happens after the first tiles.  Statistics and sums are fp32.
//
// The query heads of one key-value head read the same keys, so an item is 256 rows (tokens x heads) of one key-value
// head: two streams of 128, the rows of one tcgen05.mma, over the same tiles of 128 places.  (128 rows or fewer: the streams
// take every other tile, and are added at the end.  Head size 256: one stream, 64 places, as two do not fit.)  While one
// stream's scores become weights, the tensor cores multiply for the other.  A block is 16 warps:
//   0-7    softmax: a thread is a row; scores from tensor memory, weights back into the columns that the scores had
//   8, 10  products of one stream: scores q K^T, and weights (from tensor memory) by values
//   9      items and their tiles, by TMA, a page or a tile a copy; a place that no row needs comes as zeros
//   11     (E4M3) the keys' scales as numbers
//   12-15  values: E4M3 to bf16; values that not all rows see, if not finite, are left out of the product (0 times them is
//          not 0) and added at the item's end to the sums of the rows that do see them
// Tensor memory is full: 2 x 128 columns of scores or weights, 2 x 128 (or 256) of sums.  Shared memory holds the queries (2 x
// 32 KB), three tiles of keys and two of values at 128 wide.
//
// E4M3: keys are operands as they are stored (kind::f8f6f4).  A query row, times a power of two that brings its largest value
// into [128, 256), is the sum of two E4M3 numbers, each with a product of its own, and the raw score is scaled by the key's
// and the row's power of two.  The second number's smallest step is 2^-9: the sum is exact from 2^-2 on, 2^-9 of the row's
// largest, and below that off by 2^-10 at most, 2^-17 of it (a row with one large channel loses bits of the others).  Values
// become bf16 exactly: codes shifted into place and times one bf16 power of two.
//
// Roundings: a weight to bf16 once, by 2^-8 of itself at most, as the output is; l sums the weights before that.  (As two
// bf16 numbers, 16 bits, the products with V are twice as many, which takes a prompt of 8192 16 % more time.)
//
// How the work is cut.  Where the items fill at most one block an SM: one block an item, or several to a long item.
// Otherwise a line of all items' tiles is cut into equal pieces, one an SM, by a kernel of one block, and pieces of cut items are
// added by another, in the order of the pieces.  Results repeat bit for bit: the only atomics set bits.
//
// What bounds it.  A pair of tiles (256 rows x 128 places x 128 wide) is 2050 clocks of products at the tensor cores' rate and 2100
// of softmax (exponentials 1024, the rest adds, maxima, conversions) on the four schedulers, at once where the streams
// alternate.  Measured 3700 clocks (bf16) and 5500 (E4M3, whose values' conversion runs on the same schedulers, 900 to
// 1400 clocks, and pulls the streams into step): waits for loads from tensor memory, for barriers and for instructions, of which a
// pass over this code needs more than the nearest cache holds.
//   8192 tokens of a prompt, 64 / 8 heads of 128, window 4096, bf16:   853 us, 968 TFLOP/s (0.51 of a large product's rate)
//   60 drafted tokens on 131072, 64 / 8 heads, E4M3:                   322 us, 801 TFLOP/s; 0.85 TB/s
//   64 drafted tokens on each of 16 sequences up to 16384, E4M3:       170 us, 307 TFLOP/s (bf16: 138)
//   chunks of up to 1000 tokens of 6 sequences up to 12000, E4M3:      187 us, 435 TFLOP/s (bf16: 143)
//   24 prompts of up to 301 tokens, 16 heads on one of 64, bf16:        26 us: first tile, few steps, end
// Tried without gain: registers moved from the other warps to the softmax warps; eight warps for the values; a handshake a step that
// holds the second stream half a step behind; helpers called instead of inlined; scores 32 at a time; the
// next item's queries asked for a step earlier (1 % more for a prompt, 4 % for chunks: longer code).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "decoder_ops.h"
#include "k3moe_dev.cuh"
#include "mx8_quant.cuh"
#include "per_device.h"
#include "tc_sm103.cuh"

namespace k3moe {

namespace {

constexpr int kAxThreads = 512;    // warps 0-7 softmax, 8 and 10 products, 9 loads, 11 the keys' scales, 12-15 values
constexpr int kAxMostBlocks = 160; // pieces of the line (bounds the workspace)
// What an item costs besides its tiles, in units of the line (a tile of up to 128 rows is one, of more two).  Prompt of 4096, 64 / 8
// heads, bf16, with 1, 2, 3, 5 and 8: 352, 342, 327, 316 and 314 us; 6 ragged chunks, 32 / 4 heads, E4M3: 417, 414, 393, 364
// and 335; 16 trees, 64 / 8 heads, bf16: 266, 266, 271, 271 and 274; 7 trees, 256 wide: 59, 59, 59, 61 and 63.
constexpr int kItemLen = 3;
// (direct) Fewest tiles that a part of the longest item may have.  1, 2 and 4 take the same time within 2 us, but for 3
// sequences of 100 tokens on 1000, 32 / 4 heads, bf16, where it is 29, 33 and 33.
constexpr int kPartTiles = 2;
constexpr int kJoinParts = 4;      // parts that are added at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.4e38f;  // reference of a part without a step, which has no sums (those of a row are -inf, or far above)
constexpr float kGrowth = 8.f;     // a row's reference moves once a weight would pass 2^8 (values up to 2^119 stay within fp32)

struct AxStart {  // where a block's piece of the line begins
  long long begin;  // of the item that it begins in
  int b, head, t, pad;
};
struct AxPlan {
  long long total, share;
};

struct AxParams {
  const uint8_t *k, *v, *ks, *vs;
  int heads, pages, page_shift;
  int B, rows, Hq, G;
  const uint16_t *q;
  long long q_stride;
  const int32_t *offsets;
  int max_new;
  int others;  // sequences of at most this many new tokens are left alone
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
  AxPlan *plan;
  AxStart *start;
  int4 *meta;        // [blocks]: {sequence, head, tile, parts} of the item that begins in the block's piece and goes on
  int *first_entry;  // [B + 1]
  long long *prefix; // [entries + 1]
  float2 *stat;      // [2 blocks][rows of a tile]: reference, sum of the weights
  float *part;       // [2 blocks][dim][rows of a tile]
  int blocks, entries;  // pieces; room for the tiles of query rows
  int parts;  // (direct) blocks of an item
  uint32_t per_head;    // ceil(2^32 / G) (token_of)
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
  else if (o1 - o0 > P.others)
    s.m = o1 - o0;
  s.ctx = s.n - s.m;
  if (s.m > s.n) bad = true;
  if (bad && report) set_status(P.status, K3MOE_DEV_BOUNDS);
  return s;
}

// An item: up to 128 rows a stream of one sequence and head, and which of its tiles are this block's.
struct AxItem {
  int n, first, m, ctx;  // (Seq)
  int b, head, t, r0, rows;  // rows 0: there is none, and none follows
  int lo, sinks, sink_tiles, t0;   // (Tiles)
  int clear_below, clear_above;    // tiles that all rows see whole end at most there, or begin past there or within the sinks
  int u0, u1, units, both, slot, parts;
  __device__ __forceinline__ int tile(int u) const { return u < sink_tiles ? u : u - sink_tiles + t0; }
  __device__ __forceinline__ int steps() const { return both ? 2 * (u1 - u0) : u1 - u0; }
};
// What a block's warps share besides the tiles.
template <int NK, int NV, int NR, int TK>
struct AxShared {
  uint64_t k_full[NK], k_ready[NK], k_empty[NK], v_full[NV], v_ready[NV], v_empty[NV], r_full[NR], r_empty[NR];
  uint64_t s_full[2], p_half[2], half_done[2], p_ready[2], pv_done[2], q_ready[2];
  uint64_t go;               // the second stream may start
  uint64_t j_shown, j_read;  // the streams' joint: sums shown, sums read
  float2 stat[2][128];       // the streams' statistics: reference, sum of the weights
  AxItem item[4];            // items by turns, as the loading warp comes to them
  uint64_t item_full[4], item_empty[4];
  alignas(16) float key_scale[8][TK];
  alignas(16) float ones[TK];  // (E4M3) of the places of a tile, by turns
  float row_scale[2][2][TK > 1 ? 128 : 1];  // (E4M3) of the query rows, of items by turns
  alignas(16) uint8_t key_bytes[NK][TK > 1 ? 128 : 16];
  uint8_t lost[16];  // of a tile: bit x for the 16 places from 16 x on that lie in no page of the cache
  uint32_t odd;      // bit x: values that are not finite were left out of item x's products
  uint32_t tmem;
};

template <int D, bool E4M3>
struct AxShape {
  static constexpr int TN = D == 256 ? 64 : 128;   // places of a tile
  static constexpr int NS = D == 256 ? 1 : 2;      // streams: 128 query rows with sums of their own
  static constexpr int ROWS = 128 * NS;            // query rows of an item
  static constexpr int QB = 128 * D * 2;           // bytes of a stream's queries
  static constexpr int TILE = TN * D * 2;          // bytes of a tile's values as operands
  static constexpr int KTILE = E4M3 ? TN * D : TILE;  // of its keys
  static constexpr int RAWB = E4M3 ? TN * D + 128 : 0;  // of its values' codes and scales
  static constexpr int NK = D == 64 ? 4 : 3, NV = D == 64 ? (E4M3 ? 3 : 4) : 2, NR = E4M3 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int SW = D * (E4M3 ? 1 : 2) >= 128 ? 128 : 64;  // bytes of a swizzled row of keys and queries
  using Shared = AxShared<NK, NV, NR ? NR : 1, E4M3 ? TN : 1>;
  static constexpr int OFF_K = NS * QB, OFF_V = OFF_K + NK * KTILE, OFF_R = OFF_V + NV * TILE, OFF_S = OFF_R + NR * RAWB;
  static constexpr int SMEM = OFF_S + sizeof(Shared);
  static constexpr int S_COLS = TN;                // columns of a score buffer
  static constexpr int O_COL = 256, O_COLS = D == 256 ? 256 : 128;
};

// ---- which places the rows of an item see
struct Tiles {
  int pmin, pmax;    // positions of its first and last row
  int lo, sinks;     // seen by any of them: lo .. pmax and 0 .. sinks - 1
  int sink_tiles, t0, units;
  __device__ __forceinline__ int tile(int u) const { return u < sink_tiles ? u : u - sink_tiles + t0; }
  // Whether some row sees some of the `run` places from `place` on (pages that none sees may have been given back)
  __device__ __forceinline__ bool needs(const Seq &s, int place, int run) const {
    return place < s.n && (place + run > lo || place < sinks);
  }
};
template <int TN>
__device__ __forceinline__ Tiles tiles_of(const AxParams &P, const Seq &s, int r0, int rows) {
  Tiles t;
  if (P.masks) {
    t.pmin = s.ctx;
    t.pmax = s.n - 1;
  } else {
    t.pmin = s.ctx + r0 / P.G;
    t.pmax = s.ctx + (r0 + rows - 1) / P.G;
  }
  t.lo = P.window > 0 && t.pmin >= P.window ? t.pmin - P.window + 1 : 0;
  t.t0 = t.lo / TN;
  const int t1 = t.pmax >= 0 ? t.pmax / TN + 1 : 0;
  t.sinks = P.window > 0 ? min(P.sinks, t.pmax + 1) : 0;
  t.sink_tiles = t.sinks > 0 ? min((t.sinks - 1) / TN + 1, t.t0) : 0;
  t.units = max(1, t.sink_tiles + t1 - t.t0);
  return t;
}
// Whether some row does not see some place of the tile.
template <int TN>
__device__ __forceinline__ bool masked(const AxParams &P, const AxItem &I, int tile) {
  const int c0 = tile * TN, c1 = c0 + TN;
  return c1 > I.clear_below || (c0 <= I.clear_above && c1 > P.sinks);
}

// n / G for 0 <= n < 2^16.
__device__ __forceinline__ int token_of(const AxParams &P, int n) {
  return P.G == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), P.per_head));
}
// The page of a place; whether the cache has it.
__device__ __forceinline__ int page_of(const AxParams &P, int b, int place) {
  return P.table[static_cast<size_t>(b) * P.max_pages + (place >> P.page_shift)];
}
__device__ __forceinline__ bool is_page(const AxParams &P, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(P.pages);
}
// The e-th of the items that all sequences' rows of one head make up, by a whole warp: its sequence (-1: there are fewer),
// and which of that one's it is.
template <int ROWS>
__device__ __forceinline__ int sequence_of(const AxParams &P, int e, int &t) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    int mine = 0;
    if (b0 + lane < P.B) mine = static_cast<int>((static_cast<long long>(seq_of(P, b0 + lane, false).m) * P.G + ROWS - 1) / ROWS);
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += o;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + upto > e);
    if (past) {
      const int at = __ffs(past) - 1;
      t = e - before - __shfl_sync(0xFFFFFFFFu, upto - mine, at);
      return b0 + at;
    }
    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return -1;
}
// A block's piece of the line, item by item.
template <int TN, int ROWS>
struct Walk {
  long long from, to, begin;
  int b, head, t, tiles;
  Seq s;
  int r0, rows;  // query rows of the item
  Tiles list;
  int weight;    // of a tile on the line
  int u0, u1;    // the item's tiles that are this piece's
  bool more;

  __device__ __forceinline__ void measure(const AxParams &P) {
    r0 = t * ROWS;
    rows = min(ROWS, s.m * P.G - r0);
    list = tiles_of<TN>(P, s, r0, rows);
    weight = rows > 128 ? 2 : 1;
  }
  __device__ __forceinline__ void set_seq(const AxParams &P) {
    s = seq_of(P, b, false);
    tiles = P.first_entry[b + 1] - P.first_entry[b];
  }
  __device__ __forceinline__ int unit_at(long long x) const {
    const long long u = (x - begin - kItemLen + weight - 1) >> (weight - 1);
    return u < 0 ? 0 : u > list.units ? list.units : static_cast<int>(u);
  }
  __device__ __forceinline__ void enter() { u0 = unit_at(from), u1 = unit_at(to); }
  __device__ __forceinline__ long long length() const { return kItemLen + static_cast<long long>(list.units) * weight; }
  __device__ __forceinline__ void init(const AxParams &P, int block) {
    const long long total = P.plan->total, share = P.plan->share;
    from = block * share;
    to = min(total, from + share);
    more = from < to;
    if (!more) return;
    const AxStart st = P.start[block];
    begin = st.begin, b = st.b, head = st.head, t = st.t;
    set_seq(P);
    measure(P);
    enter();
    if (u0 >= u1) next(P);
  }
  __device__ __forceinline__ void next(const AxParams &P) {
    do {
      begin += length();
      more = begin + kItemLen < to;
      if (!more) return;
      if (++t == tiles) {
        t = 0;
        if (++head == P.heads) {
          head = 0;
          do {
            if (++b >= P.B) {
              more = false;
              return;
            }
            set_seq(P);
          } while (tiles == 0);
        }
      }
      measure(P);
      enter();
    } while (u0 >= u1);
  }
  __device__ __forceinline__ void direct(const AxParams &P, int block) {
    const int item = block / P.parts, part = block - item * P.parts, e = item / P.heads;
    head = item - e * P.heads;
    if (block == 0)
      for (int x = threadIdx.x & 31; x < P.B; x += 32) seq_of(P, x, true);
    b = sequence_of<ROWS>(P, e, t);
    more = b >= 0;
    if (!more) return;
    s = seq_of(P, b, false);
    measure(P);
    u0 = list.units * part / P.parts, u1 = list.units * (part + 1) / P.parts;
  }
  __device__ __forceinline__ void show(const AxParams &P, AxItem &I) const {
    I.n = s.n, I.first = s.first, I.m = s.m, I.ctx = s.ctx;
    I.b = b, I.head = head, I.t = t, I.r0 = r0, I.rows = rows;
    I.lo = list.lo, I.sinks = list.sinks, I.sink_tiles = list.sink_tiles, I.t0 = list.t0;
    I.clear_below = P.masks ? s.ctx : list.pmin + 1, I.clear_above = P.window > 0 ? list.pmax - P.window : -1;
    I.u0 = u0, I.u1 = u1, I.units = list.units, I.both = weight - 1;
    if (P.parts) {
      I.slot = blockIdx.x, I.parts = P.parts;
    } else {
      I.slot = 2 * blockIdx.x + (u0 > 0 ? 0 : 1), I.parts = u0 > 0 || u1 < list.units ? 2 : 1;
      if (u0 == 0 && u1 < list.units) {  // the item begins here and goes on
        const long long last = begin + kItemLen + static_cast<long long>(list.units - 1) * weight;
        P.meta[blockIdx.x] = make_int4(b, head, t, static_cast<int>(last / P.plan->share) - static_cast<int>(blockIdx.x) + 1);
      }
    }
  }
};

// ---- small device functions
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// A wait of a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mb_wait(bar, parity));
}
__device__ __forceinline__ uint32_t below(int k) { return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u; }
__device__ __forceinline__ void cp_or_zeros16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_or_zeros8(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(su32(bar))
               : "memory");
}

// Rows of 64 bytes, 64-byte swizzle, groups of eight rows 512 bytes; or of 128 (smem_desc_sw128).
template <int SW>
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr) {
  if (SW == 128) return smem_desc_sw128(saddr);
  return static_cast<uint64_t>((saddr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(4) << 61);
}
// Instruction descriptor, kind::f8f6f4: E4M3 A and B along K, fp32 sums.
__device__ __forceinline__ uint32_t idesc_e4m3(int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// Instruction descriptor, kind::f16: bf16 A and B, fp32 sums; B along K (keys) or along N (values).
__device__ __forceinline__ uint32_t idesc(int N, bool b_along_n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_along_n ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}
// Values [place][64 dimensions], 128-byte swizzle, along N: blocks of 64 dimensions `block` bytes
// apart, groups of eight places 1024 bytes.
__device__ __forceinline__ uint64_t values_desc(uint32_t saddr, uint32_t block) {
  return static_cast<uint64_t>((saddr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(block >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// The products are issued by one elected thread of a warp that runs converged, so that the operands' addresses stay in
// uniform registers: issued from a branch of lane 0 they cost about ten instructions a product, and the tensor
// cores waited for those.
//
// Four products of 16 dimensions each: descriptors 32 bytes further each; the first one adds where `acc` is not 0.
__device__ __forceinline__ void mma4_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %3, %3;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// Two products of 32 dimensions each in E4M3.
__device__ __forceinline__ void mma2_scores_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, b1;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %3, %3;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 b1, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// Weights of 64 places (8 columns each by 16 places) with their values, 2048 bytes each 16.
__device__ __forceinline__ void mma4_values(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %3, %3;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// tc_commit from the elected thread of a converged warp.
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(bar))
      : "memory");
}
// 32 columns of this thread's lane; the values are there after tc_wait_ld.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld16f(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tc_wait_ld(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // (uses stay behind the wait)
}
__device__ __forceinline__ void tc_st32r(uint32_t taddr, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
      "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]),
      "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two codes of `w` (bytes 0 and 1 of the selection) to bf16 patterns of their values times 2^-120: exponent and
// mantissa move to their places, subnormal codes to subnormal numbers.  (A NaN's code is not seen.)
__device__ __forceinline__ uint32_t codes_up(uint32_t w, uint32_t sel) {
  const uint32_t x = __byte_perm(w, 0u, sel);
  return ((x >> 4) & 0x07F007F0u) | (x & 0x80008000u);
}

// Raw scores times their keys' scales.
template <int N, int M>
__device__ __forceinline__ void scale_keys(float (&v)[M], const float *ks) {
#pragma unroll
  for (int y = 0; y < N; y += 4) {
    const float4 k = *reinterpret_cast<const float4 *>(ks + y);
    v[y] *= k.x, v[y + 1] *= k.y, v[y + 2] *= k.z, v[y + 3] *= k.w;
  }
}

__device__ const uint32_t g_no_mask[32] = {};  // of a drafted token that sees nothing

// What a row sees.
struct Row {
  int hi, lo;            // its place (causal: the last that it sees; below 0: it has none); first of the window
  const uint32_t *mask;  // (drafted) its words
  bool on;               // a row of the item
};
// The 32 places from c on, of which bit x stands for c + x.
__device__ __forceinline__ uint32_t sees(const AxParams &P, const AxItem &s, const Row &row, int c) {
  const uint32_t win = P.window > 0 ? ~below(row.lo - c) | below(P.sinks - c) : 0xFFFFFFFFu;
  if (!P.masks) return below(row.hi + 1 - c) & win;
  uint32_t v = below(s.ctx - c) & win;
  const int j = c - s.ctx;  // the new token that bit 0 stands for
  if (j > -32 && j < s.m && row.hi >= 0) {  // (a row without a place has no context: this is all that it could see)
    const int at = j >> 5, most = 2 * P.words;
    const uint32_t w0 = at >= 0 && at < most ? row.mask[at] : 0u;
    const uint32_t w1 = at + 1 >= 0 && at + 1 < most ? row.mask[at + 1] : 0u;
    v |= __funnelshift_r(w0, w1, j & 31) & below(s.m - j);
  }
  return v;
}

// Whether any of 32 dimensions of a cached value may not be finite (E4M3: a NaN's code, or a scale that makes one).
template <int D, bool E4M3>
__device__ __forceinline__ bool may_be_odd(const AxParams &P, size_t vec, int x0) {
  const uint4 *from = reinterpret_cast<const uint4 *>(P.v + (vec * D + x0) * (E4M3 ? 1 : 2));
  uint32_t odd = 0;
#pragma unroll
  for (int y = 0; y < (E4M3 ? 2 : 4); ++y) {
    const uint4 u = from[y];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int z = 0; z < 4; ++z) odd |= E4M3 ? (w[z] & 0x7F7F7F7Fu) + 0x01010101u : (w[z] & 0x7F807F80u) + 0x00800080u;
  }
  return (odd & (E4M3 ? 0x80808080u : 0x80008000u)) || (E4M3 && P.vs[vec] > 246);  // (448 2^119 is finite)
}

// Adds the values that are not finite and were left out of the products to the sums of a row that sees them.  They lie in
// tiles that not all rows see whole: an item has a few of those, however long its sequence is.  The others of the block
// wait meanwhile, within a bound, so a lane looks at a place's 32 dimensions at once, and only places with something odd are
// gone through: a tree of 60 on 131072 places, 324 us, takes 386 with a NaN in the newest place; on 16000 84 for 67 (9110
// where all places of a piece are gone through one by one).
template <int D, bool E4M3, int TN>
__device__ __noinline__ void add_left_out(const AxParams &P, const AxItem &I, const Row row, int st, uint32_t oa) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int x0 = 0; x0 < D; x0 += 32) {
    float o[32];
    __syncwarp();
    tc_ld32(oa + x0, o);
    tc_wait_ld(o);
#pragma unroll 1
    for (int u = I.u0; u < I.u1; ++u) {
      const int tile = I.tile(u);
      if ((!I.both && D < 256 && ((u - I.u0) & 1) != st) || !masked<TN>(P, I, tile)) continue;
#pragma unroll 1
      for (int c = tile * TN; c < (tile + 1) * TN && c < I.n; c += 32) {
        const int place = c + lane, page = place < I.n ? page_of(P, I.b, place) : -1;
        long long vec = -1;
        if (is_page(P, page)) {
          vec = ((static_cast<long long>(page) * P.heads + I.head) << P.page_shift) + (place & ((1 << P.page_shift) - 1));
          if (!may_be_odd<D, E4M3>(P, vec, x0)) vec = -1;
        }
        uint32_t odd = __ballot_sync(0xFFFFFFFFu, vec >= 0);
        const uint32_t seen = row.on ? sees(P, I, row, c) : 0u;
        while (odd) {
          const int at = __ffs(odd) - 1;
          odd &= odd - 1;
          const long long from = __shfl_sync(0xFFFFFFFFu, vec, at);
          if (!((seen >> at) & 1u)) continue;
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            float w;
            if (E4M3) {
              uint32_t a, z;
              e4m3x4_to_f16x2(P.v[from * D + x0 + y], a, z);
              w = __half2float(__ushort_as_half(static_cast<unsigned short>(a))) * e8m0_to_f32(P.vs[from]);
            } else {
              w = bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(P.v)[from * D + x0 + y]);
            }
            if (!isfinite(w)) o[y] += w;
          }
        }
        __syncwarp();
      }
    }
    __syncwarp();
    tc_st32r(oa + x0, o);
  }
  tc_wait_st();
}

}  // namespace

// The pieces of the line: one block measures the sequences, sums their lengths and finds where each piece begins.  Latency
// of a few scans; 3 to 5 us, which is why short calls go without.
template <int TN, int ROWS>
__global__ void __launch_bounds__(1024) attn_plan_kernel(const AxParams P) {
  __shared__ long long s_scan[32];
  __shared__ long long s_carry;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  auto scan = [&](long long v, long long &before) {  // exclusive over the block, plus the carry; the carry grows
    long long incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long w = s_scan[lane], wi = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, wi, off);
      if (lane >= off) wi += o;
    }
    const long long warps_before = __shfl_sync(0xFFFFFFFFu, wi - w, warp), all = __shfl_sync(0xFFFFFFFFu, wi, 31);
    before = s_carry + warps_before + incl - v;
    __syncthreads();
    if (tid == 0) s_carry += all;
    __syncthreads();
  };
  if (tid == 0) s_carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < P.B; b0 += 1024) {
    const int b = b0 + tid;
    long long tiles = 0, before;
    if (b < P.B) {
      const Seq s = seq_of(P, b, true);
      tiles = (static_cast<long long>(s.m) * P.G + ROWS - 1) / ROWS;
    }
    scan(tiles, before);
    if (b < P.B) P.first_entry[b] = static_cast<int>(min(before, static_cast<long long>(P.entries)));
  }
  // (there is room for all unless the offsets descend, and sequences share rows)
  const int entries = static_cast<int>(min(s_carry, static_cast<long long>(P.entries)));
  if (tid == 0) P.first_entry[P.B] = entries;
  __syncthreads();
  if (tid == 0) s_carry = 0;
  __syncthreads();
  // the last sequence whose first entry is at most e
  auto seq_at = [&](auto at_most) {
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at_most(mid))
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  };
  for (int e0 = 0; e0 < entries; e0 += 1024) {
    const int e = e0 + tid;
    long long len = 0, before;
    if (e < entries) {
      const int b = seq_at([&](int x) { return P.first_entry[x] <= e; });
      Walk<TN, ROWS> w;
      w.s = seq_of(P, b, false);
      w.t = e - P.first_entry[b];
      w.measure(P);
      len = w.length();
    }
    scan(len, before);
    if (e < entries) P.prefix[e] = before;
  }
  if (tid == 0) P.prefix[entries] = s_carry;
  __syncthreads();
  const long long total = s_carry * P.heads, share = max(8LL, (total + P.blocks - 1) / P.blocks);
  if (tid == 0) *P.plan = {total, share};
  if (tid < P.blocks) {
    P.meta[tid] = make_int4(0, 0, 0, 0);
    const long long x = tid * share;
    if (x < total) {
      const int b = seq_at([&](int y) { return P.prefix[P.first_entry[y]] * P.heads <= x; });
      const int f0 = P.first_entry[b], f1 = P.first_entry[b + 1];
      const long long p0 = P.prefix[f0], len = P.prefix[f1] - p0, base = p0 * P.heads;
      const int head = static_cast<int>((x - base) / len);
      const long long at = x - base - head * len + p0;
      int lo = f0, hi = f1 - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.prefix[mid] <= at)
          lo = mid;
        else
          hi = mid - 1;
      }
      P.start[tid] = {base + head * len + P.prefix[lo] - p0, b, head, lo - f0, 0};
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kAxThreads, 1)
    attn_extend_kernel(const __grid_constant__ AxParams P, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using S = AxShape<D, E4M3>;
  constexpr int TN = S::TN, NS = S::NS, ROWS = S::ROWS, NK = S::NK, NV = S::NV, NR = S::NR > 0 ? S::NR : 1;
  extern __shared__ __align__(1024) uint8_t ax_smem[];
  uint8_t *smem = ax_smem;
  typename S::Shared &sh = *reinterpret_cast<typename S::Shared *>(smem + S::OFF_S);
  const uint32_t sbase = su32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) mb_init(&sh.k_full[i], 1), mb_init(&sh.k_ready[i], 1), mb_init(&sh.k_empty[i], NS);
    for (int i = 0; i < NV; ++i) mb_init(&sh.v_full[i], 1), mb_init(&sh.v_ready[i], 4), mb_init(&sh.v_empty[i], NS);
    for (int i = 0; i < NR; ++i) mb_init(&sh.r_full[i], 1), mb_init(&sh.r_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mb_init(&sh.s_full[i], 1), mb_init(&sh.p_half[i], 4), mb_init(&sh.half_done[i], 1), mb_init(&sh.p_ready[i], 4);
      mb_init(&sh.pv_done[i], 1), mb_init(&sh.q_ready[i], 4);
    }
    for (int i = 0; i < 4; ++i)  // (softmax and product warps of each stream, the scales', the values')
      mb_init(&sh.item_full[i], 1), mb_init(&sh.item_empty[i], 5 * NS + (E4M3 ? 1 : 0) + 4);
    mb_init(&sh.go, 1), mb_init(&sh.j_shown, 8), mb_init(&sh.j_read, 8);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh.odd = 0;
  }
  if (E4M3 && tid < TN) sh.ones[tid] = 1.f;
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sh.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool timeout = false;
  pdl_wait();
  pdl_trigger();
  // The next item, once the loading warp has come to it; null where there is none (or it did not come).
  auto item_at = [&](uint32_t i) -> const AxItem * {
    if (!warp_wait(&sh.item_full[i & 3], (i >> 2) & 1u)) {
      timeout = true;
      return nullptr;
    }
    const AxItem *I = &sh.item[i & 3];
    return I->rows ? I : nullptr;
  };
  auto item_done = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mb_arrive(&sh.item_empty[i & 3]);
  };

  if (warp < 4 * NS) {
    // ---- softmax: a thread is a row
    const int st = warp >> 2;  // stream
    const int lrow = 32 * (warp & 3) + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(32 * (warp & 3)) << 16, oa = tmem + lane_addr + S::O_COL + st * S::O_COLS;
    // Whether a tile's second half of scores is loaded while the first one's weights are computed, in code without a loop: over
    // bf16 a prompt takes 3 % less time so, over E4M3 chunks 14 % more, by the longer code and its registers.
    constexpr bool AHEAD = !E4M3;
    const bool flat = fabsf(P.scale) * kLog2e == 0.f;  // (queries of zeros then)
    const float c1 = flat ? 1.f : fabsf(P.scale) * kLog2e;
    // This stream's queries of an item: asked for, and, once they have come, made operands.  A thread converts what it has
    // copied: eight dimensions of a row, 128 / CH rows apart, all in loops, since their instructions are met cold
    // (unrolled, these two took 25000 clocks of a short call).
    constexpr int CH = D / 8;
    const int ch = tid % CH, q_row = (tid & 127) / CH;
    const uint32_t q_to = sbase + st * S::QB;
    auto place8 = [&](int rr) -> uint32_t {  // (E4M3) of eight dimensions in a part
      const int byte = ch * 8 % S::SW, sw = S::SW == 128 ? rr & 7 : (rr >> 1) & 3;
      return (ch * 8 / S::SW) * (128 * S::SW) + rr * S::SW + (((byte >> 4) ^ sw) << 4) + (byte & 8);
    };
    auto place16 = [&](int rr) -> uint32_t { return (ch / 8) * (128 * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4); };
    int q_rows = 0;
    auto ask_q = [&](const AxItem &I) {
      const int base = I.r0 + (I.both ? 128 * st : 0), left = I.r0 + I.rows - base, i0 = base / P.G, g0 = base - i0 * P.G;
      const uint16_t *q = P.q + (static_cast<long long>(I.first) + i0) * P.q_stride + static_cast<size_t>(I.head) * P.G * D + ch * 8;
      q_rows = min(128, (left + 128 / CH - 1) & ~(128 / CH - 1));  // (whole turns of the threads: the rest is not read)
      const int ii = token_of(P, g0 + q_row), step = token_of(P, 128 / CH), more = 128 / CH - step * P.G;
      int gg = g0 + q_row - ii * P.G;
      const long long by = step * P.q_stride + more * D, wrap = P.q_stride - static_cast<long long>(P.G) * D;
      q += ii * P.q_stride + gg * D;
#pragma unroll 2
      for (int rr = q_row; rr < q_rows; rr += 128 / CH) {
        const bool on = rr < left;
        const uint16_t *from = on ? q : P.q;
        if constexpr (E4M3) {
          cp_or_zeros8(q_to + place8(rr), from, on);
          cp_or_zeros8(q_to + 128 * D + place8(rr), from + 4, on);
        } else {
          cp_or_zeros16(q_to + place16(rr), from, on);
        }
        q += by, gg += more;
        if (gg >= P.G) q += wrap, gg -= P.G;
      }
    };
    uint32_t turn = 0;
    auto take_q = [&]() {
      cp_wait_all();
      const uint32_t flip = P.scale < 0.f ? 0x80008000u : 0u, keep = flat ? 0u : 0xFFFFFFFFu;
      if constexpr (E4M3) {
#pragma unroll 2
        for (int rr = q_row; rr < q_rows; rr += 128 / CH) {
          // the row times a power of two, to a largest value in [128, 256), in two E4M3 numbers a value
          uint2 *const to = reinterpret_cast<uint2 *>(smem + st * S::QB + place8(rr)), *const to2 = to + 128 * D / 8;
          const uint2 u0 = *to, u1 = *to2;
          const uint32_t w[4] = {(u0.x ^ flip) & keep, (u0.y ^ flip) & keep, (u1.x ^ flip) & keep, (u1.y ^ flip) & keep};
          uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
          m = max(m >> 16, m & 0xFFFFu);
#pragma unroll
          for (int off = 1; off < CH; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
          const int e = m == 0 ? 0 : max(-126, min(127, 7 + 127 - static_cast<int>(m >> 7)));
          const float up = exp2i(e);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float a = __uint_as_float(w[y] << 16) * up, b = __uint_as_float(w[y] & 0xFFFF0000u) * up;
            hi[y] = m >= 0x7F80u ? 0x7F7Fu : e4m3x2(a, b);  // (a row that is not finite gives NaN)
            uint32_t h, z;
            e4m3x4_to_f16x2(hi[y], h, z);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            lo[y] = e4m3x2(a - f.x, b - f.y);
          }
          *to = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *to2 = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (ch == 0) sh.row_scale[turn & 1][st][rr] = mx_pow2(-e);
        }
      } else if (flip || !keep) {
#pragma unroll 1
        for (int rr = q_row; rr < q_rows; rr += 128 / CH) {
          uint4 *const to = reinterpret_cast<uint4 *>(smem + st * S::QB + place16(rr));
          const uint4 u = *to;
          *to = make_uint4((u.x ^ flip) & keep, (u.y ^ flip) & keep, (u.z ^ flip) & keep, (u.w ^ flip) & keep);
        }
      }
      ++turn;
      fence_async();
      __syncwarp();
      if (lane == 0) mb_arrive(&sh.q_ready[st]);
    };
    uint32_t uses[2] = {0, 0};  // steps of each score buffer
    uint32_t items = 0, joins = 0, finals = 0, tiles_before = 0;
    const AxItem *ip = item_at(0);
    if (ip && ip->steps() > st) {
      ask_q(*ip);
      take_q();
    }
    while (ip) {
      const AxItem &I = *ip;
      const bool both = I.both;
      const int r = (both ? 128 * st : 0) + lrow;  // row of the item
      Row row;
      row.on = r < I.rows;
      const int i0 = I.r0 / P.G, i = min(i0 + token_of(P, I.r0 - i0 * P.G + r), I.m - 1);  // token
      int pos = I.ctx + i;
      row.mask = reinterpret_cast<const uint32_t *>(P.masks + (P.masks ? (static_cast<long long>(I.first) + i) * P.words : 0));
      if (P.masks) {
        int seen = 0;
#pragma unroll 1
        for (int w = 0; 32 * w < I.m; ++w) seen += __popc(row.mask[w] & below(I.m - 32 * w));
        pos = I.ctx + max(0, seen - 1);
      }
      row.hi = I.ctx + i;
      row.lo = P.window > 0 && pos >= P.window ? pos - P.window + 1 : 0;
      const bool warp_on = (both ? 128 * st : 0) + 32 * (warp & 3) < I.rows;
      float m = -INFINITY, l = 0.f;  // the reference, in scores; the weights' sum
      float c = c1;                  // powers of two of a score
      bool first = true;
      const int K = I.steps(), u0 = I.u0;
      int sb = st;
      for (int k = NS == 2 ? st : 0; k < K; k += NS) {
        sb = k & 1;
        const int u = both ? k >> 1 : k, tile = I.tile(u0 + u);
        const bool some = masked<TN>(P, I, tile);
        if (!warp_wait(&sh.s_full[sb], uses[sb] & 1u)) {
          timeout = true;
          break;
        }
        ++uses[sb];
        tc_fence_after();
        // (not 0, times which a reference of -inf would be NaN; raw scores are below 2^128, so that they count for nothing)
        if (E4M3 && first) c = fmaxf(c1 * sh.row_scale[(turn - 1) & 1][st][lrow], 0x1p-149f);
        if (warp_on) {
          const float *ks = nullptr;
          if constexpr (E4M3) ks = sh.key_scale[(tiles_before + u) & 7];
          const uint32_t sa = tmem + lane_addr + sb * S::S_COLS;
          const uint32_t lost = sh.lost[(tiles_before + u) & 15];
          float base = m == -INFINITY ? 0.f : m * c;
          float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float v[64];
          if (lost || some) {
#pragma unroll 1
            for (int x = 0; x < TN; x += 32) {
              tc_ld32(sa + x, v);
              uint32_t vis = sees(P, I, row, tile * TN + x);
              if (lost >> (x / 16) & 1u) vis &= 0xFFFF0000u;
              if (lost >> (x / 16) & 2u) vis &= 0xFFFFu;
              tc_wait_ld(v);
              if constexpr (E4M3) scale_keys<32>(v, ks + x);
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (!((vis >> y) & 1u)) v[y] = -INFINITY;
              tc_st32r(sa + x, v);
            }
            tc_wait_st();
            if constexpr (E4M3) ks = sh.ones;  // (they are scaled)
          }
          // 64 places at a time: scores in, weights out (in place: their 32 columns lie behind what was read)
#pragma unroll AHEAD ? TN / 64 : 1
          for (int x = 0; x < TN; x += 64) {
            if (!AHEAD || x == 0) {
              tc_ld32(sa + x, v);
              tc_ld32(sa + x + 32, v + 32);
            }
            tc_wait_ld(v);
            if constexpr (E4M3) scale_keys<64>(v, ks + x);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int y = 0; y < 64; y += 2) mx[(y / 2) & 3] = fmaxf(fmaxf(v[y], v[y + 1]), mx[(y / 2) & 3]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // (behind the item's last row there are no queries, but what shared memory held: those rows have no say)
            if (__any_sync(0xFFFFFFFFu, row.on && (top - m) * c > kGrowth)) {
              // the row's reference moves up: sums by the quotient
              const float mn = fmaxf(m, top), f = mn == -INFINITY ? 1.f : ex2((m - mn) * c);
              m = mn;
              base = m == -INFINITY ? 0.f : m * c;
              l *= f;
#pragma unroll
              for (int y = 0; y < 2; ++y) add[y].x *= f, add[y].y *= f;
              if (!first || x > 0) {
                // after the products of the places before, or of the step before (two streams: these scores say so)
                if (x > 0 ? !warp_wait(&sh.half_done[sb], (uses[sb] - 1) & 1u)
                          : NS == 1 && !warp_wait(&sh.pv_done[sb ^ 1], (uses[sb ^ 1] - 1) & 1u))
                  timeout = true;
                tc_fence_after();
                float o[16];
#pragma unroll 1
                for (int y = 0; y < D; y += 16) {
                  tc_ld16f(oa + y, o);
                  tc_wait_ld(o);
                  uint32_t h[16];
#pragma unroll
                  for (int z = 0; z < 16; ++z) h[z] = __float_as_uint(o[z] * f);
                  tc_st16u(oa + y, h);
                }
                tc_wait_st();
              }
            }
            const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int y = 0; y < 32; y += 2) {
                const float2 e = fma2(make_float2(v[h + y], v[h + y + 1]), c2, b2), w = make_float2(ex2(e.x), ex2(e.y));
                pk[y / 2] = bf16x2(w.x, w.y);
                add[(y / 2) & 1] = add2(add[(y / 2) & 1], w);
              }
              tc_st16u(sa + (x + h) / 2, pk);
              if (AHEAD && x + 64 < TN) tc_ld32(sa + x + 64 + h, v + h);  // (the next ones are on their way meanwhile)
            }
            if (x + 64 < TN) {  // these can be multiplied while the others are computed
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mb_arrive(&sh.p_half[sb]);
            }
          }
          l += (add[0].x + add[0].y) + (add[1].x + add[1].y);
          tc_wait_st();
        } else if (TN > 64 && lane == 0) {
          mb_arrive(&sh.p_half[sb]);
        }
        first = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&sh.p_ready[sb]);
      }
      if (timeout) break;
      // ---- the item's end: the next one's queries are asked for (the last scores are there: this one's are not read
      // any more), then this one's sums
      const bool had = !first;  // whether this stream had a step
      const AxItem *const next = item_at(items + 1);
      const bool next_q = next && next->steps() > st;
      if (next_q) ask_q(*next);
      if (next_q) take_q();
      if (had) {
        if (!warp_wait(&sh.pv_done[sb], (NS == 2 ? finals : uses[sb] - 1) & 1u)) {
          timeout = true;
          break;
        }
        ++finals;
        tc_fence_after();
      }
      if ((*reinterpret_cast<volatile uint32_t *>(&sh.odd) >> (items & 31) & 1u) && had && warp_on)
        add_left_out<D, E4M3, TN>(P, I, row, st, oa);
      float mb = m == -INFINITY ? -INFINITY : m * c, f0 = 1.f, f1 = 0.f;
      const bool split = NS == 2 && !both;  // the streams share the rows: each writes half of the dimensions
      if (split) {
        sh.stat[st][lrow] = make_float2(mb, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&sh.j_shown);
        if (!warp_wait(&sh.j_shown, joins & 1u)) {
          timeout = true;
          break;
        }
        tc_fence_after();
        if (K > 1) {
          const float2 a = sh.stat[0][lrow], b = sh.stat[1][lrow];
          mb = fmaxf(a.x, b.x);
          const float base = mb == -INFINITY ? 0.f : mb;
          f0 = ex2(a.x - base), f1 = ex2(b.x - base);
          l = a.y * f0 + b.y * f1;
        } else {
          mb = sh.stat[0][lrow].x, l = sh.stat[0][lrow].y;
        }
      }
      if (warp_on) {
        const bool cut = I.parts > 1;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        // (computed here, so that it takes no registers before)
        const int at = I.r0 % P.G + r, token = token_of(P, at);
        const size_t orow = (static_cast<size_t>(I.first) + I.r0 / P.G + token) * P.Hq + I.head * P.G + at - token * P.G;
        const int x0 = split ? st * (D / 2) : 0, x1 = split ? x0 + D / 2 : D;
        const uint32_t o0 = split ? tmem + lane_addr + S::O_COL : oa, o1 = o0 + S::O_COLS;
        // Written from their own lanes, a row each, 16 bytes would be a line of their own, 32 a store (5900 clocks an
        // item); four lanes exchange theirs, and write 64 bytes of each of their rows in turn.
        const int j = lane & 3;
#pragma unroll 1
        for (int x = x0; x < x1; x += 32) {
          float o[32];
          __syncwarp();
          tc_ld32(o0 + x, o);
          tc_wait_ld(o);
          if (split && K > 1) {
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              float z[16];
              tc_ld16f(o1 + x + h, z);
              tc_wait_ld(z);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[h + y] = o[h + y] * f0 + z[y] * f1;
            }
          }
          if (cut) {
            if (!row.on) continue;
            float *part = P.part + (static_cast<size_t>(I.slot) * D + x) * ROWS + r;
#pragma unroll
            for (int y = 0; y < 32; ++y) part[y * ROWS] = o[y];
          } else {
            uint32_t w[4][4];
#pragma unroll
            for (int z = 0; z < 16; ++z) w[z / 4][z % 4] = l == 0.f ? 0u : bf16x2(o[2 * z] * inv, o[2 * z + 1] * inv);
#pragma unroll
            for (int s = 1; s < 4; s <<= 1) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if (y & s) continue;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, j & s ? w[y][z] : w[y + s][z], s);
                  if (j & s)
                    w[y][z] = got;
                  else
                    w[y + s][z] = got;
                }
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              // (a row's index fits 32 bits: out would not fit the device else)
              const size_t to = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(orow), lane - j + y);
              if (r - j + y < I.rows)
                *reinterpret_cast<uint4 *>(P.out + to * D + x + 8 * j) = make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
            }
          }
        }
        if (row.on && !(split && st)) {
          if (cut)
            P.stat[static_cast<size_t>(I.slot) * ROWS + r] = make_float2(K > 0 ? mb : kNone, l);
          else if (P.lse)
            P.lse[orow] = l == 0.f ? -INFINITY : (mb + log2f(l)) * kLn2;
        }
      }
      if (split) {  // the sums have been read: the next item's may come
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&sh.j_read);
        if (!warp_wait(&sh.j_read, joins & 1u)) {
          timeout = true;
          break;
        }
        ++joins;
      }
      tiles_before += I.u1 - u0;
      item_done(items);
      ++items;
      ip = next;
    }
  } else if (warp == 8 || (NS == 2 && warp == 10)) {
    // ---- products of one stream (or of both score buffers in turn): the scores of a step's next but one follow its
    // weights' products, which read the same columns, in the tensor cores' order
    const int st = NS == 2 ? (warp - 8) / 2 : 0;
    uint32_t tiles_before = 0, kt = 0, vt = 0, uses[2] = {0, 0}, asked = 0, goes = 0;
    const uint32_t id_s = E4M3 ? idesc_e4m3(TN) : idesc(TN, false), id_o = idesc(D, true);
    const uint64_t qd = rows_desc<S::SW>(sbase + st * S::QB);
    uint64_t *const keys = E4M3 ? sh.k_ready : sh.k_full;
    const AxItem *I;
    for (uint32_t items = 0; (I = item_at(items)) != nullptr; ++items) {
      const bool both = I->both;
      const int T = I->u1 - I->u0, K = I->steps();
      // every tile passes every stream, in order: those that it does not use it gives back at once
      auto pass_keys = [&](uint32_t t) {
        for (; kt < t; ++kt) {
          if (!warp_wait(&keys[kt % NK], (kt / NK) & 1u)) return false;
          if (lane == 0) mb_arrive(&sh.k_empty[kt % NK]);
        }
        return true;
      };
      auto pass_values = [&](uint32_t t) {
        for (; vt < t; ++vt) {
          if (!warp_wait(&sh.v_ready[vt % NV], (vt / NV) & 1u)) return false;
          if (lane == 0) mb_arrive(&sh.v_empty[vt % NV]);
        }
        return true;
      };
      auto scores = [&](int k) {
        const int sb = k & 1;
        const uint32_t t = tiles_before + (both ? k >> 1 : k), slot = t % NK;
        if (!pass_keys(t) || !warp_wait(&keys[slot], (t / NK) & 1u)) return false;
        ++kt;
        tc_fence_after();
        const uint64_t kd = rows_desc<S::SW>(sbase + S::OFF_K + slot * S::KTILE);
        if constexpr (E4M3) {
#pragma unroll
          for (int x = 0; x < 2 * (D / 64); ++x) {  // both parts of the queries
            const int part = x / (D / 64), y = x % (D / 64);  // 64 dimensions
            mma2_scores_e4m3(tmem + sb * S::S_COLS, qd + (part * (128 * D) + y * 64 / S::SW * (128 * S::SW) + y * 64 % S::SW) / 16,
                             kd + (y * 64 / S::SW * (TN * S::SW) + y * 64 % S::SW) / 16, id_s, x > 0);
          }
        } else {
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            mma4_scores(tmem + sb * S::S_COLS, qd + x * (128 * 128 / 16), kd + x * (TN * 128 / 16), id_s, x > 0);
        }
        commit(&sh.s_full[sb]);
        commit(&sh.k_empty[slot]);
        return true;
      };
      bool ok = true;
      if (st < K) {
        ok = warp_wait(&sh.q_ready[st], asked & 1u);
        ++asked;
        // of a longer item the second stream starts half a step behind, so that one's products meet the other's softmax
        const bool skew = NS == 2 && K > 8;
        if (st == 1 && skew) ok = ok && warp_wait(&sh.go, goes & 1u);
        goes += skew;
#pragma unroll 1
        for (int k = st - 2; ok && k < K; k += NS) {  // (k < 0: the first scores, of one buffer or of both)
          if (k >= 0) {
            const int sb = k & 1;
            const uint32_t t = tiles_before + (both ? k >> 1 : k), slot = t % NV;
            const uint64_t vd = values_desc(sbase + S::OFF_V + slot * S::TILE, TN * 128);
            const uint32_t od = tmem + S::O_COL + st * S::O_COLS, pa = tmem + sb * S::S_COLS;
            ok = pass_values(t) && warp_wait(&sh.v_ready[slot], (t / NV) & 1u);
            ++vt;
#pragma unroll
            for (int h = 0; h < TN / 64; ++h) {  // weights of 64 places
              ok = ok && warp_wait(h + 1 < TN / 64 ? &sh.p_half[sb] : &sh.p_ready[sb], uses[sb] & 1u);
              if (!ok) break;
              tc_fence_after();
              if (skew && k == 0 && h == 0 && lane == 0) mb_arrive(&sh.go);
              mma4_values(od, pa + h * 32, vd + h * (8192 / 16), id_o, h > 0 || k >= NS);
              if (h + 1 < TN / 64) commit(&sh.half_done[sb]);
            }
            if (!ok) break;
            ++uses[sb];
            // (E4M3: the next values are converted meanwhile, 4 % of a long tree; bf16: no difference to the copies)
            if (E4M3) commit(&sh.v_empty[slot]);
            if (k + 2 < K) ok = scores(k + 2);
            if (!E4M3) commit(&sh.v_empty[slot]);
            if (NS == 1 || k + NS >= K) commit(&sh.pv_done[sb]);
          } else if (k + 2 < K) {
            ok = scores(k + 2);
          }
        }
      }
      tiles_before += T;
      if (!ok || !pass_keys(tiles_before) || !pass_values(tiles_before)) {
        timeout = true;
        break;
      }
      item_done(items);
    }
  } else if (warp == 9) {
    // ---- items, and their loads
    uint32_t kt = 0, vt = 0, rt = 0, seq = 0, items = 0;
    const int page_size = 1 << P.page_shift, run = min(page_size, TN), runs = TN / run;
    constexpr int EB = E4M3 ? 1 : 2, BOX = D * EB < 128 ? D * EB : 128, BOXES = D * EB / BOX;  // bytes of a box's rows
    Walk<TN, ROWS> it;
    if (P.parts)
      it.direct(P, blockIdx.x);
    else
      it.init(P, blockIdx.x);
#pragma unroll 1
    for (;; ++items) {
      if (items >= 4 && !warp_wait(&sh.item_empty[items & 3], ((items >> 2) & 1u) ^ 1u)) timeout = true;
      if (timeout) break;
      if (lane == 0) {
        AxItem &I = sh.item[items & 3];
        if (it.more)
          it.show(P, I);
        else
          I.rows = 0;
        mb_arrive(&sh.item_full[items & 3]);
      }
      if (!it.more) break;
#pragma unroll 1
      for (int u = it.u0; u < it.u1 && !timeout; ++u, ++seq) {
        const int tile = it.list.tile(u);
        uint32_t lost = 0;
        int page = P.pages;  // (past the end: the copy fills in zeros)
        if (lane < runs) {
          const int place = tile * TN + lane * run;
          if (it.list.needs(it.s, place, run)) {
            page = page_of(P, it.b, place);
            if (!is_page(P, page)) {
              set_status(P.status, K3MOE_DEV_BOUNDS);
              page = P.pages;
              lost = below(run / 16) << (lane * run / 16);
            }
          }
        }
        lost = __reduce_or_sync(0xFFFFFFFFu, lost);
        const bool scales = E4M3 && page < P.pages;
        const int scaled = __popc(__ballot_sync(0xFFFFFFFFu, lane < runs && scales));
        const int at = (tile * TN + lane * run) & (page_size - 1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t *full, *empty;
          uint32_t dst, phase, bytes = 0;  // (bytes: where the scales go)
          if (kv == 0) {
            const uint32_t slot = kt % NK;
            phase = kt / NK, empty = &sh.k_empty[slot], full = &sh.k_full[slot];
            dst = sbase + S::OFF_K + slot * S::KTILE;
            if (E4M3) bytes = su32(sh.key_bytes[slot]);
            ++kt;
          } else if constexpr (E4M3) {
            const uint32_t slot = rt % NR;
            phase = rt / NR, empty = &sh.r_empty[slot], full = &sh.r_full[slot];
            dst = sbase + S::OFF_R + slot * S::RAWB, bytes = dst + TN * D;
            ++rt;
          } else {
            const uint32_t slot = vt % NV;
            phase = vt / NV, empty = &sh.v_empty[slot], full = &sh.v_full[slot];
            dst = sbase + S::OFF_V + slot * S::TILE;
            ++vt;
          }
          if (!warp_wait(empty, (phase & 1u) ^ 1u)) {
            timeout = true;
            break;
          }
          if (lane == 0) {
            if (kv == 0) sh.lost[seq & 15] = lost;
            mb_arrive_tx(full, TN * D * EB + (E4M3 ? scaled * run : 0));
          }
          __syncwarp();
          if (lane < runs) {
#pragma unroll
            for (int x = 0; x < BOXES; ++x)
              tma_load_4d(dst + x * (TN * BOX) + lane * (run * BOX), kv ? &vmap : &kmap, x * (BOX / EB), at, it.head, page, full);
            if (scales)
              bulk_load(bytes + lane * run,
                        (kv ? P.vs : P.ks) + (((static_cast<size_t>(page) * P.heads + it.head) << P.page_shift) + at), run, full);
          }
        }
      }
      if (P.parts)
        it.more = false;
      else
        it.next(P);
    }
    // every copy has landed before the block can leave
    if (timeout) {
      if constexpr (E4M3) {
        for (uint32_t i = rt < NR ? 0 : rt - NR; i < rt; ++i) mb_wait(&sh.r_full[i % NR], (i / NR) & 1u);
      } else {
        for (uint32_t i = vt < NV ? 0 : vt - NV; i < vt; ++i) mb_wait(&sh.v_full[i % NV], (i / NV) & 1u);
      }
      for (uint32_t i = kt < NK ? 0 : kt - NK; i < kt; ++i) mb_wait(&sh.k_full[i % NK], (i / NK) & 1u);
    }
  } else if (E4M3 && warp == 11) {
    // ---- the keys' scales as numbers
    uint32_t kt = 0;
    const AxItem *I;
    for (uint32_t items = 0; !timeout && (I = item_at(items)) != nullptr; ++items) {
      for (const uint32_t end = kt + I->u1 - I->u0; kt < end; ++kt) {
        if (!warp_wait(&sh.k_full[kt % NK], (kt / NK) & 1u)) {
          timeout = true;
          break;
        }
#pragma unroll
        for (int x = lane; x < TN; x += 32) sh.key_scale[kt & 7][x] = e8m0_to_f32(sh.key_bytes[kt % NK][x]);
        __syncwarp();
        if (lane == 0) mb_arrive(&sh.k_ready[kt % NK]);
      }
      item_done(items);
    }
  } else if (warp >= 12) {
    // ---- values: codes become bf16 operands, and what a row does not see must not be other than finite
    const int t128 = tid - 384;
    uint32_t vt = 0;
    const AxItem *ip;
    for (uint32_t items = 0; !timeout && (ip = item_at(items)) != nullptr; ++items) {
      const AxItem &I = *ip;
      if (t128 == 0) atomicAnd(&sh.odd, ~(1u << ((items + 16) & 31)));
#pragma unroll 1
      for (int u = I.u0; u < I.u1; ++u, ++vt) {
        const int tile = I.tile(u);
        const uint32_t slot = vt % NV, rs = vt % NR;
        if (!(E4M3 ? warp_wait(&sh.r_full[rs], (vt / NR) & 1u) && warp_wait(&sh.v_empty[slot], ((vt / NV) & 1u) ^ 1u)
                   : warp_wait(&sh.v_full[slot], (vt / NV) & 1u))) {
          timeout = true;
          break;
        }
        const uint32_t lost = sh.lost[vt & 15];
        // (where all rows see the whole tile, or what of it lies in pages of the cache, nothing has to be left out)
        const bool some = masked<TN>(P, I, tile), check = lost || some;
        uint8_t *const op = smem + S::OFF_V + slot * S::TILE;
        if constexpr (E4M3) {
          // A lane takes 16 codes of a row; eight neighbouring lanes take four times 16 of one row and the next four of
          // another, so that neither their loads nor their stores meet in a bank
          const uint8_t *raw = smem + S::OFF_R + rs * S::RAWB, *scales = raw + TN * D;
          constexpr int BOX = D < 128 ? D : 128, RW = D == 64 ? 8 : D == 128 ? 4 : 2;  // rows of a warp
          const int h = (lane >> 2) & 1, p = lane >> 3, w = warp - 12;
          const int rr0 = D == 64 ? lane >> 2 : D == 128 ? 2 * (p >> 1) + h : h;
          const int blk = D == 64 ? 0 : D == 128 ? (p & 1) ^ h : p ^ h;  // of 64 dimensions
          const int ch = 4 * blk + (lane & 3);
          const uint8_t *from = raw + (ch * 16 / BOX) * (TN * BOX) + (ch * 16) % BOX;
          uint8_t *to = op + blk * (TN * 128);
          const int c0 = 2 * (lane & 3);
#pragma unroll 2
          for (int rr = w * RW + rr0; rr < TN; rr += 4 * RW) {
            const uint4 in = *reinterpret_cast<const uint4 *>(from + rr * BOX);
            const uint32_t byte = scales[rr];
            const uint32_t cw[4] = {in.x, in.y, in.z, in.w};
            uint32_t hv[8];
            // 2^(byte - 127 + 120), or as much of it as bf16 holds
            const uint32_t f = (byte <= 134u ? (byte + 120u) << 7 : byte == 255u ? 0x7FC0u : 0x7F00u) * 0x10001u;
            uint32_t rare = byte > 134u ? 0x80808080u : 0u;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              rare |= (cw[y] & 0x7F7F7F7Fu) + 0x01010101u;  // (a NaN's code)
              hv[2 * y] = mul_bf16x2(codes_up(cw[y], 0x1404), f);
              hv[2 * y + 1] = mul_bf16x2(codes_up(cw[y], 0x3424), f);
            }
            uint8_t *row = to + rr * 128;
            const uint32_t a0 = (c0 ^ (rr & 7)) << 4, a1 = ((c0 + 1) ^ (rr & 7)) << 4;
            *reinterpret_cast<uint4 *>(row + a0) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            *reinterpret_cast<uint4 *>(row + a1) = make_uint4(hv[4], hv[5], hv[6], hv[7]);
            if (rare & 0x80808080u) {  // code by code
              const float x = e8m0_to_f32(byte);
#pragma unroll 1
              for (int y = 0; y < 16; ++y) {
                uint32_t a, z;
                e4m3x4_to_f16x2(from[rr * BOX + y], a, z);
                reinterpret_cast<uint16_t *>(row + (y < 8 ? a0 : a1))[y & 7] =
                    static_cast<uint16_t>(bf16x2(__half2float(__ushort_as_half(static_cast<unsigned short>(a))) * x, 0.f));
              }
            }
          }
          __syncwarp();
          if (lane == 0) mb_arrive(&sh.r_empty[rs]);
        }
        if (check) {
          // Places that no row sees become zeros; others that are not finite are left out, and remembered.  (Each warp its
          // own rows: in the E4M3 case those that it has converted.)
          constexpr int CH = D / 8, RW = D == 64 ? 8 : D == 128 ? 4 : 2, U = 4;
#pragma unroll 1
          for (int x0 = lane; x0 < TN / 4 * CH; x0 += 32 * U) {
            uint4 *at[U], was[U];
            bool there[U];
#pragma unroll
            for (int y = 0; y < U; ++y) {
              const int x = x0 + 32 * y, q = x / CH, ch = x % CH;
              const int rr = q / RW * (4 * RW) + (warp - 12) * RW + q % RW, place = tile * TN + rr, g16 = place & ~15;
              at[y] = reinterpret_cast<uint4 *>(op + (ch / 8) * (TN * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
              there[y] = place < I.n && (g16 + 16 > I.lo || g16 < I.sinks) && !(lost >> ((place % TN) / 16) & 1u);
              was[y] = *at[y];
            }
#pragma unroll
            for (int y = 0; y < U; ++y) {
              uint32_t hv[4] = {was[y].x, was[y].y, was[y].z, was[y].w}, odd = 0;
#pragma unroll
              for (int z = 0; z < 4; ++z) odd |= (hv[z] & 0x7F807F80u) + 0x00800080u;
              if (!there[y]) {
                *at[y] = make_uint4(0, 0, 0, 0);
              } else if (some && (odd & 0x80008000u)) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  if ((hv[z] & 0x7F80u) == 0x7F80u) hv[z] &= 0xFFFF0000u;
                  if ((hv[z] & 0x7F800000u) == 0x7F800000u) hv[z] &= 0xFFFFu;
                }
                *at[y] = make_uint4(hv[0], hv[1], hv[2], hv[3]);
                atomicOr(&sh.odd, 1u << (items & 31));
              }
            }
          }
        }
        if (E4M3 || check) fence_async();
        __syncwarp();
        if (lane == 0) mb_arrive(&sh.v_ready[slot]);
      }
      item_done(items);
    }
  }
  if (timeout) set_status(P.status, K3MOE_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Adds the parts of an item that was cut, in the order of their pieces: block (x, y, z) joins 32 dimensions of 32 rows of the
// item that begins in piece x (direct: of item x).  Bound by the sums' bytes, read once from L2: out = sum_p o_p 2^(m_p - m) over
// the same of l.  18 MB of a tree on 16000 tokens in 9 parts: 12 us cold, 8 beside the rest.  kJoinParts parts are loaded at once (one after the other, nine of them
// took 20 us).
template <int D, int ROWS>
__global__ void __launch_bounds__(128) attn_extend_join_kernel(const AxParams P) {
  __shared__ float s_f[kAxMostBlocks][32];  // the parts' factors
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  int4 me;
  if (P.parts) {
    const int e = blockIdx.x / P.heads;
    int t = 0;
    const int b = sequence_of<ROWS>(P, e, t);
    me = make_int4(b, blockIdx.x - e * P.heads, t, b < 0 ? 0 : P.parts);
  } else {
    me = P.meta[blockIdx.x];
  }
  const int parts = me.w;
  if (parts < 2) return;
  const Seq s = seq_of(P, me.x, false);
  const int r0 = me.z * ROWS, rows = min(ROWS, s.m * P.G - r0), r = 32 * blockIdx.y + lane;
  if (32 * static_cast<int>(blockIdx.y) >= rows) return;
  auto slot_of = [&](int p) {
    return static_cast<size_t>(P.parts ? parts * blockIdx.x + p : p == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + p));
  };
  float mm = -INFINITY, l = 0.f;
  for (int p0 = 0; p0 < parts; p0 += kJoinParts) {
    float2 st[kJoinParts];
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x)
      st[x] = p0 + x < parts ? P.stat[slot_of(p0 + x) * ROWS + r] : make_float2(kNone, 0.f);
    float top = mm;
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) top = fmaxf(top, st[x].x);
    const float base = top == -INFINITY ? 0.f : top;
    l *= ex2(mm - base);
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) {
      if (st[x].x != kNone) l = fmaf(st[x].y, ex2(st[x].x - base), l);
      if (p0 + x < parts && (x & 3) == warp) s_f[p0 + x][lane] = st[x].x;
    }
    mm = top;
  }
  __syncthreads();
  const float base = mm == -INFINITY ? 0.f : mm;
  const int x0 = 32 * blockIdx.z + 8 * warp;
  float o[8];
#pragma unroll
  for (int y = 0; y < 8; ++y) o[y] = 0.f;
  for (int p0 = 0; p0 < parts; p0 += kJoinParts) {
    float u[kJoinParts][8], f[kJoinParts];
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) {
      f[x] = p0 + x < parts ? s_f[p0 + x][lane] : kNone;
      const float *from = P.part + (slot_of(p0 + x < parts ? p0 + x : 0) * D + x0) * ROWS + r;
#pragma unroll
      for (int y = 0; y < 8; ++y) u[x][y] = f[x] == kNone ? 0.f : from[y * ROWS];
    }
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) {
      const float g = ex2(f[x] - base);
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = fmaf(u[x][y], g, o[y]);
    }
  }
  if (r >= rows) return;
  const int i = (r0 + r) / P.G, g = r0 + r - i * P.G;
  const size_t row = (static_cast<size_t>(s.first) + i) * P.Hq + me.y * P.G + g;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t w[4];
#pragma unroll
  for (int z = 0; z < 4; ++z) w[z] = l == 0.f ? 0u : bf16x2(o[2 * z] * inv, o[2 * z + 1] * inv);
  *reinterpret_cast<uint4 *>(P.out + row * D + x0) = make_uint4(w[0], w[1], w[2], w[3]);
  if (P.lse && x0 == 0) P.lse[row] = l == 0.f ? -INFINITY : (mm + log2f(l)) * kLn2;
}

namespace {

int entries_of(int item, int B, int rows, int G) {
  return static_cast<int>(static_cast<long long>(rows) * G / item + B);
}
size_t aligned256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct AxSpace {
  size_t plan, start, meta, first_entry, prefix, stat, part, bytes;
};
AxSpace space_of(const k3moe_kv_cache &c, int B, int rows, int Hq) {
  const int item = c.dim == 256 ? 128 : 256;
  const size_t entries = static_cast<size_t>(entries_of(item, B, rows, Hq / c.heads)) + 1;
  AxSpace s;
  s.plan = 0;
  s.start = 256;
  s.meta = s.start + aligned256(kAxMostBlocks * sizeof(AxStart));
  s.first_entry = s.meta + aligned256(kAxMostBlocks * sizeof(int4));
  s.prefix = s.first_entry + aligned256((static_cast<size_t>(B) + 1) * 4);
  s.stat = s.prefix + aligned256(entries * 8);
  s.part = s.stat + aligned256(2 * kAxMostBlocks * item * sizeof(float2));
  s.bytes = s.part + static_cast<size_t>(2) * kAxMostBlocks * item * c.dim * 4;
  return s;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Boxes of 128 bytes (or a row) by min(page_size, TN) places of one head of a page.
bool cache_map(CUtensorMap *m, const k3moe_kv_cache &c, void *base, int TN, bool swizzle) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const bool e = c.format == K3MOE_KV_E4M3;
  const cuuint64_t row = static_cast<cuuint64_t>(c.dim) * (e ? 1 : 2);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {row, row * c.page_size, row * c.page_size * c.heads};
  const cuuint32_t inner = static_cast<cuuint32_t>(e ? (c.dim < 128 ? c.dim : 128) : 64);
  const cuuint32_t box[4] = {inner,
                             static_cast<cuuint32_t>(c.page_size < TN ? c.page_size : TN), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn(m, e ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : e && inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

template <int D, bool E4M3>
int launch_extend(const k3moe_kv_cache &c, AxParams &P, cudaStream_t st) {
  using S = AxShape<D, E4M3>;
  static_assert(S::SMEM <= 232448, "shared memory of a block");
  CUtensorMap kmap, vmap;
  if (!cache_map(&kmap, c, c.k, S::TN, true) || !cache_map(&vmap, c, c.v, S::TN, !E4M3)) return -1;
  static PerDevice raised;
  cudaError_t err = cudaSuccess;
  raised.get(current_device(), [&] {
    err = cudaFuncSetAttribute(attn_extend_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    return err == cudaSuccess ? 1 : -1;
  });
  if (err != cudaSuccess) return -1;
  P.blocks = min(sm_count(), kAxMostBlocks);
  P.entries = entries_of(S::ROWS, P.B, P.rows, P.G);
  P.per_head = static_cast<uint32_t>(((1ULL << 32) + P.G - 1) / P.G);
  // No more items than SMs: a block each, or several where a sequence may be long; no plan, and mostly no joint.
  const long long items = static_cast<long long>(P.entries) * P.heads;
  P.parts = 0;
  if (items <= P.blocks) {
    // (Not where parts are long, past 12 tiles, and the items that there must be fill less than 17 of 20 blocks: a plan shares
    // them evenly.  Direct and planned: 4 sequences of 60 on 20000, 32 / 4 heads, E4M3, 166 and 127 us; 8 ragged ones 66 and
    // 59; 7 of 13, 256 wide, bf16, 68 and 58; but 2 of 200 on 8000, 32 / 4, bf16, 87 and 102.  Short parts: one of 60 on 16000,
    // 64 / 8, E4M3, 67 and 73; 2 of 60 on 4000 42 and 49; 3 of 100 on 1000 33 and 42.)
    const long long visible = static_cast<long long>(P.max_pages) << P.page_shift;
    const long long seen = P.window > 0 ? min(visible, static_cast<long long>(P.window) + P.sinks + S::ROWS / P.G) : visible;
    P.parts = static_cast<int>(max(1LL, min(P.blocks / items, seen / (kPartTiles * S::TN))));
    const long long real = P.heads * max(static_cast<long long>(P.B), (static_cast<long long>(P.rows) * P.G + S::ROWS - 1) / S::ROWS);
    if (seen > 12LL * S::TN * P.parts && real * P.parts * 20 < 17LL * P.blocks) P.parts = 0;
  }
  if (!P.parts && launch_pdl(attn_plan_kernel<S::TN, S::ROWS>, dim3(1), dim3(1024), 0, st, P) != cudaSuccess) return -1;
  const int blocks = P.parts ? static_cast<int>(items) * P.parts : P.blocks;
  if (launch_pdl(attn_extend_kernel<D, E4M3>, dim3(blocks), dim3(kAxThreads), S::SMEM, st, P, kmap, vmap) != cudaSuccess)
    return -1;
  if (P.parts == 1) return 0;
  return launch_pdl(attn_extend_join_kernel<D, S::ROWS>, dim3(P.parts ? items : blocks, S::ROWS / 32, D / 32), dim3(128), 0, st, P) ==
                 cudaSuccess
             ? 0
             : -1;
}

}  // namespace

namespace {
// Which kernels take the call: those of few columns (attn_rows.cu), of tiles, or both.  The former read a sequence's keys
// and values once for each 16 rows of a head, with little to start and end; those of tiles once for 256 (128 at dim 256), but
// take 9 to 25 us whatever the work.  So the former where each 16 rows have an SM and read little in all; and where a
// sequence has about 16 rows a head, taken over the batch.  Measured where the two meet (128 wide, 8 query heads a key):
//   16 items, E4M3   30000 tokens  37 and 50 us        128 items, E4M3   1000 tokens  19 and 27 us
//   32                6000         22     34                             6000         55     42
//                    30000         62     52             128, bf16       100           8     16
//   64                6000         36     36                             1000         26     21
// Other widths go by the bytes (E4M3): 16 items on 30000, 64 wide, 39 and 60 us, 256 wide 128 and 118; 64 items on 6000 29
// and 36, 100 and 69; 256 items on 1000, which are the tiles', 23 and 27, 42 and 65.
// One sequence of such a batch may have many rows, a prompt beside single tokens.  Where the host's bounds allow that its
// reads by 16 rows pass kApart bytes, both kinds are launched, and each sequence is its rows' kind's.  255 single tokens on
// 1000 and a prompt of 3800, 96 / 96 heads, E4M3: 11630 us in columns, 3890 in tiles, 2170 in both; 32 / 32 heads, bf16: 5620,
// 1260, 940; a prompt of 257 beside tokens on 4000, 64 / 8 heads, E4M3: 725, 1050, 507.  Launches without work cost 18 us
// (256 sequences of 2 tokens on 2000 with max_new left at all rows 285 and 307).
enum class Ways { kFew, kTiles, kBoth };
constexpr double kApart = 1e9;
// (kBoth) Most rows a head of a sequence in columns.  56 sequences of 40 rows beside 200 of 8: 686 us in columns, 601 so; 250 single
// tokens of 64 / 4 heads on 2000: 561 and 410, of 128 / 1 heads of 256 in bf16 on 3000: 233 and 232.
constexpr int kFewRows = 32;
Ways ways_of(const ExtendArgs &a) {
  const k3moe_kv_cache &c = a.c;
  const long long G = a.Hq / c.heads, columns = a.rows * G;
  const long long items = c.heads * max(static_cast<long long>(a.B), (columns + 15) / 16);
  const long long places = static_cast<long long>(a.max_pages) * c.page_size;
  const long long seen = a.window > 0 ? min(places, static_cast<long long>(a.window) + a.sinks + a.max_new) : places;
  const bool e = c.format == K3MOE_KV_E4M3;
  const double bytes = static_cast<double>(seen) * 2 * c.dim * (e ? 1 : 2);  // of an item
  if (items <= sm_count() && items * bytes <= (e ? 64e6 : 38e6) * (1 + 48.0 / items)) return Ways::kFew;
  if (columns > 16LL * a.B) return Ways::kTiles;
  if (static_cast<double>(a.max_new) * G / 16 * c.heads * bytes <= kApart || a.max_new * G <= kFewRows) return Ways::kFew;
  return G > kFewRows ? Ways::kTiles : Ways::kBoth;
}
}  // namespace

size_t attn_extend_workspace(const k3moe_kv_cache &c, int B, int rows, int Hq) {
  const size_t several = space_of(c, B, rows, Hq).bytes, one = attn_rows_workspace(c);
  return several > one ? several : one;
}

int launch_attn_extend(const ExtendArgs &a, cudaStream_t st) {
  if (a.max_new == 1 && !a.masks) return launch_attn_sinks(a, st);
  const Ways ways = ways_of(a);
  if (ways != Ways::kTiles) {
    const int rc = launch_attn_rows(a, ways == Ways::kBoth ? kFewRows : INT32_MAX, st);
    if (rc || ways == Ways::kFew) return rc;
  }
  AxParams P;
  const k3moe_kv_cache &c = a.c;
  P.k = static_cast<const uint8_t *>(c.k), P.v = static_cast<const uint8_t *>(c.v), P.ks = c.k_scales, P.vs = c.v_scales;
  P.heads = c.heads, P.pages = c.pages, P.page_shift = 0;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  P.B = a.B, P.rows = a.rows, P.Hq = a.Hq, P.G = a.Hq / c.heads;
  P.q = a.q, P.q_stride = a.q_stride, P.offsets = a.offsets, P.max_new = a.max_new, P.masks = a.masks, P.words = a.words;
  P.table = a.table, P.max_pages = a.max_pages, P.lens = a.lens, P.window = a.window, P.sinks = a.sinks;
  P.scale = a.scale, P.out = a.out, P.lse = a.lse, P.status = a.status;
  P.others = ways == Ways::kBoth ? kFewRows / P.G : 0;
  const AxSpace s = space_of(c, a.B, a.rows, a.Hq);
  uint8_t *w = static_cast<uint8_t *>(a.ws);
  P.plan = reinterpret_cast<AxPlan *>(w + s.plan), P.start = reinterpret_cast<AxStart *>(w + s.start);
  P.meta = reinterpret_cast<int4 *>(w + s.meta), P.first_entry = reinterpret_cast<int *>(w + s.first_entry);
  P.prefix = reinterpret_cast<long long *>(w + s.prefix), P.stat = reinterpret_cast<float2 *>(w + s.stat);
  P.part = reinterpret_cast<float *>(w + s.part);
  const bool e = c.format == K3MOE_KV_E4M3;
  if (c.dim == 64) return e ? launch_extend<64, true>(c, P, st) : launch_extend<64, false>(c, P, st);
  if (c.dim == 128) return e ? launch_extend<128, true>(c, P, st) : launch_extend<128, false>(c, P, st);
  if (c.dim == 256) return e ? launch_extend<256, true>(c, P, st) : launch_extend<256, false>(c, P, st);
  return -1;
}

}  // namespace k3moe
