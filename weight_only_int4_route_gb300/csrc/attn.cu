// Attention of new tokens over the paged cache: drafted trees (a bit mask per token) and prompts
// (causal), grouped query heads.
//
//   s_j = scale q . k_j over the visible keys j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j).
//
// One pass over the keys in tiles of 128 on the 5th-generation tensor cores, with a running
// maximum and sum per row.  The rows of a tile are 128 / group tokens times the group's query heads, so
// a K/V head is read once for all its query heads; even a single token fills the 128-row MMA with
// padding rather than take another path: per key tile the two products cost about 1100 tensor cycles,
// where an SM's share of the memory bandwidth (64 KB a tile at head_dim 128) costs 2800.
//
// Two streams run through one CTA, each with its own scores, weights and output accumulator in tensor
// memory and its own softmax warpgroup, so that one stream's products run under the other's softmax:
//   wide    two row tiles of an item, every key tile is used by both (prompts: tensor cores bound);
//   narrow  one row tile, the streams take alternate key tiles and are merged at the end (few rows
//           per sequence: memory bound).
//
// Work: an item is (sequence, row tile or pair of them, K/V head), its units are a few units of
// overhead (kItemCost) and its key tiles.  The units of all items, in order, are dealt to the CTAs in
// equal contiguous shares, whatever the lengths (which only the device knows); an item cut by a
// share's boundary leaves partial results (running maximum, sum, unscaled output) in the workspace,
// and a second kernel joins them in order.
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (thread = row = tensor memory lane), 8 copies of K and V
// (a lane per page), 9 MMA issue (one thread), 10 copies of Q (one thread; apart from 8, so that the
// next item's keys are under way while Q's buffer is still in use), 11 idle.  Tensor memory: scores
// S0 S1 (128 columns each, the weights replace the scores' first 64), outputs O0 O1 (head_dim columns
// each): all 512 columns at head_dim 128, so a stream's next scores wait for its second product.
//
// Measured on GB300 (bf16, 32 query and 8 K/V heads of 128 unless said), calls in a row:
//   prompt of 8191 tokens             400 us, 1372 TFLOP/s of visible pairs (0.71 of the measured matrix peak), the
//                                     power cap active; 376 us, 1462 TFLOP/s (0.76) in runs too short for it
//   6 prompts of 1 to 2500 tokens     217 us, 1099 TFLOP/s (0.57)
//   32 trees of 8-32 tokens over 500-8000 cached ones   106 us, 5.2 TB/s (0.77 of the measured copy rate)
//   5 trees over 30000-150000 cached tokens, f16, 16 and 8 heads of 64   157 us, 6.0 TB/s (0.88)
//   one token over 1000, 16 heads     15 us from a graph (9 + 3 us in the two kernels), all of it latency
// What bounds the wide form: the chain scores -> softmax -> weights -> product of a stream takes about 2500
// cycles, the MMAs of both streams 2050 of them; without any softmax the same loop takes 367 us.  The
// MMA thread's waits and the instruction cache (its loop beside the softmax's) make up the rest.  The narrow
// form reads each K and V once (DRAM bytes = the cache's), at 6.3 TB/s between a start of 4 us (finding the
// work, first pages) and the slowest CTA's end, up to 8% after the mean.
//
// Precision: scores, maxima, sums and the output accumulator are fp32; the weights are rounded to the cache's type,
// because a product of 16-bit values takes both operands of one type and V is of that type.  Their error is one
// rounding of each weight: 0.0022 of the output's norm against 64 bits in bf16 (0.00028 in f16), where the output's own
// rounding is 0.0017 (0.0002).  Weights in two 16-bit parts bring it down to that, with two second products: 181 instead
// of 157 us for the trees over long contexts.  The sums take the weights as they are before, and lse is exact to fp32.
//
// Every wait is bounded (see mbar_wait); when one expires the CTA records a code, drains its own copies
// and MMAs, frees its tensor memory and returns.
#include <atomic>
#include <cfloat>
#include <climits>

#include "kv_internal.cuh"
#include "tc_ptx.cuh"

namespace moe {

MOE_DEFINE_CHECK_WORD(attn)

__device__ int g_attn_error = 0;

int attn_error_take(int *out) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(int)) != cudaSuccess) return check_launch("attention error read");
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(int)) != cudaSuccess) return check_launch("attention error reset");
    *out = v;
  }
  return MOE_OK;
}

namespace {

constexpr int kThreads = 128;              // tree_mask
constexpr int kTile = 128;                 // rows of a row tile, keys of a key tile
constexpr int kSoftWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kQWarp = 10;
constexpr int kAttnThreads = 32 * 12;      // the third warpgroup: copies, MMA issue and an idle warp
// Registers: 384 threads launch with 168 each; the softmax warpgroups (a row of 128 scores per thread)
// take over what the third does not need: 2 x 224 + 56 = 3 x 168.
constexpr int kSoftRegs = 224, kOtherRegs = 56;
constexpr int kRingBytes = 128 << 10;      // K and V tiles in flight
constexpr int kCols = 32;                  // columns of the output that the epilogue handles at a time
constexpr int kStageBytes = 32 * kCols * 2;   // a softmax warp's 16-bit output rows of those columns
// The running maximum is only moved when a tile exceeds it by more than this (in powers of two):
// weights grow to at most 2^8 of the largest, sums and outputs stay exact in fp32, and the
// accumulator in tensor memory is hardly ever rescaled.
constexpr float kLazy = 8.f;
// Key tiles whose new tokens' values that are not finite are noted apart from each other (a causal item has three such
// tiles at most, a tree of 8000 tokens 64); of a longer tree, tiles this far apart share their notes, and a key that is
// looked at in vain adds nothing.
constexpr int kBadTiles = 64;
// What an item costs beside its key tiles (its queries, its first tiles' latency, its epilogue), in key
// tiles: shares are dealt with it counted in.  With 0, 2, 4 and 8 tiles: prompt of 8191 tokens 667, 443, 378 and 393 us;
// 6 prompts of 1 to 2500 338, 232, 214 and 222; 64 of 200 131, 119, 120 and 120; 32 trees of 8-32 115, 107, 106 and 107;
// 300 single tokens over 300 271, 271, 258 and 249; 5 trees over long contexts 155 to 156 with any.
// Not in calls so small that every key tile gets a CTA of its own (up to kSmallUnits units per CTA): there the longest
// share decides.  8 single tokens over 400: 16.9 us without the cost, 18.0 with it; prompt of 700 tokens,
// 16 heads of 64: 17.4 and 18.4.  From there on it turns: prompt of 1000 tokens 42.4 and 32.6, 16 single tokens over 1000
// and 16 heads 41.1 and 38.2.
constexpr int kItemCost = 4, kSmallUnits = 4;
enum : int { kErrQ = 11, kErrKv = 12, kErrS = 13, kErrP = 14, kErrO = 15, kErrX = 16, kErrDrain = 17 };

struct Rows {
  const int32_t *cu, *seqs, *start;
  const uint32_t *mask;
  uint16_t *out;
  float *lse;
  int n, T, q_heads, group, words;
  int tile_tokens;    // tokens of a row tile: 128 / group
  float scale_log2;   // scale * log2(e): the exponentials are taken to base 2
};

// One CTA's share boundary pieces, as the joining kernel finds them.  Slot 0: the end of an item that
// an earlier CTA began; slot 1: the beginning of an item that a later CTA ends.
struct Piece {
  int32_t valid, seq, tile, head, pieces, pad0, pad1, pad2;
};

struct Workspace {
  Piece *piece;       // [2 grid]
  float2 *ml;         // [2 grid][rows]: running maximum (to base 2), sum
  float *o;           // [2 grid][head_dim][rows]
};

// ---------------------------------------------------------------- work

__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {   // a, b >= 0; the short form where both fit
  return ((a | b) >> 31) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// sum_{i < n} floor((step i + b) / 128).  Steps that divide 128 or are multiples of it (group sizes that are
// powers of two) have a closed form; else by swapping the roles of the axes as in Euclid's
// algorithm.
__device__ int64_t floor_sum(int64_t n, int step, int64_t b) {
  if (step % kTile == 0) return int64_t(step / kTile) * (n * (n - 1) / 2) + n * (b / kTile);
  if ((step & (step - 1)) == 0) {   // floor((step i + b) / 128) = floor((i + floor(b / step)) / q), q = 128 / step
    const int sh = 31 - __clz(kTile / step);
    auto first = [&](int64_t x) {   // sum_{i < x} floor(i / q)
      const int64_t a = x >> sh;
      return ((a * (a - 1)) << sh) / 2 + a * (x - (a << sh));
    };
    const int64_t b0 = b >> (31 - __clz(step));
    return first(b0 + n) - first(b0);
  }
  int64_t sum = 0, m = kTile, a = step;
  while (n > 0) {
    if (a >= m) {
      sum += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// A sequence of the call: its rows and how far they look.
struct Seq {
  int row0, nq;       // first packed row, new tokens
  int slot;           // table row (clamped; a skipped sequence has keys == 0)
  int start, keys;    // cached tokens before the new ones; keys in the cache
  int tiles;          // row tiles (of items)
};
__device__ __forceinline__ Seq load_seq(const KvView &c, const Rows &r, int tokens, int b) {
  Seq s;
  const int r0 = min(max(__ldg(r.cu + b), 0), r.T), r1 = min(max(__ldg(r.cu + b + 1), 0), r.T);
  s.row0 = r0;
  s.nq = max(r1 - r0, 0);
  const int slot = __ldg(r.seqs + b), st = __ldg(r.start + b);
  const int64_t room = int64_t(c.max_pages) << c.page_shift;   // < 2^28
  const bool ok = slot >= 0 && slot < c.slots && st >= 0 && st <= room;
  s.slot = ok ? slot : 0;
  s.start = ok ? st : 0;
  s.keys = ok ? int(min(int64_t(st) + s.nq, room)) : 0;
  s.tiles = (s.nq + tokens - 1) / tokens;
  return s;
}
// Key tiles of item row tile m.
__device__ __forceinline__ int key_tiles(const Rows &r, const Seq &s, int tokens, int m) {
  if (s.keys == 0) return 1;   // a skipped sequence: one tile that nobody sees
  return r.mask ? (s.start + s.nq + kTile - 1) / kTile : (s.start + min(s.nq, (m + 1) * tokens) + kTile - 1) / kTile;
}
// Key tiles of item row tiles 0 .. m - 1 together.
__device__ __forceinline__ int64_t key_tiles_before(const Rows &r, const Seq &s, int tokens, int m) {
  if (s.keys == 0) return m;
  if (r.mask) return int64_t(m) * ((s.start + s.nq + kTile - 1) / kTile);
  const int full = min(m, s.tiles - 1);   // the last tile may have fewer tokens
  int64_t n = full > 0 ? floor_sum(full, tokens, int64_t(s.start) + tokens + kTile - 1) : 0;
  if (m > full) n += key_tiles(r, s, tokens, s.tiles - 1);
  return n;
}

// Exclusive prefix sums of two values over the first kPlaceThreads threads of the block (whole warps, which alone
// call it); returns the totals.
constexpr int kPlaceThreads = 256;
__device__ __forceinline__ void place_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kPlaceThreads) : "memory"); }
struct Pair64 {
  int64_t a, b;
};
__device__ __forceinline__ Pair64 block_scan_pair(Pair64 v, Pair64 *before, Pair64 *scratch /*[32]*/) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = kPlaceThreads / 32;
  Pair64 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o);
    if (lane >= o) {
      x.a += a;
      x.b += b;
    }
  }
  if (lane == 31) scratch[warp] = x;
  place_sync();
  Pair64 base = {0, 0}, total = {0, 0};
  for (int w = 0; w < nw; ++w) {
    if (w < warp) base = {base.a + scratch[w].a, base.b + scratch[w].b};
    total = {total.a + scratch[w].a, total.b + scratch[w].b};
  }
  place_sync();
  *before = {base.a + x.a - v.a, base.b + x.b - v.b};
  return total;
}

// The CTA's place in the work.
struct Place {
  int64_t units, unit0;   // its units, the first of them counted over all
  int64_t share;          // units per CTA; the first `more` CTAs have one more
  int more, cost;         // cost: units of overhead per item
  int seq, tile, head, in_item;   // in_item: units of the first item that belong to earlier CTAs
  // the CTA whose share holds unit u
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t cut = more * (share + 1);
    return int(u < cut ? div64(u, share + 1) : more + div64(u - cut, share));
  }
};

// The first kPlaceThreads threads call it; sh is shared, and complete after the next barrier of the block.
__device__ void find_place(const KvView &c, const Rows &r, int tokens, Place *sh, Pair64 *scratch) {
  const int tid = threadIdx.x, nt = kPlaceThreads, H = c.kv_heads;
  auto count = [&](int b) -> Pair64 {   // key tiles and items of sequence b
    if (b >= r.n) return {0, 0};
    const Seq s = load_seq(c, r, tokens, b);
    return {s.nq > 0 ? H * key_tiles_before(r, s, tokens, s.tiles) : 0, int64_t(H) * s.tiles};
  };
  Pair64 v = {0, 0}, before = {0, 0}, total = {0, 0};
  for (int b0 = 0; b0 < r.n; b0 += nt) {
    v = count(b0 + tid);
    const Pair64 sum = block_scan_pair(v, &before, scratch);
    total = {total.a + sum.a, total.b + sum.b};
  }
  const int cost = total.a + kItemCost * total.b > int64_t(kSmallUnits) * gridDim.x ? kItemCost : 0;
  const int64_t units = total.a + cost * total.b, grid = min(int64_t(gridDim.x), max(units, int64_t(1)));
  const int64_t share = div64(units, grid), cta = blockIdx.x;
  const int more = int(units - share * grid);
  const int64_t u0 = share * cta + min(cta, int64_t(more)), mine = cta < grid ? share + (cta < more ? 1 : 0) : 0;
  if (tid == 0) {
    sh->units = mine;
    sh->unit0 = u0;
    sh->share = share;
    sh->more = more;
    sh->cost = cost;
  }
  if (mine > 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < r.n; b0 += nt) {
      Pair64 sum = total;
      if (r.n > nt) {   // one round of threads covers the usual call: its scan is still in registers
        v = count(b0 + tid);
        sum = block_scan_pair(v, &before, scratch);
      }
      const int64_t at = base + before.a + cost * before.b;
      if (u0 >= at && u0 < at + v.a + cost * v.b) {
        const int b = b0 + tid;
        const Seq s = load_seq(c, r, tokens, b);
        int64_t off = u0 - at;
        auto units_before = [&](int m) { return H * (key_tiles_before(r, s, tokens, m) + int64_t(cost) * m); };
        int lo = 0, hi = s.tiles - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (units_before(mid) <= off) lo = mid;
          else hi = mid - 1;
        }
        off -= units_before(lo);
        const int len = key_tiles(r, s, tokens, lo) + cost;
        sh->seq = b;
        sh->tile = lo;
        sh->head = int(div64(off, len));
        sh->in_item = int(off - int64_t(sh->head) * len);
      }
      base += sum.a + cost * sum.b;
    }
  }
}

// Walks the pieces of items in the CTA's share; every warp walks the same way.  The walk lives in shared
// memory, one per warp: a softmax thread needs its registers for a row of scores.
struct Walk {
  int64_t left, unit;       // units left, first unit of the present piece
  int seq, tile, head;
  int in_item, take;        // the piece: units [in_item, in_item + take) of the item
  int t0, cnt, total;       // its key tiles [t0, t0 + cnt) of the item's total
  Seq s;
  int n, heads, tokens, cost;
  __device__ void begin(const KvView &c, const Rows &r, int tokens_, const Place &p) {
    left = p.units;
    unit = p.unit0;
    seq = p.seq;
    tile = p.tile;
    head = p.head;
    in_item = p.in_item;
    n = r.n;
    heads = c.kv_heads;
    tokens = tokens_;
    cost = p.cost;
    if (left > 0) {
      s = load_seq(c, r, tokens, seq);
      open(r);
      if (cnt == 0) next(c, r);   // the share's first units are overhead only
    }
  }
  __device__ __forceinline__ void open(const Rows &r) {
    total = key_tiles(r, s, tokens, tile);
    take = int(min(int64_t(total + cost - in_item), left));
    t0 = max(in_item - cost, 0);
    cnt = max(in_item + take - cost, 0) - t0;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && cnt == total; }
  __device__ void next(const KvView &c, const Rows &r) {
    left -= take;
    unit += take;
    if (left <= 0) return;
    in_item = 0;
    if (++head == heads) {
      head = 0;
      if (++tile >= s.tiles) {
        tile = 0;
        do {
          ++seq;
          s = load_seq(c, r, tokens, seq);
        } while (s.nq == 0 && seq + 1 < n);
      }
    }
    open(r);
    if (cnt == 0) left = 0;   // only a share's last units can be overhead alone: the item is the next CTA's
  }
  // The first key tile that some row of stream st does not see whole.
  __device__ __forceinline__ int edge(const Rows &r, bool wide, int st) const {
    if (s.keys == 0) return 0;
    return (r.mask ? s.start : min(s.start + tile * tokens + (wide ? st * r.tile_tokens : 0) + 1, s.keys)) / kTile;
  }
  // Key tiles of stream st in this piece.  wide: the row tile's own limit; narrow: alternate tiles.
  __device__ __forceinline__ int stream_tiles(const Rows &r, bool wide, int st) const {
    if (!wide) return (cnt + 1 - st) >> 1;
    const int tok0 = tile * tokens + st * r.tile_tokens;
    if (tok0 >= s.nq) return 0;
    if (s.keys == 0 || r.mask) return cnt;
    const int lim = (s.start + min(s.nq, tok0 + r.tile_tokens) + kTile - 1) / kTile;
    return max(0, min(cnt, lim - t0));
  }
};

// ---------------------------------------------------------------- tensor core pieces

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return h2_as_u32(__floats2half2_rn(lo, hi));
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return h2_as_u32(__floats2bfloat162_rn(lo, hi));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 y;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

// One lane of the warp, the same one each time; the compiler knows that a single thread runs what follows and
// keeps descriptors in uniform registers, where the MMA instructions take them from.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// The 16-wide steps of head_dim of one scores tile: both operands K-major in 64-element swizzle columns (step i
// starts 32 bytes further, from the fifth on in the next 16 KB).  A whole tile's MMAs are one statement: the single
// issuing thread's instructions are what two streams' tiles wait for.  Only the descriptors' low words change: their
// address field cannot carry (shared addresses stay below 256 KB).
template <int STEPS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc, int steps) {
  static_assert(STEPS == 4 || STEPS == 8, "head_dim up to 64 or 128");
  if (steps == STEPS) {
    if constexpr (STEPS == 8)
      asm volatile(
        "{\n .reg .pred t, f;\n .reg .b32 ql, kl;\n .reg .b64 qd, kd;\n setp.ne.b32 f, 0, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.u32 ql, %1, 0;\n add.u32 kl, %3, 0;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, f;\n"
        " add.u32 ql, %1, 2;\n add.u32 kl, %3, 2;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 4;\n add.u32 kl, %3, 4;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 6;\n add.u32 kl, %3, 6;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 1024;\n add.u32 kl, %3, 1024;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 1026;\n add.u32 kl, %3, 1026;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 1028;\n add.u32 kl, %3, 1028;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 1030;\n add.u32 kl, %3, 1030;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        "}\n" ::"r"(d), "r"(uint32_t(q)), "r"(uint32_t(q >> 32)), "r"(uint32_t(k)), "r"(uint32_t(k >> 32)), "r"(idesc)
        : "memory");
    else
      asm volatile(
        "{\n .reg .pred t, f;\n .reg .b32 ql, kl;\n .reg .b64 qd, kd;\n setp.ne.b32 f, 0, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.u32 ql, %1, 0;\n add.u32 kl, %3, 0;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, f;\n"
        " add.u32 ql, %1, 2;\n add.u32 kl, %3, 2;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 4;\n add.u32 kl, %3, 4;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        " add.u32 ql, %1, 6;\n add.u32 kl, %3, 6;\n mov.b64 qd, {ql, %2};\n mov.b64 kd, {kl, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], qd, kd, %5, t;\n"
        "}\n" ::"r"(d), "r"(uint32_t(q)), "r"(uint32_t(q >> 32)), "r"(uint32_t(k)), "r"(uint32_t(k >> 32)), "r"(idesc)
        : "memory");
    return;
  }
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const uint64_t off = uint64_t(((i >> 2) * kTile * 128 + (i & 3) * 32) >> 4);
    tc_mma_ss(d, q + off, k + off, idesc, i != 0);
  }
}
// The eight 16-key steps of one output tile: weights in tensor memory, V N-major.
__device__ __forceinline__ void mma_output(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred t, p;\n .reg .b32 a, vl;\n .reg .b64 vd;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.u32 a, %1, 0;\n add.u32 vl, %2, 0;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, p;\n"
      " add.u32 a, %1, 8;\n add.u32 vl, %2, 128;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 16;\n add.u32 vl, %2, 256;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 24;\n add.u32 vl, %2, 384;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 32;\n add.u32 vl, %2, 512;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 40;\n add.u32 vl, %2, 640;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 48;\n add.u32 vl, %2, 768;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      " add.u32 a, %1, 56;\n add.u32 vl, %2, 896;\n mov.b64 vd, {vl, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [a], vd, %4, t;\n"
      "}\n" ::"r"(d), "r"(p), "r"(uint32_t(v)), "r"(uint32_t(v >> 32)), "r"(idesc), "r"(acc)
      : "memory");
}

// V tile as the B operand of the second product: N = head_dim is the contiguous direction (128-byte
// swizzled rows of 64 elements, one per key), K = keys.  Leading offset: to the next 64 elements of N;
// stride offset: to the next 8 keys.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFFu);
  d |= uint64_t((kTile * 128) >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
constexpr uint32_t kTransposeB = 1u << 16;   // instruction descriptor: B is N-major

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(su32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar))
      : "memory");
}

// A row of 128 scores, in one statement so that nothing uses a register before the wait.
__device__ __forceinline__ void tc_ld_row(uint32_t taddr, float (&v)[kTile]) {
  asm volatile(
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%128];\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, "
      "%43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, "
      "%63}, [%128 + 32];\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, "
      "%75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, "
      "%95}, [%128 + 64];\n"
      " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, "
      "%106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, "
      "%122, %123, %124, %125, %126, %127}, [%128 + 96];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]),
        "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
        "=f"(v[30]), "=f"(v[31]), "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]),
        "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]),
        "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]), "=f"(v[49]), "=f"(v[50]),
        "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]), "=f"(v[57]),
        "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]), "=f"(v[64]),
        "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
        "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]),
        "=f"(v[79]), "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]),
        "=f"(v[86]), "=f"(v[87]), "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]),
        "=f"(v[93]), "=f"(v[94]), "=f"(v[95]), "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]),
        "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]), "=f"(v[104]), "=f"(v[105]), "=f"(v[106]),
        "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]), "=f"(v[112]), "=f"(v[113]),
        "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]), "=f"(v[120]),
        "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]), "=f"(v[126]), "=f"(v[127])
      : "r"(taddr)
      : "memory");
}

// Shared memory of a CTA: Q (two row tiles, or two buffers of one), the rings of K and V tiles, the
// streams' maxima and sums for the narrow merge, the softmax warps' output staging, barriers.
template <int DP> struct Smem {
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kStages = kRingBytes / kTileBytes / 2;   // each a K tile and a V tile
  static constexpr int kQ = 0, kRing = 2 * kTileBytes, kXml = kRing + kRingBytes, kStage = kXml + 4 * kTile * 8,
                       kScratch = kStage + kSoftWarps * kStageBytes, kBar = kScratch + 32 * 16,
                       kBars = 2 + 2 + 2 * kStages + 4 * 2 + 4 + 1;
  static constexpr int kPlace = kBar + kBars * 8, kWalks = kPlace + int(sizeof(Place)),
                       kFlags = kWalks + kAttnThreads / 32 * int(sizeof(Walk));
  static constexpr int kNotes = kFlags + 16;
  static constexpr int kBytes = kNotes + 4 * kBadTiles * 16 + 1024 /* alignment */;
};
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "shared memory");
static_assert(sizeof(Place) % 8 == 0 && sizeof(Walk) % 8 == 0, "the flags follow them");

template <typename T, int DP, bool WIDE>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv, const KvView c,
                const Rows r, const uint16_t *layer_pool, const Workspace ws) {
  if (threadIdx.x == 0) {   // the maps are kernel parameters: no need to wait for the kernel before
    prefetch_map(&map_q);
    prefetch_map(&map_kv);
  }
  pdl_enter();
  using S = Smem<DP>;
  constexpr int kS = S::kStages, kTB = S::kTileBytes;
  // Copy p of a piece brings K of key tile p and V of key tile p - kLag: what the MMA thread uses together (the second
  // product of one tile, and the scores of the stream's next one), so it waits and lets go once for both.
  constexpr int kLag = WIDE ? 1 : 2;
  constexpr bool kF16 = std::is_same<T, __half>::value;
  // weights are exp2(s - max + kShift): f16 keeps small weights away from its underflow (the largest,
  // 2^(8 + 7), stays below 65504); bf16 has fp32's range
  constexpr float kShift = kF16 ? 7.f : 0.f;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  float2 *xml = reinterpret_cast<float2 *>(base + S::kXml);
  uint64_t *bar = reinterpret_cast<uint64_t *>(base + S::kBar);
  uint64_t *q_full = bar, *q_free = bar + 2, *kv_full = bar + 4, *kv_free = kv_full + kS, *s_full = kv_free + kS,
           *p_ready = s_full + 2, *o_full = p_ready + 2, *o_free = o_full + 2, *x_full = o_free + 2,
           *drain = x_full + 4;
  Pair64 *scratch = reinterpret_cast<Pair64 *>(base + S::kScratch);
  Place *place = reinterpret_cast<Place *>(base + S::kPlace);
  Walk *walks = reinterpret_cast<Walk *>(base + S::kWalks);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(base + S::kFlags);
  // keys of new tokens whose V is not finite, a bit each: [buffer][tile][4 words] (see the softmax)
  volatile uint32_t *all_notes = reinterpret_cast<volatile uint32_t *>(base + S::kNotes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + S::kFlags + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tokens = WIDE ? 2 * r.tile_tokens : r.tile_tokens;   // tokens of an item
  // warps 0-7 find the CTA's work while the others set up what every CTA needs
  if (warp < kPlaceThreads / 32) {
    find_place(c, r, tokens, place, scratch);
  } else if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  } else if (warp == kLoadWarp && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], WIDE ? 4 : 8);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_free[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&x_full[i], 2);   // the two warps with the same rows
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    ws.piece[2 * blockIdx.x].valid = 0;
    ws.piece[2 * blockIdx.x + 1].valid = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Walk &w = walks[warp];
  if (lane == 0) w.begin(c, r, tokens, *place);
  __syncwarp();
  // read anew by every role: a register kept across them would be spilled, and with shared memory taking nearly all
  // of the L1 a spilled value comes from the L2
  const volatile uint32_t *tmem_base = tmem_slot;
  if (place->units == 0) {
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(*tmem_base), "r"(512u));
    return;
  }
  const int ksteps = (c.head_dim + 15) / 16;   // 16-wide steps of head_dim that hold anything
  auto next_item = [&] {   // a whole warp's step
    __syncwarp();
    if (lane == 0) w.next(c, r);
    __syncwarp();
  };
  // a single thread's wait, and a whole warp's: there a wait that one lane gave up on has failed for all, or the lanes
  // would part between the warp's barriers and the block's
  auto wait = [&](uint64_t *b, uint32_t parity, int code) {
    return mbar_wait(b, parity & 1, abort_flag, code, &g_attn_error);
  };
  auto wait_warp = [&](uint64_t *b, uint32_t parity, int code) {
    return __all_sync(0xffffffffu, wait(b, parity, code)) != 0;
  };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ------------------------------------------------ copies: a lane per page of a tile
      const int ps = c.page_size(), per = ps < kTile ? kTile / ps : 1, box = min(ps, kTile);
      const int halves = DP / 64;
      uint32_t count = 0;
      bool ok = true;
      for (; ok && w.more(); next_item()) {
        const int cnt = w.cnt, t0 = w.t0, keys = w.s.keys, head = w.head;
        const int32_t *tab = c.table + int64_t(w.s.slot) * c.max_pages;
        // page of this lane's part of key tile j; c.pages (outside the map: reads as zero) past the keys
        auto page_of = [&](int j) -> int {
          const int key = (t0 + j) * kTile + lane * ps;
          if (j >= cnt || lane >= per || key >= keys) return c.pages;
          const int p = __ldg(tab + (key >> c.page_shift));
          if (p >= 0 && p < c.pages) return p;
          if (MOE_CHECKED) check_fail(kCheckPage);
          return c.pages;
        };
        int page = page_of(0), page1 = c.pages, page2 = c.pages;   // of key tiles p, p - 1, p - 2
        for (int p = 0; p < cnt + kLag; ++p, ++count) {
          const uint32_t s = count % kS;
          const int next = page_of(p + 1);
          if (!(ok = wait_warp(&kv_free[s], count / kS + 1, kErrKv))) break;
          const bool k = p < cnt, v = p >= kLag;
          if (lane == 0) mbar_expect_tx(&kv_full[s], (k ? kTB : 0) + (v ? kTB : 0));
          __syncwarp();
          if (lane < per) {
            const uint32_t dst = su32(base + S::kRing + s * 2 * kTB) + lane * box * 128;
            auto copy = [&](int j, uint32_t to, int pg, int which) {
              const int slot = ((t0 + j) * kTile) & (ps - 1);   // nonzero in 256-token pages only
#pragma unroll
              for (int h = 0; h < halves; ++h)
                tma_load_4d(to + h * kTile * 128, &map_kv, 64 * h, slot, head, 2 * pg + which, &kv_full[s]);
            };
            if (k) copy(p, dst, page, 0);
            if (v) copy(p - kLag, dst + kTB, WIDE ? page1 : page2, 1);
          }
          page2 = page1;
          page1 = page;
          page = next;
        }
      }
      if (lane == 0) {   // every copy must have landed before the CTA exits, also where another role gave up
        volatile int never = 0;
        for (uint32_t i = count > kS ? count - kS : 0; i < count; ++i)
          mbar_wait(&kv_full[i % kS], (i / kS) & 1, &never, kErrDrain, &g_attn_error);
      }
      __syncwarp();
    } else if (warp == kQWarp) {
      // ------------------------------------------------ copies of Q: a box is a row tile, 64 elements wide
      if (lane == 0) {
        constexpr int kHalves = DP / 64, kTiles = WIDE ? 2 : 1;
        constexpr uint32_t kQBufs = WIDE ? 1 : 2;
        const uint32_t bytes = uint32_t(r.tile_tokens * r.group) * 128u * kHalves * kTiles;
        uint32_t items = 0;
        for (; w.more(); w.next(c, r), ++items) {
          const uint32_t qb = items % kQBufs, use = items / kQBufs;
          if (!wait(&q_free[qb], use + 1, kErrQ)) break;
          mbar_expect_tx(&q_full[qb], bytes);
          const int tok = w.s.row0 + w.tile * tokens;
#pragma unroll
          for (int x = 0; x < kHalves * kTiles; ++x) {
            const int h = x % kHalves, t = x / kHalves;
            tma_load_3d(su32(base + S::kQ + (qb + t) * kTB + h * kTile * 128), &map_q, 64 * h, w.head * r.group,
                        tok + t * r.tile_tokens, &q_full[qb]);
          }
        }
        volatile int never = 0;   // the last fill of each buffer
        for (uint32_t i = items > kQBufs ? items - kQBufs : 0; i < items; ++i)
          mbar_wait(&q_full[i % kQBufs], (i / kQBufs) & 1, &never, kErrDrain, &g_attn_error);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------ MMA issue
      // Event e of a piece is stream e & 1's tile e / 2, key tile e / 2 (wide) or e (narrow): the scores of
      // the first two events, then per event its second product and the scores of the event after next
      // (the same stream's next tile, which may overwrite the weights just used: MMAs run in order).
      if (elect_one()) {
        const uint32_t tmem = *tmem_base;
        const int bf = kF16 ? 0 : 1;
        const uint32_t id_s = idesc_f16(bf, kTile, kTile), id_o = idesc_f16(bf, kTile, ksteps * 16) | kTransposeB;
        const uint64_t q_desc = sw128_desc(su32(base + S::kQ)), k_desc = sw128_desc(su32(base + S::kRing)),
                       v0_desc = v_desc(su32(base + S::kRing + kTB));
        // barriers by their shared-memory addresses
        const uint32_t bars = su32(bar), b_kv_full = bars + 4 * 8, b_kv_free = b_kv_full + kS * 8, b_s_full = b_kv_free + kS * 8,
                       b_p_ready = b_s_full + 16, b_o_full = b_p_ready + 16, b_o_free = b_o_full + 16;
        auto wait_at = [&](uint32_t b, uint32_t parity, int code) {
          return mbar_wait_at(b, parity & 1, abort_flag, code, &g_attn_error);
        };
        uint32_t items = 0, stage = 0, use = 0;   // the ring's present stage and its use's parity
        uint32_t phases = 0;   // bit st: p_ready, bit 2 + st: o_free (an array would live in local memory)
        bool ok = true;
        for (; ok && w.more(); w.next(c, r), ++items) {
          const int qb = WIDE ? 0 : items & 1;
          const int n0 = w.stream_tiles(r, WIDE, 0), n1 = w.stream_tiles(r, WIDE, 1);
          const int events = WIDE ? 2 * w.cnt : w.cnt;
          ok = wait(&q_full[qb], WIDE ? items : items >> 1, kErrQ);
          const uint64_t q0 = q_desc + uint64_t(qb * (kTB >> 4)), q1 = q0 + uint64_t(WIDE ? kTB >> 4 : 0);
          // i: the stream's tile; st is a constant in every copy of these (an index into registers)
          auto scores = [&](int st, int i) {
            if (i < (st ? n1 : n0)) {
              mma_scores<DP / 16>(tmem + st * kTile, st ? q1 : q0, k_desc + uint64_t(stage * (2 * kTB >> 4)), id_s, ksteps);
              tc_commit_at(b_s_full + st * 8);
            }
          };
          auto output = [&](int st, int i) -> bool {
            const int n = st ? n1 : n0;
            if (i < n) {
              if (i == 0 && !wait_at(b_o_free + st * 8, (phases >> (2 + st)) ^ 1, kErrO)) return false;
              if (!wait_at(b_p_ready + st * 8, phases >> st, kErrP)) return false;
              phases ^= 1u << st;
              tc_fence_after();
              mma_output(tmem + 2 * kTile + st * DP, tmem + st * kTile, v0_desc + uint64_t(stage * (2 * kTB >> 4)), id_o, i != 0);
              if (i + 1 == n) {
                tc_commit_at(b_o_full + st * 8);
                phases ^= 4u << st;
              }
            }
            return true;
          };
#pragma unroll 1   // the loop shares the instruction cache with the softmax: twice its size measured 9% slower
          for (int i = -1; ok && 2 * i < events; ++i) {
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              const int e = 2 * i + st;
              if (!ok || e >= events) break;
              if (!WIDE || st == 0) {
                if (!(ok = wait_at(b_kv_full + stage * 8, use, kErrKv))) break;
                tc_fence_after();
              }
              if (i >= 0 && !(ok = output(st, i))) break;
              if (e + 2 < events) {
                scores(st, i + 1);
                if (e + 3 == events) tc_commit(&q_free[qb]);   // the item's last scores: Q may be replaced
              }
              if (!WIDE || st == 1) {
                tc_commit_at(b_kv_free + stage * 8);
                stage = stage + 1 == kS ? 0 : stage + 1;
                use ^= stage == 0 ? 1 : 0;
              }
            }
          }
        }
        tc_commit(drain);
        volatile int never = 0;
        mbar_wait(drain, 0, &never, kErrDrain, &g_attn_error);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    // ------------------------------------------------ softmax and epilogue
    const uint32_t tmem = *tmem_base;
    const int st = warp >> 2, q4 = warp & 3, row = q4 * 32 + lane;
    const int tok_in = row / r.group, g = row - tok_in * r.group;
    const uint32_t lanes = uint32_t(q4 * 32) << 16;
    const uint32_t t_s = tmem + lanes + st * kTile, t_o = tmem + lanes + 2 * kTile + st * DP;
    const int D = c.head_dim;
    uint8_t *stage = base + S::kStage + warp * kStageBytes;
    uint32_t copies = 0, ns = 0, no[2] = {0, 0}, nx = 0;   // copies: those of the pieces before
    uint32_t turns = 0;   // bit 0, 1: which of two buffers of notes is next (wide: for items that stream 1 works on, others)
    bool ok = true;
    for (; ok && w.more(); next_item()) {
      const int n = w.stream_tiles(r, WIDE, st), t0 = w.t0, start = w.s.start, keys = w.s.keys;
      const int tok = w.tile * tokens + (WIDE ? st * r.tile_tokens : 0) + tok_in;
      bool live = tok_in < r.tile_tokens && tok < w.s.nq;
      const int prow = w.s.row0 + tok;   // packed row
      const uint32_t *bits = r.mask && live ? r.mask + int64_t(prow) * r.words : nullptr;
      const bool valid = live;           // a row of the call; live: it sees something
      if (bits) {
        uint32_t any = 0;
        for (int i = 0; i < r.words; ++i) any |= __ldg(bits + i);
        live = any != 0;
      }
      const bool work = __any_sync(0xffffffffu, live);
      // keys this row may see
      const int lim = keys == 0 ? 0 : (r.mask ? keys : min(start + tok + 1, keys));
      // edge: the first tile that some row of the stream does not see whole.  clean: the first whose V it cleans; one stream
      // does it for both, the first one as far as it goes (its product with a tile is issued before the other's).
      const int edge = w.edge(r, WIDE, st), edge0 = WIDE && st ? w.edge(r, WIDE, 0) : edge;
      const int other = start + w.tile * tokens + r.tile_tokens;   // wide: how far the last row of stream 0 looks
      const int clean = !WIDE || st == 0 ? edge0 : (r.mask || keys == 0 ? INT_MAX : (other + kTile - 1) / kTile);
      // The item's notes, from tile `first` on.  Two buffers in turn: a warp may be at the next item's first tile while others
      // still read, but no further, since later scores follow a product that waits for the o_free of the item before.  Stream 0
      // passes items that stream 1 has no part in without such a wait for stream 1, so those have two buffers of their own.
      const int kind = !WIDE || w.tile * tokens + r.tile_tokens < w.s.nq ? 0 : 1, first = max(edge0, t0);
      volatile uint32_t *notes = all_notes + (2 * kind + (turns >> kind & 1u)) * 4 * kBadTiles;
      turns ^= 1u << kind;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i) {
        const int j = WIDE ? i : 2 * i + st, tile = t0 + j;
        if (!(ok = wait_warp(&s_full[st], ns, kErrS))) break;
        ++ns;
        tc_fence_after();
        if (work) {
          if (tile >= edge) {
            // An edge tile: scores that the row does not see become -inf, in place and 32 at a time, in a loop: selecting
            // among a row's 128 registers would be four times the code in the middle of the tiles' loop, which is
            // fetched past on every tile (packed prompts of 1 to 2500 tokens: 229 against 219 us).
            const int key0 = tile * kTile;
#pragma unroll 1
            for (int x = 0; x < kTile; x += 32) {   // bit y: the row sees key key0 + x + y
              const int k0 = key0 + x, in = min(max(lim - k0, 0), 32);
              uint32_t see = in >= 32 ? 0xffffffffu : (1u << in) - 1u;
              if (r.mask) {
                const int rel = k0 - start;   // new token of bit 0
                uint32_t word = 0xffffffffu;
                if (rel > -32) {
                  const int a = rel >= 0 ? rel >> 5 : -1;
                  const uint32_t lo = a < 0 ? 0xffffffffu : (bits && a < r.words ? __ldg(bits + a) : 0u);
                  const uint32_t hi = bits && a + 1 < r.words ? __ldg(bits + a + 1) : 0u;
                  word = __funnelshift_r(lo, hi, rel & 31);
                }
                see &= word;
              }
              if (!live) see = 0;
              if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t sc[16];
                tc_ld16(t_s + x + 16 * h, sc);
#pragma unroll
                for (int y = 0; y < 16; ++y) sc[y] = (see >> (16 * h + y)) & 1u ? sc[y] : 0xff800000u;
                tc_st16(t_s + x + 16 * h, sc);
              }
            }
            tc_wait_st();
          }
          float v[kTile];
          tc_ld_row(t_s, v);
          float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int x = 4; x < kTile - 4; x += 8) {
#pragma unroll
            for (int y = 0; y < 4; ++y) top[y] = max3(top[y], v[x + 2 * y], v[x + 2 * y + 1]);
          }
          float mt = max3(max3(top[0], top[1], v[kTile - 1]), max3(top[2], v[kTile - 4], v[kTile - 3]),
                          fmaxf(top[3], v[kTile - 2])) * r.scale_log2;
          if (mt > FLT_MAX) mt = FLT_MAX;   // a score of +inf: its weight is inf, not inf - inf, and so are the sum and lse
          const bool grow = i == 0 ? mt > m : mt > m + kLazy || (m == -INFINITY && mt > m);
          if (i > 0 && __any_sync(0xffffffffu, grow)) {
            // the products that have been added to O are complete: this tile's scores were issued behind them
            const float down = grow ? ex2(m - mt) : 1.f;
            l *= down;
#pragma unroll 1
            for (int x = 0; x < ksteps * 16; x += 16) {
              uint32_t o[16];
              tc_ld16(t_o + x, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * down);
              tc_st16(t_o + x, o);
            }
          }
          if (grow) m = mt;
          const float ref = m == -INFINITY ? 0.f : m - kShift;
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              float2 a = fma2({v[32 * x + 2 * y], v[32 * x + 2 * y + 1]}, r.scale_log2, -ref);
              a = {ex2(a.x), ex2(a.y)};
              sum[y & 1] = add2(sum[y & 1], a);
              p[y] = pack2<T>(a.x, a.y);
            }
            tc_st16(t_s + 16 * x, p);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tc_wait_st();
        }
        if (tile >= clean) {
          // V rows that some row must not see: what lies past the keys is zeroed, and so is what is not finite among the new
          // tokens (0 x NaN would reach every row).  Their keys are noted: rows that do see them get the values added in the
          // epilogue.
          constexpr uint32_t kExp = (kF16 ? 0x7C00u : 0x7F80u) * 0x10001u, kLow = (kF16 ? 0x0400u : 0x0080u) * 0x10001u;
          const uint32_t vi = copies + j + kLag;
          if (!(ok = wait_warp(&kv_full[vi % kS], vi / kS, kErrKv))) break;
          const int key = tile * kTile + row;   // this thread's row of the V tile
          uint32_t high = 0;   // an exponent of all ones plus its lowest bit carries into the sign's place
          uint4 *vrow = reinterpret_cast<uint4 *>(base + S::kRing + vi % kS * 2 * kTB + kTB + row * 128);
          if (key >= start) {
#pragma unroll 1
            for (int h = 0; h < DP / 64; ++h) {
              uint4 *e = vrow + h * kTile * 8;   // (x ^ row) & 7: 8 rows, 8 columns, no bank twice
              if (key >= keys) {
#pragma unroll
                for (int x = 0; x < 8; ++x) e[(x ^ row) & 7] = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const uint4 v = e[(x ^ row) & 7];
                high |= ((v.x & kExp) + kLow) | ((v.y & kExp) + kLow) | ((v.z & kExp) + kLow) | ((v.w & kExp) + kLow);
              }
            }
          }
          const bool take = (high & 0x80008000u) != 0;
          const uint32_t note = __ballot_sync(0xffffffffu, take);
          if (lane == 0) {
            volatile uint32_t *to = notes + ((tile - first) & (kBadTiles - 1)) * 4 + q4;
            *to = tile - first < kBadTiles ? note : *to | note;
          }
          if (take) {
#pragma unroll 1
            for (int x = 0; x < DP / 8; ++x) {
              uint4 *e = vrow + (x >> 3) * kTile * 8 + (x & 7);
              auto clear = [&](uint32_t v) {   // 0 in place of what is not finite
                const uint32_t up = ((v & kExp) + kLow) & 0x80008000u;
                return v & ~(up | (up - (up >> 15)));
              };
              *e = make_uint4(clear(e->x), clear(e->y), clear(e->z), clear(e->w));
            }
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[st]);
      }
      if (!ok) break;
      copies += w.cnt + kLag;
      if (!live) {
        m = -INFINITY;
        l = 0.f;
      }
      // the running maximum that goes with l and O as they are
      float ref = m == -INFINITY ? -INFINITY : m - kShift;
      float f0 = 1.f, f1 = 0.f;   // narrow: factors of the two streams' outputs
      const int n1 = WIDE ? 0 : w.cnt >> 1;
      if constexpr (WIDE) {
        if (n > 0) {
          if (!(ok = wait_warp(&o_full[st], no[0], kErrO))) break;
          ++no[0];
        }
      } else {
        // both warps of these rows get the other stream's maximum and sum, and then each merges every
        // other 32 columns of the two accumulators
        float2 *mine = xml + (nx & 1) * 2 * kTile + row;
        mine[st * kTile] = make_float2(ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_full[q4]);
        if (!(ok = wait_warp(&x_full[q4], nx, kErrX))) break;
        ++nx;
        const float2 b = mine[(st ^ 1) * kTile];
        const float top = fmaxf(ref, b.x);
        const float fm = ref == -INFINITY ? 0.f : ex2(ref - top), fo = b.x == -INFINITY ? 0.f : ex2(b.x - top);
        f0 = st == 0 ? fm : fo;
        f1 = st == 0 ? fo : fm;
        l = st == 0 ? l * f0 + b.y * f1 : b.y * f0 + l * f1;   // the same sum in both warps
        ref = top;
        if (!(ok = wait_warp(&o_full[0], no[0], kErrO))) break;
        ++no[0];
        if (n1 > 0) {
          if (!(ok = wait_warp(&o_full[1], no[1], kErrO))) break;
          ++no[1];
        }
      }
      __syncwarp();
      tc_fence_after();
      const int64_t prow_h = int64_t(prow) * r.q_heads + w.head * r.group + g;
      const int slot = w.t0 == 0 ? 1 : 0;
      const bool whole = w.whole();
      constexpr int kPartRows = WIDE ? 2 * kTile : kTile;
      const int part_row = (WIDE ? st * kTile : 0) + row;
      const int64_t part = int64_t(2 * blockIdx.x + slot) * kPartRows;
      // what this lane stores: 16 bytes at (lane & 3) of rows 8 y + lane / 4, in every 32 columns
      const uint32_t rows_valid = __ballot_sync(0xffffffffu, valid);
      uint16_t *to[4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        to[y] = r.out + __shfl_sync(0xffffffffu, prow_h, 8 * y + (lane >> 2)) * D + 8 * (lane & 3);
      // columns x0 .. x0 + 31 of the output row
      const float inv = l == 0.f ? 0.f : 1.f / l;
      auto emit = [&](int x0, const float *o) {
        if (whole) {
          // through shared memory, so that a store instruction covers 64 bytes of 8 rows: 16 bytes of 32
          // rows each would take the L1 32 lines an instruction
          __syncwarp();
          uint8_t *sw = stage + lane * (kCols * 2);
#pragma unroll
          for (int y = 0; y < kCols / 8; ++y)
            *reinterpret_cast<uint4 *>(sw + ((y ^ (lane >> 1)) & 3) * 16) =
                make_uint4(pack2<T>(o[8 * y] * inv, o[8 * y + 1] * inv), pack2<T>(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                           pack2<T>(o[8 * y + 4] * inv, o[8 * y + 5] * inv), pack2<T>(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int rr = 8 * y + (lane >> 2);
            if ((rows_valid >> rr & 1u) && x0 + 8 * (lane & 3) < D)
              *reinterpret_cast<uint4 *>(to[y] + x0) =
                  *reinterpret_cast<const uint4 *>(stage + rr * (kCols * 2) + (((lane & 3) ^ (rr >> 1)) & 3) * 16);
          }
        } else if (valid) {   // columns apart, rows together: a store covers 32 rows of a column
          float *dst = ws.o + part * DP + int64_t(x0) * kPartRows + part_row;
#pragma unroll
          for (int y = 0; y < kCols; ++y) dst[y * kPartRows] = o[y];
        }
      };
      if constexpr (WIDE) {
#pragma unroll 1   // code off the tiles' path is kept small: see the edge tiles
        for (int x0 = 0; x0 < ksteps * 16; x0 += kCols) {
          float o[kCols];
          __syncwarp();
          if (n > 0 && work) tc_ld32(t_o + x0, o);
          if (n == 0 || !work || l == 0.f) {
#pragma unroll
            for (int y = 0; y < kCols; ++y) o[y] = 0.f;
          }
          emit(x0, o);
        }
      } else {
        for (int x0 = kCols * st; x0 < ksteps * 16; x0 += 2 * kCols) {
          float o[kCols], o1[kCols];
          __syncwarp();
          if (work) tc_ld32(tmem + lanes + 2 * kTile + x0, o);
#pragma unroll
          for (int y = 0; y < kCols; ++y) o[y] = f0 == 0.f ? 0.f : o[y] * f0;
          if (n1 > 0 && work) {
            tc_ld32(tmem + lanes + 2 * kTile + DP + x0, o1);
#pragma unroll
            for (int y = 0; y < kCols; ++y) o[y] = f1 == 0.f ? o[y] : fmaf(o1[y], f1, o[y]);
          }
          emit(x0, o);
        }
      }
      // New tokens' values that were taken out of the second product: a row that sees one gets it here (whatever its weight,
      // the result is the same infinity or NaN).  Only the noted keys are visited: a prompt of 8191 tokens, 8 heads of 128, takes
      // 139 us without any, 141 us with two in it, 220 us with 16 tokens of nothing else, 4.0 ms where every value is one.
      const int words = 4 * (t0 + (WIDE ? n : w.cnt) - first);
      uint32_t any = 0;
      for (int x = lane; x < min(words, 4 * kBadTiles); x += 32) any |= notes[x];
      if (__any_sync(0xffffffffu, any != 0)) {
        __syncwarp();   // the output rows are in memory
        const int sees = valid && l != 0.f ? min(r.mask ? min(lim, start + 32 * r.words) : lim, (t0 + w.cnt) * kTile) : 0;
#pragma unroll 1
        for (int x = 0; x < words; ++x) {
          const uint32_t word = notes[x & (4 * kBadTiles - 1)];
          if (word == 0) continue;
          // lane y finds where key key0 + y lies; bit y of vis: this row sees it
          const int key0 = first * kTile + 32 * x, key = key0 + lane, rel = key0 - start;
          int64_t at = -1;
          if ((word >> lane & 1u) && key >= start && key < keys) {
            const int p = __ldg(c.table + int64_t(w.s.slot) * c.max_pages + (key >> c.page_shift));
            if (p >= 0 && p < c.pages)
              at = ((int64_t(2 * p + 1) * c.kv_heads + w.head) * c.page_size() + (key & (c.page_size() - 1))) * D;
          }
          uint32_t vis = 0;
#pragma unroll 1
          for (int y = max(-rel, 0); y < 32 && key0 + y < sees; ++y)
            if (!bits || (__ldg(bits + ((rel + y) >> 5)) >> ((rel + y) & 31) & 1u)) vis |= 1u << y;
          vis &= __ballot_sync(0xffffffffu, at >= 0);
          uint32_t todo = vis;
#pragma unroll
          for (int y = 1; y < 32; y <<= 1) todo |= __shfl_xor_sync(0xffffffffu, todo, y);
#pragma unroll 1
          for (int x0 = WIDE ? 0 : kCols * st; x0 < D; x0 += WIDE ? kCols : 2 * kCols) {   // the columns that this warp wrote
            float add[kCols];
#pragma unroll
            for (int z = 0; z < kCols; ++z) add[z] = 0.f;
#pragma unroll 1
            for (uint32_t left = todo; left != 0; left &= left - 1) {
              const int y = __ffs(left) - 1;
              const uint4 *row_v = reinterpret_cast<const uint4 *>(layer_pool + __shfl_sync(0xffffffffu, at, y) + x0);
              const bool here = vis >> y & 1u;
              uint4 e[kCols / 8];
#pragma unroll
              for (int z = 0; z < kCols / 8; ++z) e[z] = x0 + 8 * z < D ? __ldg(row_v + z) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int z = 0; z < kCols; ++z) {
                const float f = to_f32(reinterpret_cast<const T *>(e)[z]);
                add[z] += here && !(fabsf(f) < INFINITY) ? f : 0.f;
              }
            }
#pragma unroll
            for (int z = 0; z < kCols; z += 8) {
              bool some = false;
#pragma unroll
              for (int y = 0; y < 8; ++y) some |= add[z + y] != 0.f;
              if (!some) continue;
              if (whole) {
                uint4 *to_row = reinterpret_cast<uint4 *>(r.out + prow_h * D + x0 + z);
                uint4 e = *to_row;
                T *v = reinterpret_cast<T *>(&e);
#pragma unroll
                for (int y = 0; y < 8; ++y) v[y] = from_f32<T>(to_f32(v[y]) + add[z + y]);
                *to_row = e;
              } else {
                float *to_part = ws.o + part * DP + int64_t(x0 + z) * kPartRows + part_row;
#pragma unroll
                for (int y = 0; y < 8; ++y) add[z + y] += to_part[y * kPartRows];
#pragma unroll
                for (int y = 0; y < 8; ++y) to_part[y * kPartRows] = add[z + y];
              }
            }
          }
        }
      }
      if (valid && (WIDE || st == 0)) {
        if (whole) {
          if (r.lse) r.lse[prow_h] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
        } else {
          ws.ml[part + part_row] = make_float2(ref, l);
        }
      }
      if (!whole && tid == 0) {
        const int last = place->owner(w.unit - w.in_item + w.total + w.cost - 1);   // the item's last unit
        Piece p = {1, w.seq, w.tile, w.head, last - int(blockIdx.x) + 1, 0, 0, 0};
        ws.piece[2 * blockIdx.x + slot] = p;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (WIDE ? n > 0 : true) mbar_arrive(&o_free[WIDE ? st : 0]);
        if (!WIDE && n1 > 0) mbar_arrive(&o_free[1]);
      }
    }
  }

  // ---- teardown: everyone done, release tensor memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(*tmem_base), "r"(512u));
}

// Join the pieces of the item that CTA blockIdx.x began and did not finish, in the order of the CTAs
// (so that runs agree).  A thread owns four columns of a row.  grid: (CTAs of the first kernel, columns)
template <typename T, int DP, bool WIDE>
__global__ void __launch_bounds__(256) attn_join_kernel(const KvView c, const Rows r, const Workspace ws) {
  pdl_enter();
  const int cta = blockIdx.x;
  const Piece p = ws.piece[2 * cta + 1];
  if (!p.valid) return;
  constexpr int kRows = WIDE ? 2 * kTile : kTile;
  const int tokens = WIDE ? 2 * r.tile_tokens : r.tile_tokens;
  const Seq s = load_seq(c, r, tokens, p.seq);
  const int x = int(blockIdx.y) * 256 + int(threadIdx.x), row = x % kRows, d = 4 * (x / kRows);
  const int st = row / kTile, tok_in = (row - st * kTile) / r.group, g = row - st * kTile - tok_in * r.group;
  const int tok = p.tile * tokens + st * r.tile_tokens + tok_in;
  if (tok_in >= r.tile_tokens || tok >= s.nq) return;
  // kBatch pieces' loads are in flight together: one after the other their latencies would add up
  constexpr int kBatch = 8;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < p.pieces; i0 += kBatch) {
    float2 ml[kBatch];
    float v[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i < p.pieces) {
        const int64_t at = int64_t(i0 + i == 0 ? 2 * cta + 1 : 2 * (cta + i0 + i)) * kRows;
        ml[i] = ws.ml[at + row];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[i][y] = ws.o[at * DP + (d + y) * kRows + row];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (ml[i].y == 0.f) continue;
      const float top = fmaxf(m, ml[i].x), a = m == -INFINITY ? 0.f : ex2(m - top), b = ex2(ml[i].x - top);
      l = l * a + ml[i].y * b;
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = o[y] * a + v[i][y] * b;
      m = top;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = int64_t(s.row0 + tok) * r.q_heads + p.head * r.group + g;
  if (d < c.head_dim)
    *reinterpret_cast<uint2 *>(r.out + at * c.head_dim + d) =
        make_uint2(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv));
  if (r.lse && d == 0) r.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// One thread per row: walk up to the context, setting the bit of every ancestor.
__global__ void __launch_bounds__(kThreads) tree_mask_kernel(const int32_t *__restrict__ parents,
                                                             const int32_t *__restrict__ cu,
                                                             const int32_t *__restrict__ start, int n, int T, int words,
                                                             uint32_t *__restrict__ mask, int32_t *__restrict__ pos) {
  pdl_enter();
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= T) return;
  const int b = seq_of_row(cu, n, t);
  if (b < 0) return;
  const int t0 = cu[b];
  int depth = 0, i = t - t0;
  bool ok = t0 >= 0;
  // parents have smaller indices, so the walk ends
  for (int a = i; ok; ++depth) {
    const int p = a < 32 * words ? parents[t0 + a] : -2;
    if (p < -1 || p >= a) ok = false;
    if (p < 0) break;
    a = p;
  }
  uint32_t *row = mask + int64_t(t) * words;
  for (int w = 0; w < words; ++w) row[w] = 0;
  if (ok)
    for (int a = i; a >= 0; a = parents[t0 + a]) row[a >> 5] |= 1u << (a & 31);
  if (pos) pos[t] = start[b] + (ok ? depth : 0);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_tree_mask(const int32_t *parents, const int32_t *cu, const int32_t *start, int64_t n, int64_t T,
                             int64_t mask_words, uint32_t *mask, int32_t *pos, moe_stream_t stream) {
  MOE_REQUIRE(n >= 0 && n < (int64_t(1) << 22) && T >= 0 && T < (int64_t(1) << 30), "n or T out of range");
  MOE_REQUIRE(mask_words >= 1 && mask_words <= 1024, "need 1 <= mask_words <= 1024 (%lld)", (long long)mask_words);
  if (n == 0 || T == 0) return MOE_OK;
  MOE_REQUIRE(parents && cu && mask && (start || !pos), "null pointer argument");
  MOE_REQUIRE(aligned16(parents) && aligned16(cu) && aligned16(start) && aligned16(mask) && aligned16(pos),
              "pointers must be 16-byte aligned");
  launch_pdl(tree_mask_kernel, dim3(unsigned(cdiv(T, kThreads))), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream),
             parents, cu, start, int(n), int(T), int(mask_words), mask, pos);
  return check_launch("tree_mask");
}

namespace {

struct AttnPlan {
  int grid, dp;
  bool wide;
  size_t o_ml, o_o, bytes;
};
// Two row tiles per item when a sequence brings more rows than one tile holds on average: then
// both streams share every key tile; with fewer rows the second row tile would be padding.  One and two row tiles, 32 query
// and 8 K/V heads of 128: 64 single tokens over 2000 99 and 110 us; 32 trees over 4000 of 32 tokens (128 rows) 104 and 113,
// of 33 185 and 119, of 64 188 and 129; 32 prompts of 40 29 and 23; 4 prompts of 500 38 and 35.  The average misjudges
// two row tiles over few keys (8 times 64 tokens over 1000: 29 and 33) and mixtures: a prompt of 2000 beside 32 single
// tokens over 4000 takes 125 and 135 (two are chosen), one of 600 beside 20 takes 72 and 78 (one is).
bool wide_form(const moe_kv_desc *d, int64_t T, int64_t n, int64_t q_heads) { return T * (q_heads / d->kv_heads) > n * kTile; }
AttnPlan plan_attention(const moe_kv_desc *d, bool wide) {
  AttnPlan p{};
  p.grid = num_sms();
  p.dp = d->head_dim <= 64 ? 64 : 128;
  p.wide = wide;
  const size_t rows = size_t(2 * p.grid) * (p.wide ? 2 : 1) * kTile;
  p.o_ml = align256(size_t(2 * p.grid) * sizeof(Piece));
  p.o_o = p.o_ml + align256(rows * sizeof(float2));
  p.bytes = p.o_o + rows * p.dp * sizeof(float);
  return p;
}

struct AttnCall {
  const moe_kv_desc *d;
  const moe_kv *kv;
  int64_t layer;
  const void *q;
  int64_t qt;
  AttnPlan pl;
  char *ws;
  cudaStream_t st;
};

template <typename T, int DP, bool WIDE> int launch_attention_as(const AttnCall &a, const Rows &r) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("attention: cudaGetDevice");
  if (dev < 0 || dev >= 64) return set_error(MOE_ERR_UNSUPPORTED, "attention: device index %d >= 64", dev);
  const KvView c = kv_view(a.d, a.kv);
  const CUtensorMapDataType type =
      std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  CUtensorMap mq, mk;
  {   // q as (T, heads, head_dim): a box is a row tile, 64 elements wide
    const cuuint64_t dims[3] = {cuuint64_t(c.head_dim), cuuint64_t(r.q_heads), cuuint64_t(r.T)};
    const cuuint64_t strides[2] = {cuuint64_t(c.head_dim) * 2, cuuint64_t(a.qt) * 2};
    const cuuint32_t box[3] = {64u, cuuint32_t(r.group), cuuint32_t(r.tile_tokens)};
    const CUresult e = enc(&mq, type, 3, const_cast<void *>(a.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e != CUDA_SUCCESS) return set_error(MOE_ERR_CUDA, "query tensor map encode failed (%d)", int(e));
  }
  {   // the layer's pool as (2 pages, heads, slots, head_dim): a box is a page (half a 256-token page)
    const cuuint64_t ps = cuuint64_t(c.page_size()), D = cuuint64_t(c.head_dim), H = cuuint64_t(c.kv_heads);
    const cuuint64_t dims[4] = {D, ps, H, 2 * cuuint64_t(c.pages)};
    const cuuint64_t strides[3] = {D * 2, ps * D * 2, H * ps * D * 2};
    const cuuint32_t box[4] = {64u, cuuint32_t(ps < kTile ? ps : kTile), 1u, 1u};
    const CUresult e = enc(&mk, type, 4, c.pool + a.layer * c.layer_elems(), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e != CUDA_SUCCESS) return set_error(MOE_ERR_CUDA, "cache tensor map encode failed (%d)", int(e));
  }
  Workspace ws{reinterpret_cast<Piece *>(a.ws), reinterpret_cast<float2 *>(a.ws + a.pl.o_ml),
               reinterpret_cast<float *>(a.ws + a.pl.o_o)};
  auto kern = attn_kernel<T, DP, WIDE>;
  constexpr int smem = Smem<DP>::kBytes;
  static std::atomic<bool> attr_set[64];   // the opt-in is a per-device attribute of the kernel
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return check_launch("attention attribute");
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  launch_pdl(kern, dim3(unsigned(a.pl.grid)), dim3(kAttnThreads), smem, a.st, mq, mk, c, r,
             static_cast<const uint16_t *>(c.pool + a.layer * c.layer_elems()), ws);
  MOE_TRY(check_launch("attention"));
  constexpr int rows = WIDE ? 2 * kTile : kTile;
  launch_pdl(attn_join_kernel<T, DP, WIDE>, dim3(unsigned(a.pl.grid), unsigned(rows * (DP / 4) / 256)), dim3(256), 0, a.st, c, r,
             ws);
  return check_launch("attention: join");
}
template <typename T> int launch_attention(const AttnCall &a, const Rows &r) {
  if (a.pl.dp == 64) return a.pl.wide ? launch_attention_as<T, 64, true>(a, r) : launch_attention_as<T, 64, false>(a, r);
  return a.pl.wide ? launch_attention_as<T, 128, true>(a, r) : launch_attention_as<T, 128, false>(a, r);
}

int check_attention(const moe_kv_desc *d, int64_t T, int64_t n, int64_t q_heads) {
  MOE_TRY(check_kv_desc(d));
  MOE_REQUIRE(T >= 0 && T < (int64_t(1) << 30) && n >= 0 && n < (int64_t(1) << 22), "T or n out of range");
  MOE_SUPPORT(d->head_dim <= 128, "attention takes head_dim <= 128 (%lld)", (long long)d->head_dim);
  MOE_REQUIRE(q_heads >= 1 && q_heads % d->kv_heads == 0, "q_heads must be a multiple of kv_heads (%lld, %lld)",
              (long long)q_heads, (long long)d->kv_heads);
  MOE_SUPPORT(q_heads / d->kv_heads <= 128, "at most 128 query heads per K/V head (%lld)",
              (long long)(q_heads / d->kv_heads));
  return MOE_OK;
}
}  // namespace

extern "C" size_t moe_attention_workspace_size(const moe_kv_desc *desc, int64_t T, int64_t n, int64_t q_heads) {
  if (check_attention(desc, T, n, q_heads) != MOE_OK || T == 0 || n == 0) return 0;
  return plan_attention(desc, wide_form(desc, T, 1, q_heads)).bytes;   // as many tokens of one sequence need the most
}

extern "C" int moe_attention(const moe_kv_desc *desc, const moe_kv *kv, int64_t layer, const void *q,
                             int64_t q_token_stride, int64_t q_heads, int64_t T, const int32_t *cu, const int32_t *seqs,
                             const int32_t *start, int64_t n, const uint32_t *mask, int64_t mask_words, float scale,
                             void *out, float *lse, void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_attention(desc, T, n, q_heads));
  MOE_REQUIRE(layer >= 0 && layer < desc->layers, "layer %lld is not in the cache", (long long)layer);
  MOE_REQUIRE(q_token_stride % 8 == 0 && (T <= 1 || q_token_stride >= q_heads * desc->head_dim) &&
                  q_token_stride < (int64_t(1) << 38),
              "q's token stride must be a multiple of 8 that holds the heads (%lld)", (long long)q_token_stride);
  MOE_REQUIRE(mask == nullptr || (mask_words >= 1 && mask_words <= 1024), "need 1 <= mask_words <= 1024 (%lld)",
              (long long)mask_words);
  // times log2(e) it has to be finite still: a score of 0 would be 0 x inf
  MOE_REQUIRE(scale > 0.f && scale <= 2.3e38f, "scale must be positive, at most 2.3e38 (%g)", double(scale));
  if (T == 0 || n == 0) return MOE_OK;
  MOE_REQUIRE(q && cu && seqs && start && out, "null pointer argument");
  MOE_REQUIRE(aligned16(q) && aligned16(cu) && aligned16(seqs) && aligned16(start) && aligned16(mask) && aligned16(out) &&
                  aligned16(lse),
              "pointers must be 16-byte aligned");
  const AttnPlan pl = plan_attention(desc, wide_form(desc, T, n, q_heads));
  MOE_REQUIRE(workspace && aligned16(workspace), "workspace must be non-null and 16-byte aligned");
  if (workspace_bytes < pl.bytes)
    return set_error(MOE_ERR_WORKSPACE, "attention workspace %zu < %zu bytes", workspace_bytes, pl.bytes);
  Rows r{};
  r.cu = cu;
  r.seqs = seqs;
  r.start = start;
  r.mask = mask;
  r.out = static_cast<uint16_t *>(out);
  r.lse = lse;
  r.n = int(n);
  r.T = int(T);
  r.q_heads = int(q_heads);
  r.group = int(q_heads / desc->kv_heads);
  r.words = int(mask_words);
  r.tile_tokens = kTile / r.group;
  r.scale_log2 = scale * 1.4426950408889634f;
  AttnCall a{desc, kv, layer, q, T <= 1 ? q_heads * desc->head_dim : q_token_stride, pl, static_cast<char *>(workspace),
             reinterpret_cast<cudaStream_t>(stream)};
  return desc->dtype == MOE_F16 ? launch_attention<__half>(a, r) : launch_attention<__nv_bfloat16>(a, r);
}
