// Paged key/value cache: growing, forking (copy on write), compacting, freeing and copying pages, and
// writing new tokens.
//
// The free pages are those nobody holds (refs == 0) and allocation takes the lowest-numbered ones in
// the order (sequence of the call, place in the sequence): no free list whose order would depend on
// the order of atomic pushes, so every result is the same on every run and any launch shape.
//
// Bookkeeping is latency (a few dependent reads per call), data is bandwidth.  Measured on GB300: 104 pages of
// 16 layers copied (872 MB moved) in 129 us, 6.8 TB/s; 405 new tokens of 24 sequences
// written to 32 layers (106 MB) in 18.5 us, 5.7 TB/s, and the accepted ones moved up (31 MB) in 9 us;
// the page side of a compaction 4 us; extend of 8 sequences 4.4 us where the free pages are found among the first 1000,
// 5.7 and 21.5 us where they are the last of 10^4 and 10^5 (one block looks at 4096 pages a round).
#include "kv_internal.cuh"

namespace moe {

MOE_DEFINE_CHECK_WORD(kv)

int check_kv_desc(const moe_kv_desc *d) {
  MOE_REQUIRE(d != nullptr, "desc is NULL");
  MOE_REQUIRE(is16(d->dtype), "desc.dtype must be MOE_F16 or MOE_BF16");
  MOE_REQUIRE(d->layers >= 1 && d->layers <= 4096, "need 1 <= layers <= 4096 (%lld)", (long long)d->layers);
  MOE_REQUIRE(d->pages >= 1 && d->pages < (int64_t(1) << 30), "need 1 <= pages < 2^30 (%lld)", (long long)d->pages);
  MOE_REQUIRE(is_pow2(d->page_size) && d->page_size >= 8 && d->page_size <= 256,
              "page_size must be a power of two in [8, 256] (%lld)", (long long)d->page_size);
  MOE_REQUIRE(d->kv_heads >= 1 && d->kv_heads <= 1024, "need 1 <= kv_heads <= 1024 (%lld)", (long long)d->kv_heads);
  MOE_REQUIRE(d->head_dim >= 8 && d->head_dim % 8 == 0 && d->head_dim <= 256,
              "head_dim must be a multiple of 8, at most 256 (%lld)", (long long)d->head_dim);
  MOE_REQUIRE(d->slots >= 1 && d->slots < (int64_t(1) << 30) && d->max_pages >= 1 && d->max_pages < (int64_t(1) << 20) &&
                  d->slots * d->max_pages < (int64_t(1) << 31),
              "need slots >= 1, 1 <= max_pages < 2^20, slots * max_pages < 2^31");
  return MOE_OK;
}

int check_kv(const moe_kv_desc *d, const moe_kv *kv) {
  MOE_TRY(check_kv_desc(d));
  MOE_REQUIRE(kv && kv->pool && kv->table && kv->lens && kv->refs, "null pointer argument");
  MOE_REQUIRE(aligned16(kv->pool) && aligned16(kv->table) && aligned16(kv->lens) && aligned16(kv->refs),
              "pointers must be 16-byte aligned");
  return MOE_OK;
}

namespace {

constexpr int kThreads = 256;
constexpr int kBook = 1024;   // threads of the one-block bookkeeping kernel

// Page `p` of the table, or -1 where it must not be followed.
__device__ __forceinline__ int valid_page(const KvView &c, int p) {
  if (p >= 0 && p < c.pages) return p;
  if (MOE_CHECKED && p != -1) check_fail(kCheckPage);
  return -1;
}

__device__ __forceinline__ int pages_for(const KvView &c, int64_t len) {
  return int((len + c.page_size() - 1) >> c.page_shift);
}

// One holder less of page p (never below zero).
__device__ __forceinline__ void release(const KvView &c, int p) {
  if ((p = valid_page(c, p)) < 0) return;
  if (atomicSub(&c.refs[p], 1) <= 0) atomicAdd(&c.refs[p], 1);
}

// Where a sequence starts to take pages, and whether its partly filled last page must be copied.
struct Growth {
  int slot, old, want, first, shared;   // shared: the page to copy or -1; slot -1: skipped
};
__device__ __forceinline__ Growth growth(const KvView &c, const int32_t *seqs, const int32_t *n_new, int i) {
  Growth g{-1, 0, 0, 0, -1};
  const int q = seqs[i], add = n_new[i];
  if (q < 0 || q >= c.slots || add < 0) return g;
  const int len = c.lens[q];
  if (len < 0) return g;
  g.slot = q;
  g.old = len;
  const int have = pages_for(c, len);
  g.want = pages_for(c, int64_t(len) + add);
  g.first = have;
  if (add > 0 && (len & (c.page_size() - 1)) != 0 && have <= c.max_pages) {
    const int p = valid_page(c, c.table[int64_t(q) * c.max_pages + have - 1]);
    if (p >= 0 && c.refs[p] > 1) {
      g.first = have - 1;
      g.shared = p;
    }
  }
  return g;
}

// Workspace of extend: prefix[n + 1] of the pages each sequence needs, cow[2 n] (source, copy) pairs,
// page[pages] the pages taken.
struct ExtendWs {
  int32_t *prefix, *cow, *page;
};

// One block: needs and their prefix sum, the lowest free pages, then tables, counts and lengths.
__global__ void __launch_bounds__(kBook) kv_extend_kernel(const KvView c, const int32_t *__restrict__ seqs,
                                                          const int32_t *__restrict__ n_new, int n,
                                                          int32_t *__restrict__ start, const ExtendWs w) {
  pdl_enter();
  __shared__ int scratch[32];
  __shared__ int fits;
  const int tid = threadIdx.x;
  if (tid == 0) fits = 1;
  __syncthreads();
  // the first holders' counts are on their way while the needs are worked out; the first round of sequences stays
  // in registers (the usual call has no other)
  auto held4 = [&](int p) -> int4 {
    if (p + 3 < c.pages) return *reinterpret_cast<const int4 *>(c.refs + p);
    if (p >= c.pages) return make_int4(1, 1, 1, 1);
    return make_int4(c.refs[p], p + 1 < c.pages ? c.refs[p + 1] : 1, p + 2 < c.pages ? c.refs[p + 2] : 1, 1);
  };
  int4 held = held4(4 * tid);
  const Growth mine = tid < n ? growth(c, seqs, n_new, tid) : Growth{-1, 0, 0, 0, -1};
  auto growth_of = [&](int i) { return i == tid ? mine : growth(c, seqs, n_new, i); };
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += kBook) {
    const int i = i0 + tid;
    int need = 0, at = 0;
    if (i < n) {
      const Growth g = growth_of(i);
      if (g.slot >= 0) {
        if (g.want > c.max_pages) fits = 0;
        else need = max(0, g.want - g.first);
      }
    }
    const int sum = block_exclusive_scan(min(need, c.pages + 1), &at, scratch);
    if (i < n) w.prefix[i] = total + at;
    total += sum;
    if (total > c.pages) break;   // more than there are (and keeps the sums small)
  }
  if (tid == 0) w.prefix[n] = total;
  __syncthreads();
  int found = 0;
  if (fits && total <= c.pages) {
    for (int p0 = 0; p0 < c.pages && found < total; p0 += 4 * kBook) {
      const int p = p0 + 4 * tid;
      if (p0 > 0) held = held4(p);
      const int free4[4] = {held.x == 0, held.y == 0, held.z == 0, held.w == 0};
      int at = 0;
      const int sum = block_exclusive_scan(free4[0] + free4[1] + free4[2] + free4[3], &at, scratch);
      at += found;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (free4[y] && at < total) w.page[at] = p + y;
        at += free4[y];
      }
      found += sum;
    }
  }
  __syncthreads();
  const bool ok = fits && total <= c.pages && found >= total;
  // decisions first (they read lens, table and refs), then the changes
  for (int i = tid; i < n; i += kBook) {
    const Growth g = growth_of(i);
    start[i] = ok && g.slot >= 0 ? g.old : -1;
    const bool copy = ok && g.shared >= 0;
    w.cow[2 * i] = copy ? g.shared : -1;
    w.cow[2 * i + 1] = copy ? w.page[w.prefix[i]] : -1;
  }
  __syncthreads();
  if (!ok) return;
  for (int i = tid; i < n; i += kBook) {
    const int q = seqs[i];
    if (start[i] < 0) continue;
    const int old = start[i], have = pages_for(c, old), first = w.cow[2 * i] >= 0 ? have - 1 : have;
    const int k0 = w.prefix[i], k1 = w.prefix[i + 1];
    for (int k = k0; k < k1; ++k) {
      c.table[int64_t(q) * c.max_pages + first + (k - k0)] = w.page[k];
      c.refs[w.page[k]] = 1;
    }
    if (w.cow[2 * i] >= 0) atomicSub(&c.refs[w.cow[2 * i]], 1);
    c.lens[q] = old + n_new[i];
  }
}

// Page copies, every layer: the blocks walk the list of pairs (32 of them per look) and share the pieces of every
// copy to be made, so that a list without any costs a launch and one load.
constexpr int kPiece = kThreads * 8;   // 16-byte vectors of a page that a block moves at a time
template <typename Pair> __device__ __forceinline__ void copy_pages(const KvView &c, int n, Pair pair) {
  const int lane = threadIdx.x & 31;
  const int64_t per = 2 * c.half_elems() / 8, pieces = (per + kPiece - 1) / kPiece;   // per page
  uint4 *pool = reinterpret_cast<uint4 *>(c.pool);
  for (int i0 = 0; i0 < n; i0 += 32) {
    int src = -1, dst = -1;
    if (i0 + lane < n) pair(i0 + lane, &src, &dst);
    const unsigned todo = __ballot_sync(0xffffffffu, src >= 0 && dst >= 0 && src != dst);
    const int64_t each = pieces * c.layers, all = each * __popc(todo);
    for (int64_t x = blockIdx.x; x < all; x += gridDim.x) {
      const int nth = int(x / each), from = int(__fns(todo, 0, nth + 1));   // the nth pair to be copied
      const int64_t s = __shfl_sync(0xffffffffu, src, from), d = __shfl_sync(0xffffffffu, dst, from);
      const int64_t y0 = x - nth * each, layer = y0 / pieces, v0 = (y0 - layer * pieces) * kPiece + threadIdx.x;
      uint4 *base = pool + layer * (c.layer_elems() / 8);
      uint4 v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        if (v0 + y * kThreads < per) v[y] = base[s * per + v0 + y * kThreads];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        if (v0 + y * kThreads < per) base[d * per + v0 + y * kThreads] = v[y];
    }
  }
}

__global__ void __launch_bounds__(kThreads) kv_cow_kernel(const KvView c, const int32_t *__restrict__ cow, int n) {
  pdl_enter();
  copy_pages(c, n, [&](int i, int *s, int *d) {
    *s = cow[2 * i];
    *d = cow[2 * i + 1];
  });
}

__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const KvView c, const int32_t *__restrict__ src,
                                                           const int32_t *__restrict__ dst, int n) {
  pdl_enter();
  copy_pages(c, n, [&](int i, int *s, int *d) {
    *s = valid_page(c, src[i]);
    *d = valid_page(c, dst[i]);
  });
}

// One block per pair.
__global__ void __launch_bounds__(kThreads) kv_fork_kernel(const KvView c, const int32_t *__restrict__ src,
                                                           const int32_t *__restrict__ dst) {
  pdl_enter();
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || s >= c.slots || d < 0 || d >= c.slots || s == d || c.lens[d] != 0) return;
  const int len = c.lens[s], used = min(pages_for(c, max(len, 0)), c.max_pages);
  __syncthreads();   // every thread has read lens[d]
  for (int i = threadIdx.x; i < used; i += kThreads) {
    const int p = c.table[int64_t(s) * c.max_pages + i];
    c.table[int64_t(d) * c.max_pages + i] = p;
    if (valid_page(c, p) >= 0) atomicAdd(&c.refs[p], 1);
  }
  if (threadIdx.x == 0) c.lens[d] = len;
}

__global__ void __launch_bounds__(kThreads) kv_free_kernel(const KvView c, const int32_t *__restrict__ seqs) {
  pdl_enter();
  const int q = seqs[blockIdx.x];
  if (q < 0 || q >= c.slots) return;
  const int used = min(pages_for(c, max(c.lens[q], 0)), c.max_pages);
  __syncthreads();   // every thread has read lens[q]
  for (int i = threadIdx.x; i < used; i += kThreads) release(c, atomicExch(&c.table[int64_t(q) * c.max_pages + i], -1));
  if (threadIdx.x == 0) c.lens[q] = 0;
}

// What a compaction does to sequence i: slot, where it starts, how many stay.
struct Kept {
  int slot, start, len, k0, count;   // slot -1: skipped
};
__device__ __forceinline__ Kept kept(const KvView &c, const int32_t *seqs, const int32_t *start, const int32_t *cu_keep,
                                     int64_t keep_len, int i) {
  Kept k{-1, 0, 0, 0, 0};
  const int q = seqs[i], s = start[i], k0 = cu_keep[i], k1 = cu_keep[i + 1];
  if (q < 0 || q >= c.slots || s < 0 || k0 < 0 || k1 < k0 || k1 > keep_len) return k;
  const int len = c.lens[q];
  if (int64_t(s) + (k1 - k0) > len || pages_for(c, len) > c.max_pages) return k;
  k.slot = q;
  k.start = s;
  k.len = len;
  k.k0 = k0;
  k.count = k1 - k0;
  return k;
}

// Moves of sequence k on one layer.  A thread owns one 16-byte piece of a row (K or V, head) and walks
// the kept tokens in order: entry j is read at offset keep[j] >= j and written at offset j, and no later
// entry reads an offset already written (ascending: keep[j'] >= j' > j); so a batch may be read before
// it is written.  from / to: where the batch's tokens lie in a layer, worked out once for the block.
constexpr int kMoves = 128, kMoveBatch = 8;
struct MoveTable {
  int64_t from[kMoves], to[kMoves];   // element offset of the token's slot in K of head 0, -1: nothing to move
};
__device__ void move_tokens(const KvView &c, const Kept &k, const int32_t *__restrict__ keep, MoveTable *mt, int layer0,
                            int layers, int piece0, int stride) {
  const int dv = c.head_dim / 8, pieces = 2 * c.kv_heads * dv, ps = c.page_size();
  const int32_t *tab = c.table + int64_t(k.slot) * c.max_pages;
  for (int j0 = 0; j0 < k.count; j0 += kMoves) {
    const int n = min(kMoves, k.count - j0);
    __syncthreads();   // the table before has been used
    for (int j = threadIdx.x; j < kMoves; j += blockDim.x) {
      int64_t f = -1, t = -1;
      if (j < n) {
        const int from = keep[k.k0 + j0 + j];
        const bool ascends = j0 + j == 0 || from > keep[k.k0 + j0 + j - 1];
        if (ascends && from > j0 + j && from < k.len - k.start) {
          auto at = [&](int pos) -> int64_t {
            const int p = valid_page(c, tab[pos >> c.page_shift]);
            return p < 0 ? -1 : (int64_t(p) * 2 * c.kv_heads * ps + (pos & (ps - 1))) * c.head_dim;
          };
          f = at(k.start + from);
          t = at(k.start + j0 + j);
          if (f < 0 || t < 0) f = t = -1;
        }
      }
      mt->from[j] = f;
      mt->to[j] = t;
    }
    __syncthreads();
    for (int e = piece0; e < pieces * layers; e += stride) {
      const int layer = e / pieces, x = e - layer * pieces, row = x / dv;
      uint16_t *base = c.pool + int64_t(layer0 + layer) * c.layer_elems() + int64_t(row) * ps * c.head_dim + (x - row * dv) * 8;
      for (int j = 0; j < n; j += kMoveBatch) {
        uint4 v[kMoveBatch];
#pragma unroll
        for (int y = 0; y < kMoveBatch; ++y)   // n <= kMoves, a multiple of the batch: entries past n are -1
          if (mt->from[j + y] >= 0) v[y] = *reinterpret_cast<const uint4 *>(base + mt->from[j + y]);
#pragma unroll
        for (int y = 0; y < kMoveBatch; ++y)
          if (mt->from[j + y] >= 0) *reinterpret_cast<uint4 *>(base + mt->to[j + y]) = v[y];
      }
    }
  }
}

__device__ __forceinline__ void shrink(const KvView &c, const Kept &k) {
  const int len = k.start + k.count;
  for (int i = pages_for(c, len) + threadIdx.x; i < pages_for(c, k.len); i += blockDim.x)
    release(c, atomicExch(&c.table[int64_t(k.slot) * c.max_pages + i], -1));
  if (threadIdx.x == 0) c.lens[k.slot] = len;
}

// grid: (pieces, layers, sequences)
__global__ void __launch_bounds__(kThreads) kv_move_kernel(const KvView c, const int32_t *__restrict__ seqs,
                                                           const int32_t *__restrict__ start,
                                                           const int32_t *__restrict__ cu_keep,
                                                           const int32_t *__restrict__ keep, int64_t keep_len, int n) {
  pdl_enter();
  __shared__ MoveTable mt;
  for (int i = blockIdx.z; i < n; i += gridDim.z) {
    const Kept k = kept(c, seqs, start, cu_keep, keep_len, i);
    if (k.slot >= 0)
      move_tokens(c, k, keep, &mt, int(blockIdx.y), 1, int(blockIdx.x * kThreads + threadIdx.x), int(gridDim.x * kThreads));
  }
}

// Lengths and pages, after the moves; in small caches (kMoveInside) the moves too.  One block per sequence.
__global__ void __launch_bounds__(kThreads) kv_shrink_kernel(const KvView c, const int32_t *__restrict__ seqs,
                                                             const int32_t *__restrict__ start,
                                                             const int32_t *__restrict__ cu_keep,
                                                             const int32_t *__restrict__ keep, int64_t keep_len, int move) {
  pdl_enter();
  __shared__ MoveTable mt;
  const Kept k = kept(c, seqs, start, cu_keep, keep_len, blockIdx.x);
  if (k.slot < 0) return;
  if (move) move_tokens(c, k, keep, &mt, 0, c.layers, int(threadIdx.x), kThreads);
  __syncthreads();   // every thread has read the length and the table
  shrink(c, k);
}

struct Rows {
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t kt, kl, vt, vl, qt;
  const int32_t *cu, *seqs, *start, *pos;
  const float *cos_sin;
  int n, T, q_heads, rot, inter, layer;
  int64_t n_pos;
};

// A thread owns one unit (see rope.cu) of kItems of a token's 2 kv_heads + q_heads heads on one layer.  Where the
// token goes (its sequence, slot and page) is worked out once per block and token, under the latency of the
// data's loads.  grid: (units, layers).
template <typename T, int V, int MODE, int kItems>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvView c, const Rows r, int units, int turned) {
  pdl_enter();
  __shared__ int64_t slot_of[kThreads + 1];   // element offset in a layer of K of head 0, -1: not written
  const int D = c.head_dim, H = c.kv_heads, heads = 2 * H + r.q_heads;
  const unsigned groups = unsigned(heads + kItems - 1) / kItems, per = groups * unsigned(units);
  auto token = [&](int64_t x) { return (x >> 32) == 0 ? int64_t(unsigned(x) / per) : x / per; };
  const int64_t x0 = int64_t(blockIdx.x) * kThreads, x = x0 + threadIdx.x, t0 = token(x0), t = token(x);
  const unsigned in = unsigned(x - t * per), group = in / unsigned(units);
  const int unit = int(in - group * unsigned(units)), h0 = int(group) * kItems;
  const bool have = t < r.T;
  RopeUnit<T, V, MODE> u[kItems];
  const int layer = int(blockIdx.y);
  if (have) {
    const T *k = reinterpret_cast<const T *>(r.k) + layer * r.kl + t * r.kt;
    const T *v = reinterpret_cast<const T *>(r.v) + layer * r.vl + t * r.vt;
    const T *q = reinterpret_cast<const T *>(r.q) + t * r.qt;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int h = h0 + i;
      if (h < heads)
        u[i].load(h < H ? k + int64_t(h) * D : (h < 2 * H ? v + int64_t(h - H) * D : q + int64_t(h - 2 * H) * D), unit, turned,
                  r.rot);
    }
  }
  Angles<V, MODE> g;
  if (MODE != kRopeNone && have && unit < turned)
    load_angles<V, MODE>(g, r.cos_sin, r.n_pos, __ldg(r.pos + t), r.rot, unit, 0, [] {
      if (MOE_CHECKED) check_fail(kCheckPos);
    });
  const int64_t tk = t0 + threadIdx.x;   // the block's tokens
  if (tk <= token(x0 + kThreads - 1) && tk < r.T) {
    int64_t slot = -1;
    const int b = seq_of_row(r.cu, r.n, int(tk));
    if (b >= 0) {
      const int s = __ldg(r.seqs + b), st = __ldg(r.start + b);
      const int64_t at = int64_t(st) + tk - __ldg(r.cu + b);
      if (s >= 0 && s < c.slots && st >= 0 && (at >> c.page_shift) < c.max_pages) {
        const int p = valid_page(c, c.table[int64_t(s) * c.max_pages + (at >> c.page_shift)]);
        if (p >= 0) slot = (int64_t(p) * 2 * H * c.page_size() + (at & (c.page_size() - 1))) * D;
      }
    }
    slot_of[threadIdx.x] = slot;
  }
  __syncthreads();
  if (!have) return;
  const int64_t slot = slot_of[t - t0];
  T *pool = reinterpret_cast<T *>(c.pool) + int64_t(r.layer + layer) * c.layer_elems() + slot;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int h = h0 + i;
    if (h >= 2 * H) {
      if (h < heads)
        u[i].store(reinterpret_cast<T *>(r.q_out) + (t * r.q_heads + (h - 2 * H)) * D, unit, turned, r.rot, g);
    } else if (slot >= 0) {
      T *dst = pool + int64_t(h) * c.page_size() * D;
      if (h < H) u[i].store(dst, unit, turned, r.rot, g);
      else u[i].copy(dst, unit, turned, r.rot);
    }
  }
}

unsigned clamp_grid(int64_t v, int64_t most) { return unsigned(v < 1 ? 1 : (v < most ? v : most)); }

int check_ids(const void *a, const void *b, int64_t n) {
  MOE_REQUIRE(n >= 0 && n < (int64_t(1) << 22), "need 0 <= n < 2^22 (%lld)", (long long)n);
  if (n == 0) return MOE_OK;
  MOE_REQUIRE(a && b, "null pointer argument");
  MOE_REQUIRE(aligned16(a) && aligned16(b), "pointers must be 16-byte aligned");
  return MOE_OK;
}

// Blocks of a page-copy kernel for at most n copies: enough to fill the SMs, no more than there are pieces.
dim3 page_grid(const KvView &c, int64_t n) {
  return dim3(clamp_grid(cdiv(2 * c.half_elems() / 8, kPiece) * c.layers * n, int64_t(num_sms()) * 8));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_extend_workspace_size(const moe_kv_desc *desc, int64_t n) {
  if (check_kv_desc(desc) != MOE_OK || n < 0 || n >= (int64_t(1) << 22)) return 0;
  return align256(size_t(n + 1) * 4) + align256(size_t(n) * 8) + align256(size_t(desc->pages) * 4);
}

extern "C" int moe_kv_extend(const moe_kv_desc *desc, const moe_kv *kv, const int32_t *seqs, const int32_t *n_new,
                             int64_t n, int32_t *start, void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_ids(seqs, n_new, n));
  if (n == 0) return MOE_OK;
  MOE_REQUIRE(start && aligned16(start), "start must be non-null and 16-byte aligned");
  const size_t need = moe_kv_extend_workspace_size(desc, n);
  MOE_REQUIRE(workspace && aligned16(workspace), "workspace must be non-null and 16-byte aligned");
  if (workspace_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "cache extend workspace %zu < %zu bytes", workspace_bytes, need);
  const KvView c = kv_view(desc, kv);
  char *ws = static_cast<char *>(workspace);
  ExtendWs w{reinterpret_cast<int32_t *>(ws), reinterpret_cast<int32_t *>(ws + align256(size_t(n + 1) * 4)),
             reinterpret_cast<int32_t *>(ws + align256(size_t(n + 1) * 4) + align256(size_t(n) * 8))};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  launch_pdl(kv_extend_kernel, dim3(1), dim3(kBook), 0, st, c, seqs, n_new, int(n), start, w);
  MOE_TRY(check_launch("kv_extend"));
  launch_pdl(kv_cow_kernel, page_grid(c, n), dim3(kThreads), 0, st, c, static_cast<const int32_t *>(w.cow), int(n));
  return check_launch("kv_extend: copy on write");
}

extern "C" int moe_kv_fork(const moe_kv_desc *desc, const moe_kv *kv, const int32_t *src, const int32_t *dst, int64_t n,
                           moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_ids(src, dst, n));
  if (n == 0) return MOE_OK;
  launch_pdl(kv_fork_kernel, dim3(unsigned(n)), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), kv_view(desc, kv),
             src, dst);
  return check_launch("kv_fork");
}

extern "C" int moe_kv_free(const moe_kv_desc *desc, const moe_kv *kv, const int32_t *seqs, int64_t n, moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_ids(seqs, seqs, n));
  if (n == 0) return MOE_OK;
  launch_pdl(kv_free_kernel, dim3(unsigned(n)), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), kv_view(desc, kv),
             seqs);
  return check_launch("kv_free");
}

extern "C" int moe_kv_compact(const moe_kv_desc *desc, const moe_kv *kv, const int32_t *seqs, const int32_t *start,
                              const int32_t *cu_keep, const int32_t *keep, int64_t keep_len, int64_t n,
                              moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_ids(seqs, start, n));
  MOE_REQUIRE(keep_len >= 0 && keep_len < (int64_t(1) << 31), "keep_len out of range");
  if (n == 0) return MOE_OK;
  MOE_REQUIRE(cu_keep && (keep || keep_len == 0), "null pointer argument");
  MOE_REQUIRE(aligned16(cu_keep) && aligned16(keep), "pointers must be 16-byte aligned");
  const KvView c = kv_view(desc, kv);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // One launch where a sequence's rows of all layers are few enough for a block (up to kMoveInside pieces of 16 bytes
  // per token): the second launch costs more than the lost parallelism.  Extend, compaction and roll back of 4 sequences
  // with 13 drafted tokens, one launch against two: 9.2 and 10.3 us with 32 pieces, 10.3 and 10.8 with 512, 10.8 both with
  // 768, 13.3 and 10.8 with 2048; of 24 sequences with 24 tokens 10.7 and 11.8 with 256, 11.8 both with 512, 18.5 and 13.1
  // with 2048.
  constexpr int64_t kMoveInside = 512;
  const int64_t pieces = int64_t(2) * c.kv_heads * (c.head_dim / 8);
  const bool inside = pieces * c.layers <= kMoveInside;
  if (keep_len > 0 && !inside) {
    const dim3 grid(clamp_grid(cdiv(pieces, kThreads), 1024), unsigned(c.layers), clamp_grid(n, 65535));
    launch_pdl(kv_move_kernel, grid, dim3(kThreads), 0, st, c, seqs, start, cu_keep, keep, keep_len, int(n));
    MOE_TRY(check_launch("kv_compact"));
  }
  launch_pdl(kv_shrink_kernel, dim3(unsigned(n)), dim3(kThreads), 0, st, c, seqs, start, cu_keep, keep, keep_len,
             int(inside && keep_len > 0));
  return check_launch("kv_compact: pages");
}

extern "C" int moe_kv_copy(const moe_kv_desc *desc, const moe_kv *kv, const int32_t *src, const int32_t *dst, int64_t n,
                           moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_ids(src, dst, n));
  if (n == 0) return MOE_OK;
  const KvView c = kv_view(desc, kv);
  launch_pdl(kv_copy_kernel, page_grid(c, n), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), c, src, dst, int(n));
  return check_launch("kv_copy");
}

extern "C" int moe_kv_append(const moe_kv_desc *desc, const moe_kv *kv, int64_t layer, int64_t n_layers,
                             const moe_kv_rows *rows, moe_stream_t stream) {
  MOE_TRY(check_kv(desc, kv));
  MOE_REQUIRE(rows != nullptr, "rows is NULL");
  const moe_kv_rows &r = *rows;
  MOE_REQUIRE(layer >= 0 && n_layers >= 1 && layer + n_layers <= desc->layers, "layers [%lld, %lld) are not in the cache",
              (long long)layer, (long long)(layer + n_layers));
  MOE_REQUIRE(r.T >= 0 && r.T < (int64_t(1) << 30), "T out of range");
  MOE_TRY(check_ids(r.seqs, r.start, r.n));
  MOE_REQUIRE(r.k_token_stride >= 0 && r.v_token_stride >= 0 && r.k_layer_stride >= 0 && r.v_layer_stride >= 0 &&
                  r.k_token_stride % 8 == 0 && r.v_token_stride % 8 == 0 && r.k_layer_stride % 8 == 0 &&
                  r.v_layer_stride % 8 == 0,
              "strides must be non-negative multiples of 8");
  MOE_REQUIRE(r.q == nullptr || (r.cos_sin != nullptr && n_layers == 1), "q needs cos_sin and a single layer");
  if (r.T == 0 || (r.n == 0 && r.q == nullptr)) return MOE_OK;
  MOE_REQUIRE(r.k && r.v && (r.cu || r.n == 0), "null pointer argument");
  MOE_REQUIRE(aligned16(r.k) && aligned16(r.v) && aligned16(r.cu), "pointers must be 16-byte aligned");
  if (r.cos_sin) {
    MOE_REQUIRE(r.pos && aligned16(r.pos) && aligned16(r.cos_sin), "pos must be non-null, pos and cos_sin 16-byte aligned");
    MOE_REQUIRE(r.rot >= 2 && r.rot % 2 == 0 && r.rot <= desc->head_dim, "rot must be even, 2 <= rot <= head_dim (rot=%lld)",
                (long long)r.rot);
    MOE_REQUIRE(r.n_pos >= 1 && r.n_pos < (int64_t(1) << 31), "n_pos out of range");
  }
  if (r.q) {
    MOE_REQUIRE(r.q_heads >= 1 && r.q_heads <= 65536, "q_heads out of range");
    MOE_REQUIRE(r.q_token_stride >= 0 && r.q_token_stride % 8 == 0, "strides must be non-negative multiples of 8");
    MOE_REQUIRE(r.q_out && aligned16(r.q) && aligned16(r.q_out) && r.q != r.q_out,
                "q_out must be non-null, apart from q, both 16-byte aligned");
  }
  const KvView c = kv_view(desc, kv);
  Rows a{};
  a.k = static_cast<const uint16_t *>(r.k);
  a.v = static_cast<const uint16_t *>(r.v);
  a.q = static_cast<const uint16_t *>(r.q);
  a.q_out = static_cast<uint16_t *>(r.q_out);
  a.kt = r.k_token_stride;
  a.kl = r.k_layer_stride;
  a.vt = r.v_token_stride;
  a.vl = r.v_layer_stride;
  a.qt = r.q_token_stride;
  a.cu = r.cu;
  a.seqs = r.seqs;
  a.start = r.start;
  a.pos = r.pos;
  a.cos_sin = r.cos_sin;
  a.n = int(r.n);
  a.T = int(r.T);
  a.q_heads = r.q ? int(r.q_heads) : 0;
  a.rot = r.cos_sin ? int(r.rot) : 0;
  a.inter = r.interleaved ? 1 : 0;
  a.layer = int(layer);
  a.n_pos = r.n_pos;
  // without rotation every vector is a copy
  const int V = r.cos_sin ? rope_vec(2, r.rot, r.interleaved) : 8;
  const int units = rope_units(V, int(desc->head_dim), a.rot, a.inter);   // rot 0 without rotation
  const int turned = (a.inter ? a.rot : a.rot / 2) / V;
  const int64_t heads = 2 * desc->kv_heads + a.q_heads;
  const int mode = !a.cos_sin ? kRopeNone : (a.inter ? kRopeInter : kRopeHalf);
  const bool many = r.T * heads * units * n_layers >= int64_t(num_sms()) * 1024 * (mode == kRopeHalf ? 4 : 8);   // as in moe_rope
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto typed = [&](auto zero) -> int {
    return rope_dispatch<2>(mode, V, many, [&](auto m, auto vec, auto per) -> int {
      const int64_t blocks = cdiv(r.T * cdiv(heads, int64_t(decltype(per)::value)) * units, kThreads);
      MOE_SUPPORT(blocks < (int64_t(1) << 31), "T * heads too large");
      launch_pdl(kv_append_kernel<decltype(zero), decltype(vec)::value, decltype(m)::value, decltype(per)::value>,
                 dim3(unsigned(blocks), unsigned(n_layers)), dim3(kThreads), 0, st, c, a, units, turned);
      return MOE_OK;
    });
  };
  MOE_TRY(desc->dtype == MOE_F16 ? typed(__half{}) : typed(__nv_bfloat16{}));
  return check_launch("kv_append");
}
