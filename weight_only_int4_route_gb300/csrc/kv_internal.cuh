// Shared by the attention-side translation units (rope.cu, kv.cu, attn.cu): the cache's
// geometry on the device, the row -> sequence search and the rotation of one pair.
#pragma once

#include <type_traits>

#include "moe_internal.cuh"

namespace moe {

enum : int { kCheckPage = 8, kCheckPos = 16 };

int check_word_take_rope(int *out);
int check_word_take_kv(int *out);
int check_word_take_attn(int *out);
int attn_error_take(int *out);   // device error word of the attention kernel

inline bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int check_kv_desc(const moe_kv_desc *d);
int check_kv(const moe_kv_desc *d, const moe_kv *kv);

// The cache as the kernels see it.  Offsets into the pool are 64-bit (a pool exceeds 2^31 elements
// from a few GB on).
struct KvView {
  uint16_t *pool;
  int32_t *table, *lens, *refs;
  int layers, pages, page_shift, kv_heads, head_dim, slots, max_pages;
  __host__ __device__ int page_size() const { return 1 << page_shift; }
  // elements of one (page, K or V): kv_heads x page_size x head_dim
  __host__ __device__ int64_t half_elems() const { return int64_t(kv_heads) * page_size() * head_dim; }
  __host__ __device__ int64_t layer_elems() const { return int64_t(pages) * 2 * half_elems(); }
};

inline KvView kv_view(const moe_kv_desc *d, const moe_kv *kv) {
  KvView v{};
  v.pool = static_cast<uint16_t *>(kv->pool);
  v.table = kv->table;
  v.lens = kv->lens;
  v.refs = kv->refs;
  v.layers = int(d->layers);
  v.pages = int(d->pages);
  while ((int64_t(1) << v.page_shift) < d->page_size) ++v.page_shift;
  v.kv_heads = int(d->kv_heads);
  v.head_dim = int(d->head_dim);
  v.slots = int(d->slots);
  v.max_pages = int(d->max_pages);
  return v;
}

// Sequence that owns packed row r: the i with cu[i] <= r < cu[i + 1], or -1.
__device__ __forceinline__ int seq_of_row(const int32_t *__restrict__ cu, int n, int r) {
  if (n < 1 || r < __ldg(cu) || r >= __ldg(cu + n)) return -1;
  int lo = 0, hi = n - 1;   // the last i with cu[i] <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ---- rotation of heads in vectors of V elements (16 bytes where the sizes allow)

// Moved as one word of its size (an array of 16-bit values would be moved value by value).
template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <typename T, int V> struct Pack {
  using W = typename Word<int(sizeof(T)) * V>::type;
  W w;
  __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const W *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<W *>(p) = w; }
  __device__ __forceinline__ float get(int i) const { return to_f32(reinterpret_cast<const T *>(&w)[i]); }
  __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<T *>(&w)[i] = from_f32<T>(x); }
};

// Largest vector, in elements, that divides what has to be divided: half-layout pairs lie rot / 2 apart, interleaved
// ones side by side; head_dim is a multiple of 8.
inline int rope_vec(int elem_bytes, int64_t rot, int interleaved) {
  const int64_t unit = interleaved ? rot : rot / 2;
  int v = 16 / elem_bytes;
  while (v > 1 && unit % v != 0) v /= 2;
  return v;   // interleaved: rot is even, so at least 2
}

enum : int { kRopeNone = 0, kRopeHalf = 1, kRopeInter = 2 };   // none: heads are copied

// Units of a head: its rotated vectors (pairs of vectors in the half layout), then the vectors that are copied.
__host__ __device__ inline int rope_units(int V, int head_dim, int rot, int inter) {
  return (inter ? rot : rot / 2) / V + (head_dim - rot) / V;
}

// The cosines and sines of one unit: V of each (half layout) or V / 2 (interleaved).  NaN for positions outside
// the table.
template <int V, int MODE> struct Angles {
  static constexpr int kN = MODE == kRopeNone ? 0 : (MODE == kRopeInter ? V / 2 : V);
  float c[kN > 0 ? kN : 1], s[kN > 0 ? kN : 1];
};
template <int V, int MODE, typename Bad>
__device__ __forceinline__ void load_angles(Angles<V, MODE> &a, const float *cos_sin, int64_t n_pos, int p, int rot, int unit,
                                            int inverse, Bad bad) {
  constexpr int n = Angles<V, MODE>::kN;
  const bool inside = p >= 0 && p < n_pos;
  if (!inside) bad();
  const float *row = cos_sin + int64_t(inside ? p : 0) * rot + unit * n;
  // rows start at multiples of rot, even: pairs are read together where rot / 2 is even too
  if (n >= 2 && (rot & 3) == 0) {
#pragma unroll
    for (int i = 0; i + 1 < n; i += 2) {
      const float2 c = __ldg(reinterpret_cast<const float2 *>(row + i));
      const float2 s = __ldg(reinterpret_cast<const float2 *>(row + rot / 2 + i));
      a.c[i] = c.x;
      a.c[i + 1] = c.y;
      a.s[i] = s.x;
      a.s[i + 1] = s.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      a.c[i] = __ldg(row + i);
      a.s[i] = __ldg(row + rot / 2 + i);
    }
  }
#pragma unroll
  for (int i = 0; i < n; ++i) {
    a.c[i] = inside ? a.c[i] : NAN;
    a.s[i] = inside ? (inverse ? -a.s[i] : a.s[i]) : NAN;
  }
}

// One unit: (a, b) -> (a c - b s, a s + b c) in fp32, one rounding; units past the rotated ones are copied.
template <typename T, int V, int MODE> struct RopeUnit {
  Pack<T, V> a, b;
  __device__ __forceinline__ void load(const T *src, int unit, int turned, int rot) {
    if (MODE != kRopeNone && unit < turned) {
      a.load(src + unit * V);
      if (MODE == kRopeHalf) b.load(src + rot / 2 + unit * V);
    } else {
      a.load(src + rot + (unit - turned) * V);
    }
  }
  __device__ __forceinline__ void copy(T *dst, int unit, int turned, int rot) const {   // the unit as it is
    if (MODE == kRopeNone || unit >= turned) {
      a.store(dst + rot + (unit - turned) * V);
    } else {
      a.store(dst + unit * V);
      if (MODE == kRopeHalf) b.store(dst + rot / 2 + unit * V);
    }
  }
  __device__ __forceinline__ void store(T *dst, int unit, int turned, int rot, const Angles<V, MODE> &g) const {
    if (MODE == kRopeNone || unit >= turned) {
      a.store(dst + rot + (unit - turned) * V);
    } else if constexpr (MODE == kRopeInter) {
      Pack<T, V> y;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float x0 = a.get(2 * i), x1 = a.get(2 * i + 1);
        y.set(2 * i, x0 * g.c[i] - x1 * g.s[i]);
        y.set(2 * i + 1, x0 * g.s[i] + x1 * g.c[i]);
      }
      y.store(dst + unit * V);
    } else if constexpr (MODE == kRopeHalf) {
      Pack<T, V> y, z;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x0 = a.get(i), x1 = b.get(i);
        y.set(i, x0 * g.c[i] - x1 * g.s[i]);
        z.set(i, x0 * g.s[i] + x1 * g.c[i]);
      }
      y.store(dst + unit * V);
      z.store(dst + rot / 2 + unit * V);
    }
  }
};

// Launch helper: go(MODE, V, items a thread) as compile-time constants.  items: 128 bytes of loads (a unit of the half
// layout is two vectors) in large calls, one unit in small ones.
template <int BYTES, typename Go> int rope_dispatch(int mode, int V, bool many, Go go) {
  auto with = [&](auto m, auto v) -> int {
    constexpr int kMany = decltype(m)::value == kRopeHalf ? 4 : 8;
    return many ? go(m, v, std::integral_constant<int, kMany>()) : go(m, v, std::integral_constant<int, 1>());
  };
  auto with_vec = [&](auto m) -> int {
    if constexpr (BYTES == 2)
      if (V == 8) return with(m, std::integral_constant<int, 8>());
    if (V == 4) return with(m, std::integral_constant<int, 4>());
    if constexpr (decltype(m)::value == kRopeHalf)
      if (V == 1) return with(m, std::integral_constant<int, 1>());
    return with(m, std::integral_constant<int, 2>());
  };
  if (mode == kRopeNone) return with(std::integral_constant<int, kRopeNone>(), std::integral_constant<int, 16 / BYTES>());
  if (mode == kRopeHalf) return with_vec(std::integral_constant<int, kRopeHalf>());
  return with_vec(std::integral_constant<int, kRopeInter>());
}

}  // namespace moe
