// Shared by the attention-side translation units (rope.cu, kv.cu, attn.cu): the cache's
// geometry on the device, the row -> sequence search and the rotation of one pair.
#pragma once

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

}  // namespace moe
