// Attention of new tokens over the paged cache: drafted trees (a bit mask per token) and prompts
// (causal), grouped query heads.
//
//   s_j = scale q . k_j over the visible keys j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j).
//
// One pass over the keys with a running maximum and sum: when the maximum grows, what has been
// summed so far is scaled down.
#include "kv_internal.cuh"

namespace moe {

MOE_DEFINE_CHECK_WORD(attn)

namespace {

constexpr int kThreads = 128;

struct Rows {
  const uint16_t *q;
  int64_t qt;
  const int32_t *cu, *seqs, *start;
  const uint32_t *mask;
  uint16_t *out;
  float *lse;
  int n, T, q_heads, words, layer;
  float scale_log2;   // scale * log2(e): the exponentials are taken to base 2
};

// One warp per (row, query head); a lane scores one key of 32, then owns head_dim / 32 output
// elements for the weighted sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_simple_kernel(const KvView c, const Rows r) {
  pdl_enter();
  __shared__ float qs[kThreads / 32][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = int64_t(blockIdx.x) * (kThreads / 32) + warp;
  if (item >= int64_t(r.T) * r.q_heads) return;
  const int t = int(item / r.q_heads), h = int(item - int64_t(t) * r.q_heads), D = c.head_dim;
  const int b = seq_of_row(r.cu, r.n, t);
  if (b < 0) return;
  const T *q = reinterpret_cast<const T *>(r.q) + t * r.qt + int64_t(h) * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = to_f32(q[d]);
  __syncwarp();
  const int slot = r.seqs[b], start = r.start[b], i = t - r.cu[b], nq = r.cu[b + 1] - r.cu[b];
  int64_t keys = 0;
  if (slot >= 0 && slot < c.slots && start >= 0) {
    keys = int64_t(start) + (r.mask ? nq : i + 1);
    keys = min(keys, int64_t(c.max_pages) << c.page_shift);
  }
  const uint32_t *bits = r.mask ? r.mask + int64_t(t) * r.words : nullptr;
  if (r.mask) {
    bool any = false;
    for (int w = 0; w < r.words; ++w) any |= bits[w] != 0;
    if (!any) keys = 0;
  }
  const int32_t *tab = c.table + int64_t(max(slot, 0)) * c.max_pages;
  const int H = c.kv_heads, hk = h / (r.q_heads / H);
  const T *pool = reinterpret_cast<const T *>(c.pool) + r.layer * c.layer_elems();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t j0 = 0; j0 < keys; j0 += 32) {
    const int64_t j = j0 + lane;
    bool see = j < keys;
    if (see && bits && j >= start) {
      const int64_t a = j - start;
      see = a < int64_t(r.words) * 32 && ((bits[a >> 5] >> (a & 31)) & 1u);
    }
    const T *krow = nullptr;
    if (see) {
      const int p = tab[j >> c.page_shift];
      if (p >= 0 && p < c.pages)
        krow = pool + ((int64_t(p) * 2 * H + hk) * c.page_size() + (j & (c.page_size() - 1))) * D;
      else if (MOE_CHECKED) check_fail(kCheckPage);
    }
    float s = 0.f;
    if (krow)
      for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], to_f32(krow[d]), s);
    s = see ? s * r.scale_log2 : -INFINITY;
    float top = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
    const float down = exp2f(m - base), p = exp2f(s - base);
    l *= down;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= down;
    m = mn;
    float sum = p;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    l += sum;
    const int64_t vofs = int64_t(H) * c.page_size() * D;   // V lies behind the page's K
    for (int k = 0; k < 32; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      const T *kr = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(krow), k));
      if (!kr) continue;   // not visible: not read
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (lane + 32 * x < D) o[x] = fmaf(pk, to_f32(kr[vofs + lane + 32 * x]), o[x]);
    }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (lane + 32 * x < D)
      reinterpret_cast<T *>(r.out)[(int64_t(t) * r.q_heads + h) * D + lane + 32 * x] = from_f32<T>(o[x] * inv);
  if (r.lse && lane == 0) r.lse[int64_t(t) * r.q_heads + h] = (m + log2f(l)) * 0.6931471805599453f;
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
  if (check_attention(desc, T, n, q_heads) != MOE_OK) return 0;
  return 0;
}

extern "C" int moe_attention(const moe_kv_desc *desc, const moe_kv *kv, int64_t layer, const void *q,
                             int64_t q_token_stride, int64_t q_heads, int64_t T, const int32_t *cu, const int32_t *seqs,
                             const int32_t *start, int64_t n, const uint32_t *mask, int64_t mask_words, float scale,
                             void *out, float *lse, void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  MOE_TRY(check_kv(desc, kv));
  MOE_TRY(check_attention(desc, T, n, q_heads));
  MOE_REQUIRE(layer >= 0 && layer < desc->layers, "layer %lld is not in the cache", (long long)layer);
  MOE_REQUIRE(q_token_stride >= 0 && q_token_stride % 8 == 0, "strides must be non-negative multiples of 8");
  MOE_REQUIRE(mask == nullptr || (mask_words >= 1 && mask_words <= 1024), "need 1 <= mask_words <= 1024 (%lld)",
              (long long)mask_words);
  MOE_REQUIRE(scale > 0.f && scale <= 3.0e38f, "scale must be positive and finite");
  if (T == 0 || n == 0) return MOE_OK;
  MOE_REQUIRE(q && cu && seqs && start && out, "null pointer argument");
  MOE_REQUIRE(aligned16(q) && aligned16(cu) && aligned16(seqs) && aligned16(start) && aligned16(mask) && aligned16(out) &&
                  aligned16(lse),
              "pointers must be 16-byte aligned");
  Rows r{};
  r.q = static_cast<const uint16_t *>(q);
  r.qt = q_token_stride;
  r.cu = cu;
  r.seqs = seqs;
  r.start = start;
  r.mask = mask;
  r.out = static_cast<uint16_t *>(out);
  r.lse = lse;
  r.n = int(n);
  r.T = int(T);
  r.q_heads = int(q_heads);
  r.words = int(mask_words);
  r.layer = int(layer);
  r.scale_log2 = scale * 1.4426950408889634f;
  const int64_t blocks = cdiv(T * q_heads, kThreads / 32);
  MOE_SUPPORT(blocks < (int64_t(1) << 31), "T * q_heads too large");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvView c = kv_view(desc, kv);
  if (desc->dtype == MOE_F16) launch_pdl(attn_simple_kernel<__half>, dim3(unsigned(blocks)), dim3(kThreads), 0, st, c, r);
  else launch_pdl(attn_simple_kernel<__nv_bfloat16>, dim3(unsigned(blocks)), dim3(kThreads), 0, st, c, r);
  return check_launch("attention");
}
