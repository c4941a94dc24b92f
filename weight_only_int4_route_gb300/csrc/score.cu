// Log probabilities of given tokens, entropy and top alternatives of rows of logits.
//
// With z_j = scale * x_j, in powers of two (c = scale log2 e):
//   lse = ln sum_j exp z_j,  logprob_t = z_t - lse,  entropy = lse - sum_j p_j z_j
// One pass over the row: every thread keeps its largest logit m, the reference M = fl(m c), Z = sum 2^(x c - M) and
// S = sum 2^(x c - M) (x c - M), and moves them when m grows: Z' = Z 2^(M - M'), S' = 2^(M - M') (S + (M - M') Z).
// M is one fp32 number that every later step uses, so its rounding is in no result.  entropy = ln 2 (log2 Z - S / Z): S <= 0, so
// nothing cancels.
//
// Top alternatives, in the order of (logit descending, id ascending): a thread knows its best element.  The threads are cut
// into G >= k groups; the smallest of the groups' best elements has at least k elements at or above it, so only elements from it
// on can be among the k, and only threads whose best element is have any.  Those threads' elements are read again (from the
// L2, a few per cent of the row), what passes is collected, and an element's place is the number of elements before it.
// Where the row is laid out so that too many pass, the k best are found one after the other.
//
// Few long rows are shared by the CTAs of a cluster, which send their sums and their k best to the first one.
// Bound by memory for many rows, by the length of this chain for a few.
#include <type_traits>

#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxK = 64;
// Elements collected at most.  What a row of equal logits passes, or all there are if some thread has none, fits: 8 x 256
// and up to 14 single elements at the ends.
constexpr int kCand = 2112;
constexpr int kMaxParts = 8;        // CTAs of a row (the portable cluster size)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct ScoreArgs {
  const void *x;
  int64_t stride;
  const int32_t *ids;
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t *top_ids;
  float scale;
  int V, n_ids, k;
};

template <typename T, int N> struct alignas(16) Vec {
  T v[N];
};

// Order of elements as one unsigned number: logits descending, then ids ascending; 0 is before no element.  -0 and 0 are equal.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t id) {
  uint32_t b = __float_as_uint(x + 0.f);
  b = b & 0x80000000u ? ~b : b | 0x80000000u;
  return uint64_t(b) << 32 | uint32_t(~id);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = uint32_t(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint32_t key_id(uint64_t key) { return ~uint32_t(key); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) { return __shfl_xor_sync(0xffffffffu, (unsigned long long)v, o); }

// Sums of a set of elements: largest logit, Z and S relative to M = fl(m c).  m is NaN if any element is.
struct Sums {
  float m, z, s;
};
// The reference of a largest logit; an empty side's is 0, so that x c - M stays -inf.
__device__ __forceinline__ float reference(float m, float c) { return m == -INFINITY ? 0.f : __fmul_rn(m, c); }
// b into a.
__device__ __forceinline__ void join(Sums &a, const Sums &b, float c) {
  const float m = max_nan(a.m, b.m), M = reference(m, c);
  auto moved = [&](const Sums &o, float &z, float &s) {
    const float d = __fsub_rn(reference(o.m, c), M), f = ex2(d);
    z = o.z == 0.f ? 0.f : o.z * f;
    s = o.z == 0.f ? 0.f : f * fmaf(d, o.z, o.s);
  };
  float za, sa, zb, sb;
  moved(a, za, sa);
  moved(b, zb, sb);
  a = {m, za + zb, sa + sb};
}

// What a CTA of a cluster sends to the first one.
struct Part {
  uint64_t best[kMaxK];
  Sums sums;
};

template <typename T, int PARTS>
__global__ void __launch_bounds__(kThreads, 4) score_kernel(const ScoreArgs p) {
  pdl_enter();
  constexpr int VE = 16 / int(sizeof(T));
  using V4 = Vec<T, VE>;
  __shared__ Part parts[PARTS];
  __shared__ uint64_t cand[kCand];
  __shared__ uint64_t s_key[kWarps];
  __shared__ Sums s_sums[kWarps];
  __shared__ uint8_t s_lane[kWarps][32];
  __shared__ int s_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = PARTS > 1 ? int(cluster_rank()) : 0;
  const int64_t row = blockIdx.x / PARTS;
  if (PARTS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");   // all have started: waited for below
  const T *x = static_cast<const T *>(p.x) + row * p.stride;
  const float c = p.scale * kLog2e;
  // single elements up to the first 16-byte boundary and after the last, vectors between
  const int head = min(p.V, int((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / int(sizeof(T)));
  const int nv = (p.V - head) / VE, tail = p.V - head - nv * VE;
  const int per = (nv + PARTS - 1) / PARTS, v0 = min(nv, part * per), v1 = min(nv, v0 + per);
  const V4 *vec = reinterpret_cast<const V4 *>(x + head);
  const bool has_head = part == 0 && tid < head, has_tail = part == 0 && tid < tail;
  const int tail_id = head + nv * VE + tid;

  Sums u = {-INFINITY, 0.f, 0.f};
  float M = 0.f;
  // the thread's best element; its first one where all are -inf
  int best = has_head ? tid : (v0 + tid < v1 ? head + (v0 + tid) * VE : (has_tail ? tail_id : -1));
  auto take = [&](auto n, const float *e, int id) {
    constexpr int N = decltype(n)::value;
    float top = e[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = max_nan(top, e[j]);
    if (!(top <= u.m)) {
      const float m = max_nan(u.m, top), Mn = reference(m, c), d = __fsub_rn(M, Mn);
      if (u.z != 0.f) {
        const float f = ex2(d);
        u.s = f * fmaf(d, u.z, u.s);
        u.z *= f;
      }
      u.m = m;
      M = Mn;
#pragma unroll
      for (int j = N - 1; j >= 0; --j)
        if (e[j] == top) best = id + j;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      // 0 times -inf would be NaN: an exponent this low is 0 as well
      const float t = fmaxf(fmaf(e[j], c, -M), -1e4f), w = ex2(t);
      u.z += w;
      u.s = fmaf(w, t, u.s);
    }
  };
  auto one = [&](int id) {
    const float e = to_f32(x[id]);
    take(std::integral_constant<int, 1>{}, &e, id);
  };
  if (has_head) one(tid);
  constexpr int kBatch = 4;   // loads in flight
  for (int v = v0 + tid; v < v1; v += kBatch * kThreads) {
    V4 r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (v + i * kThreads < v1) r[i] = vec[v + i * kThreads];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (v + i * kThreads < v1) {
        float e[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) e[j] = to_f32(r[i].v[j]);
        take(std::integral_constant<int, VE>{}, e, head + (v + i * kThreads) * VE);
      }
  }
  if (has_tail) one(tail_id);

  // ---- the CTA's sums
  const float own_m = u.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b = {__shfl_xor_sync(0xffffffffu, u.m, o), __shfl_xor_sync(0xffffffffu, u.z, o), __shfl_xor_sync(0xffffffffu, u.s, o)};
    join(u, b, c);
  }
  if (lane == 0) s_sums[warp] = u;
  const uint64_t key = p.k > 0 && best >= 0 ? key_of(own_m, uint32_t(best)) : 0;
  uint64_t from = key;
  // groups of 32, 16, 8 or 4 threads: their best elements, the smallest of them
  const int wide = p.k <= 8 ? 32 : (p.k <= 16 ? 16 : (p.k <= 32 ? 8 : 4));
  for (int o = 1; o < wide; o <<= 1) from = max(from, shfl_xor64(from, o));
  for (int o = wide; o < 32; o <<= 1) from = min(from, shfl_xor64(from, o));
  if (lane == 0) s_key[warp] = from;
  if (tid == 0) s_n = 0;
  if (tid < p.k) parts[part].best[tid] = 0;
  __syncthreads();
  u = s_sums[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) join(u, s_sums[w], c);

  // ---- the CTA's k best (a row that holds a NaN has none)
  if (p.k > 0 && u.m == u.m) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) from = min(from, s_key[w]);
    auto offer = [&](float e, int id) {
      const uint64_t mine = key_of(e, uint32_t(id));
      if (mine >= from) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kCand) cand[at] = mine;
      }
    };
    const unsigned who = __ballot_sync(0xffffffffu, key != 0 && key >= from);
    if (who >> lane & 1) s_lane[warp][__popc(who & ((1u << lane) - 1))] = uint8_t(lane);
    __syncwarp();
    if (has_head) offer(to_f32(x[tid]), tid);
    if (has_tail) offer(to_f32(x[tail_id]), tail_id);
    const int each = (v1 - v0 + kThreads - 1) / kThreads, total = __popc(who) * each;
    for (int i = lane; i < total; i += 32) {
      const int n = i / each, v = v0 + warp * 32 + s_lane[warp][n] + (i - n * each) * kThreads;
      if (v >= v1) continue;
      const V4 r = vec[v];
#pragma unroll
      for (int j = 0; j < VE; ++j) offer(to_f32(r.v[j]), head + v * VE + j);
    }
    __syncthreads();
    const int n = s_n;
    if (n <= kCand) {
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t mine = cand[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += cand[j] > mine;
        if (place < p.k) parts[part].best[place] = mine;
      }
    } else {
      // one after the other: the best element after the last one found
      uint64_t last = ~uint64_t(0);
      for (int found = 0; found < p.k && last != 0; ++found) {
        uint64_t mine = 0;
        auto look = [&](float e, int id) {
          const uint64_t o = key_of(e, uint32_t(id));
          if (o < last) mine = max(mine, o);
        };
        if (has_head) look(to_f32(x[tid]), tid);
        if (has_tail) look(to_f32(x[tail_id]), tail_id);
        for (int v = v0 + tid; v < v1; v += kThreads) {
          const V4 r = vec[v];
#pragma unroll
          for (int j = 0; j < VE; ++j) look(to_f32(r.v[j]), head + v * VE + j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine = max(mine, shfl_xor64(mine, o));
        __syncthreads();
        if (lane == 0) s_key[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mine = max(mine, s_key[w]);
        last = mine;
        if (tid == 0) parts[part].best[found] = mine;
      }
    }
  }

  // ---- the row's: every CTA's to the first one
  if (PARTS > 1) {
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    if (part != 0) {
      if (tid < p.k) {
        const uint32_t to = map_to_rank(&parts[part].best[tid], 0);
        asm volatile("st.shared::cluster.b64 [%0], %1;\n" ::"r"(to), "l"(parts[part].best[tid]) : "memory");
      }
      if (tid == 0) {
        const uint32_t to = map_to_rank(&parts[part].sums, 0);
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to), "f"(u.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + 4), "f"(u.z) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + 8), "f"(u.s) : "memory");
      }
    }
    __syncwarp();
    cluster_sync();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < PARTS; ++w) join(u, parts[w].sums, c);
  } else {
    __syncthreads();
  }

  const float Mr = reference(u.m, c), nan = __int_as_float(0x7fc00000);
  const float lz = log2f(u.z);
  auto logprob = [&](float e) {
    if (u.m != u.m) return nan;
    if (u.m == -INFINITY) return -INFINITY;
    if (u.m == INFINITY) return e == INFINITY ? nan : -INFINITY;
    return (fmaf(e, c, -Mr) - lz) * kLn2;
  };
  for (int i = tid; i < p.n_ids; i += kThreads) {
    const int id = p.ids[row * p.n_ids + i];
    p.logprob[row * p.n_ids + i] = id >= 0 && id < p.V ? logprob(to_f32(x[id])) : nan;
  }
  if (tid == 0) {
    const bool finite = fabsf(u.m) < INFINITY;
    if (p.lse) p.lse[row] = finite ? (Mr + lz) * kLn2 : u.m;
    if (p.entropy) p.entropy[row] = finite ? (lz - u.s / u.z) * kLn2 : (u.m == -INFINITY ? 0.f : nan);
  }
  const int there = u.m == u.m ? min(p.k, p.V) : 0;
  for (int i = tid; i < PARTS * p.k; i += kThreads) {
    const uint64_t mine = parts[i / p.k].best[i % p.k];
    int place = 0;
    if (PARTS == 1) place = i;
    else
      for (int w = 0; w < PARTS; ++w)
        for (int j = 0; j < p.k; ++j) place += parts[w].best[j] > mine;
    if (mine != 0 && place < there) {
      p.top_ids[row * p.k + place] = int(key_id(mine));
      p.top_logprob[row * p.k + place] = logprob(key_value(mine));
    }
  }
  for (int i = there + tid; i < p.k; i += kThreads) {
    p.top_ids[row * p.k + i] = -1;
    p.top_logprob[row * p.k + i] = u.m == u.m ? -INFINITY : nan;
  }
}

template <typename T, int PARTS> int launch_parts(const ScoreArgs &p, int64_t T_, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PARTS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(T_ * PARTS));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = PARTS > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, score_kernel<T, PARTS>, p);
  return check_launch("token_logprobs");
}

template <typename T> int launch_score(const ScoreArgs &p, int64_t T_, cudaStream_t st) {
  // a row's CTAs: as many as leave every SM its 4 blocks and a CTA at least 2048 elements
  const int64_t slots = int64_t(num_sms()) * 4;
  int n = 1;
  while (n < kMaxParts && T_ * n < slots && p.V / (2 * n) >= 2048) n *= 2;
  if (n == 1) return launch_parts<T, 1>(p, T_, st);
  if (n == 2) return launch_parts<T, 2>(p, T_, st);
  if (n == 4) return launch_parts<T, 4>(p, T_, st);
  return launch_parts<T, 8>(p, T_, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_token_logprobs(const void *logits, int64_t stride, int dtype, int64_t T, int64_t V, float scale,
                                  const int32_t *ids, int64_t n_ids, float *logprob, float *entropy, float *lse, int k,
                                  int32_t *top_ids, float *top_logprob, moe_stream_t stream) {
  MOE_REQUIRE(dtype == MOE_F16 || dtype == MOE_BF16 || dtype == MOE_F32, "bad dtype %d", dtype);
  MOE_REQUIRE(T >= 0 && T < (int64_t(1) << 27) && V >= 1 && V < (int64_t(1) << 30), "T or V out of range");
  MOE_REQUIRE(stride >= V || T <= 1, "rows overlap");
  MOE_REQUIRE(scale > 0.f && scale <= 3.402823466e38f / kLog2e, "scale must be positive and finite");
  MOE_REQUIRE(n_ids >= 0 && n_ids < (int64_t(1) << 30), "n_ids out of range");
  MOE_SUPPORT(k >= 0 && k <= kMaxK, "0 <= k <= %d (k=%d)", kMaxK, k);
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(logits && (reinterpret_cast<uintptr_t>(logits) & (dtype_size(dtype) - 1)) == 0,
              "logits must be non-null and start on an element");
  MOE_REQUIRE(n_ids == 0 || (ids && logprob), "ids without logprob");
  MOE_REQUIRE(k == 0 || (top_ids && top_logprob), "k without its outputs");
  MOE_REQUIRE(aligned16(ids) && aligned16(logprob) && aligned16(entropy) && aligned16(lse) && aligned16(top_ids) &&
                  aligned16(top_logprob),
              "pointers must be 16-byte aligned");
  ScoreArgs p{logits, stride, ids, logprob, entropy, lse, top_logprob, top_ids, scale, int(V), int(n_ids), k};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_F16 ? launch_score<__half>(p, T, st)
                          : (dtype == MOE_BF16 ? launch_score<__nv_bfloat16>(p, T, st) : launch_score<float>(p, T, st));
}
