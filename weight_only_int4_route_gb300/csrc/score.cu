// Log probabilities of given tokens, entropy and top alternatives of rows of logits.
//
// With z_j = scale * x_j:  lse = ln sum_j exp z_j,  logprob_t = z_t - lse,  entropy = lse - sum_j p_j z_j.
// One pass over the row: every thread keeps a reference M, Z = sum 2^t and S = sum 2^t t, t = (x - M) c, c = scale log2(e).  M
// starts as the largest logit of the warp's first loads and follows only what is above it by more than 2^6 in weight (Z' = Z f,
// S' = f (S + d Z), f = 2^d, d = (M - M') c): a reference that followed every new largest logit would move in some
// lane of a warp at nearly every step.  entropy = ln Z - ln 2 S / Z, and with M within 2^6 of the row's largest no digits cancel
// but those that a factor of 64 is worth (ln 64 = 4.2 beside an entropy of up to ln V).
// An element costs a conversion, half a maximum and half a clamp (in pairs, in its own type), a 2^x and three fp32 operations:
// the exponent is x c - fl(M c), and what the rounding of M c put in is taken out of the sums at the end.
//
// Top alternatives, in the order of (logit descending, id ascending): a thread knows its largest logit.  A value `from` is
// found, by halving intervals, that at least k threads and few more reach with theirs: the k best are at or above it, and only
// these threads hold any such.  Their elements are read again (from the L2, a few per cent of the row), what passes is
// collected, and an element's place is the number of elements before it.  Where more pass than fit, the k best are found one
// after the other.
//
// Few long rows are shared by the CTAs of a cluster, which send their sums and their k best to the first one.
// Bound by the instructions of a row's elements beside memory for many rows, by the length of this chain for a few.  Measured on
// GB300 (k = 8 or 5): 4096 rows of 65521 in bf16 104 us, 5.2 TB/s (without alternatives 90 us; 6 waves of rows where 5.4 would
// do); 320 rows of 131072 23.5 us; one row of 32000 in fp32 5.8 us, of which the alternatives are 2.
#include <type_traits>

#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kResident = 5;        // blocks of an SM (51 registers a thread; with 4 many rows took 4 % longer, 320 rows 20 %)
constexpr int kMaxK = 64;
constexpr int kCand = 1024;         // elements collected at most
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

// Order of elements as one unsigned number: logits descending, then ids ascending; 0 is before no element.  -0 and 0 are equal.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t b) { return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b); }
__device__ __forceinline__ uint64_t key_of(float x, uint32_t id) { return uint64_t(ordered(x)) << 32 | uint32_t(~id); }
__device__ __forceinline__ float key_value(uint64_t key) { return value_of(uint32_t(key >> 32)); }
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

// What masked elements count as: far below any logit that matters, and times log2(e) still finite.
__device__ __forceinline__ float lowest(__half) { return -65504.f; }
__device__ __forceinline__ float lowest(__nv_bfloat16) { return -0x1p120f; }
__device__ __forceinline__ float lowest(float) { return -0x1p120f; }

// Sixteen bytes of a row: its elements in fp32 and their largest (NaN if one is).  CLAMP: elements below lowest(T) come as
// lowest(T): 0 times -inf would be NaN where a weight of 0 is meant.
template <bool CLAMP = false> __device__ __forceinline__ float open(const uint4 &r, float (&e)[8], __half) {
  uint32_t w[4] = {r.x, r.y, r.z, r.w}, t0, t1;
  asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(t0) : "r"(w[0]), "r"(w[1]));
  asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(t1) : "r"(w[2]), "r"(w[3]));
  asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(t0) : "r"(t0), "r"(t1));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (CLAMP) asm("max.NaN.f16x2 %0, %0, %1;\n" : "+r"(w[i]) : "r"(0xfbfffbffu));
    const float2 v = __half22float2(u32_as_h2(w[i]));
    e[2 * i] = v.x;
    e[2 * i + 1] = v.y;
  }
  const float2 t = __half22float2(u32_as_h2(t0));
  return max_nan(t.x, t.y);
}
template <bool CLAMP = false> __device__ __forceinline__ float open(const uint4 &r, float (&e)[8], __nv_bfloat16) {
  uint32_t w[4] = {r.x, r.y, r.z, r.w}, t0, t1;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(t0) : "r"(w[0]), "r"(w[1]));
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(t1) : "r"(w[2]), "r"(w[3]));
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(t0) : "r"(t0), "r"(t1));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (CLAMP) asm("max.NaN.bf16x2 %0, %0, %1;\n" : "+r"(w[i]) : "r"(0xfb80fb80u));
    e[2 * i] = __uint_as_float(w[i] << 16);
    e[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return max_nan(__uint_as_float(t0 << 16), __uint_as_float(t0 & 0xffff0000u));
}
template <bool CLAMP = false> __device__ __forceinline__ float open(const uint4 &r, float (&e)[4], float) {
  e[0] = __uint_as_float(r.x);
  e[1] = __uint_as_float(r.y);
  e[2] = __uint_as_float(r.z);
  e[3] = __uint_as_float(r.w);
  const float top = max_nan(max_nan(e[0], e[1]), max_nan(e[2], e[3]));
  if (CLAMP) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = fmaxf(e[j], -0x1p120f);
  }
  return top;
}

// Sums of a set of elements: largest logit m (NaN if any element is), reference M, Z and S.  S is in units of the exponent: in
// units of x it would pass fp32's range under small scales.
struct alignas(16) Sums {
  float m, M, z, s;
};
// (x - M) c.  x - M alone may pass fp32's range, the difference of their halves does not.
__device__ __forceinline__ float exponent(float x, float M, float c) { return __fmul_rn(fmaf(-0.5f, M, 0.5f * x), c) * 2.f; }
// z and s moved to reference M.  Nothing is left where the factor is 0 (0 times an infinite difference would be NaN) or where
// nothing was (z = 0, whose reference does not count).
__device__ __forceinline__ void move_to(float M, float c, const Sums &o, float &z, float &s) {
  const float d = exponent(o.M, M, c), f = ex2(d);
  const bool any = f != 0.f && o.z != 0.f;
  z = any ? o.z * f : 0.f;
  s = any ? f * fmaf(d, o.z, o.s) : 0.f;
}
// The sums of n parts, in their order.
template <typename At> __device__ __forceinline__ Sums join(int n, float c, At at) {
  Sums u = {-INFINITY, -INFINITY, 0.f, 0.f};
  for (int i = 0; i < n; ++i) {
    const Sums o = at(i);
    u.m = max_nan(u.m, o.m);
    if (o.z != 0.f) u.M = fmaxf(u.M, o.M);
  }
  for (int i = 0; i < n; ++i) {
    float z, s;
    move_to(u.M, c, at(i), z, s);
    u.z += z;
    u.s += s;
  }
  return u;
}

// What a CTA of a cluster sends to the first one.
struct Part {
  uint64_t best[kMaxK];
  Sums sums;
};

template <typename T, int PARTS>
__global__ void __launch_bounds__(kThreads, kResident) score_kernel(const ScoreArgs p) {
  pdl_enter();
  constexpr int VE = 16 / int(sizeof(T));
  __shared__ Part parts[PARTS];
  __shared__ uint64_t cand[kCand];
  __shared__ uint32_t s_key[kThreads];
  __shared__ uint64_t s_best[kWarps];
  __shared__ Sums s_sums[kWarps];
  __shared__ uint8_t s_lane[kWarps][32];
  __shared__ int s_n;
  __shared__ uint32_t s_from;
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
  const uint4 *vec = reinterpret_cast<const uint4 *>(x + head);
  const bool has_head = part == 0 && tid < head, has_tail = part == 0 && tid < tail;
  const int tail_id = head + nv * VE + tid;

  const bool any = has_head || has_tail || v0 + tid < v1;
  float m = -INFINITY, M = 0.f, Mc = 0.f, limit = -INFINITY;   // Mc = fl(M c)
  const float slack = 6.f / c;
  float z = 0.f, zs = 0.f;   // sums of 2^t and 2^t t, t = x c - Mc
  auto follow = [&](float top) {
    const float to = __fmul_rn(top, c), d = Mc - to, f = ex2(d);
    const bool none = limit == -INFINITY || f == 0.f;   // no element yet, or 0 times an infinite d
    zs = none ? 0.f : f * fmaf(d, z, zs);
    z = none ? 0.f : f * z;
    M = top;
    Mc = to;
    limit = top + slack;
  };
  auto add = [&](float e) {
    const float t = fmaf(e, c, -Mc), w = ex2(t);
    z += w;
    zs = fmaf(w, t, zs);
  };
  auto one = [&](int id) {
    const float e = to_f32(x[id]);
    m = max_nan(m, e);
    if (!(e <= limit)) follow(e);
    add(fmaxf(e, lowest(T())));
  };
  // the first given token's logit on its way
  const int64_t asked = row * p.n_ids + tid;
  const int id = tid < p.n_ids && part == 0 ? p.ids[asked] : -1;
  const float logit = id >= 0 && id < p.V ? to_f32(x[id]) : 0.f;
  constexpr int kBatch = 4, kStep = kBatch * kThreads;   // loads in flight
  auto batch = [&](int from, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    const int v = from + tid;
    uint4 r[kBatch];
    float e[kBatch][VE], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (kWhole || v + i * kThreads < v1) r[i] = vec[v + i * kThreads];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (kWhole || v + i * kThreads < v1) top = max_nan(top, open<true>(r[i], e[i], T()));
    m = max_nan(m, top);
    if (from == v0) {   // the first reference: the largest of the warp's first loads
      const float high = value_of(__reduce_max_sync(0xffffffffu, ordered(top)));
      if (fabsf(high) < INFINITY) follow(high);
    }
    if (!(top <= limit)) follow(top);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (kWhole || v + i * kThreads < v1) {
#pragma unroll
        for (int j = 0; j < VE; ++j) add(e[i][j]);
      }
  };
  int from = v0;
  for (; from + kStep <= v1; from += kStep) batch(from, std::true_type{});
  if (from < v1) batch(from, std::false_type{});
  if (has_head) one(tid);
  if (has_tail) one(tail_id);
  // t was short of (x - M) c by Mc - M c, the product's rounding
  const float off = fmaf(M, c, -Mc), g = ex2(-off);
  z *= g;
  zs = fmaf(zs, g, -off * z);
  if (m == -INFINITY) z = zs = 0.f;
  // Masked elements may have had weight (largest logits near the type's lowest, small scales), products been infinite, or the rounding
  // of M c been past the half unit that |M c| < 2^24 means (from 2^31 on t overflows): again, with differences that are
  // clamped.  A thread whose largest is nothing beside its warp's has nothing to add: a row masked by a large finite value is
  // read once more only where a warp sees nothing else (2048 rows of 32000 in bf16, one token in 20 not masked 36.7 us, one in
  // 2000 45; deciding by the CTA's largest costs registers: 4096 rows of 65521 104 us and 112).  M c again and not Mc: that
  // would be one register more in the loop (107 us).
  const bool poor = fabsf(m) < INFINITY && !((lowest(T()) - M) * c < -200.f && fabsf(__fmul_rn(M, c)) < 0x1p24f && c > 0x1p-40f && c < 64.f);
  const float most = value_of(__reduce_max_sync(0xffffffffu, ordered(m)));   // the warp's (see below for NaN)
  if (poor) {
    z = zs = 0.f;
    M = m;
    const bool nothing = exponent(m, most, c) < -200.f;
    auto again = [&](float e) {
      const float t = fmaxf(exponent(e, M, c), -1000.f), w = ex2(t);   // -inf: a weight of 0 under any scale
      z += w;
      zs = fmaf(w, t, zs);
    };
    for (int v = nothing ? v1 : v0 + tid; v < v1; v += kThreads) {
      float e[VE];
      open(vec[v], e, T());
      for (int j = 0; j < VE; ++j) again(e[j]);
    }
    if (has_head && !nothing) again(to_f32(x[tid]));
    if (has_tail && !nothing) again(to_f32(x[tail_id]));
  }
  // ---- the CTA's sums
  const uint32_t key = any ? ordered(m) : 0;   // 0: below every logit
  Sums u;
  {
    const uint32_t high = __reduce_max_sync(0xffffffffu, z != 0.f ? ordered(M) : 0u);
    u.M = high ? value_of(high) : 0.f;
    move_to(u.M, c, Sums{m, M, z, zs}, u.z, u.s);
    u.m = __any_sync(0xffffffffu, m != m) ? __int_as_float(0x7fc00000) : most;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      u.z += __shfl_xor_sync(0xffffffffu, u.z, o);
      u.s += __shfl_xor_sync(0xffffffffu, u.s, o);
    }
  }
  if (lane == 0) s_sums[warp] = u;
  if (p.k > 0) s_key[tid] = key;
  if (tid == 0) s_n = 0;
  if (tid < p.k) parts[part].best[tid] = 0;
  __syncthreads();
  u = join(kWarps, c, [&](int w) { return s_sums[w]; });

  // ---- the CTA's k best (a row that holds a NaN has none)
  if (p.k > 0 && u.m == u.m) {
    // the largest value (as an ordered number) that at least k threads reach, or one near it
    if (warp == 0) {
      uint32_t mine[kWarps], low = ~0u, high = ordered(u.m);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mine[w] = s_key[w * 32 + lane];
        low = min(low, mine[w]);
      }
      low = __reduce_min_sync(0xffffffffu, low);   // every thread reaches it
      while (low < high) {
        const uint32_t mid = low + (high - low + 1) / 2;
        int n = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) n += mine[w] >= mid;
        n = __reduce_add_sync(0xffffffffu, n);
        if (n >= p.k) {
          low = mid;
          if (n <= p.k + p.k / 4) break;
        } else {
          high = mid - 1;
        }
      }
      if (lane == 0) s_from = low;
    }
    __syncthreads();
    const uint32_t from = s_from;
    const float least = value_of(from);   // -0 counts as 0; from = 0 is NaN, below which nothing is
    auto offer = [&](float e, int id) {
      const int place = atomicAdd(&s_n, 1);
      if (place < kCand) cand[place] = key_of(e, uint32_t(id));
    };
    const unsigned who = __ballot_sync(0xffffffffu, key != 0 && key >= from);
    if (who >> lane & 1) s_lane[warp][__popc(who & ((1u << lane) - 1))] = uint8_t(lane);
    __syncwarp();
    const int each = (v1 - v0 + kThreads - 1) / kThreads, total = __popc(who) * each;
    // the elements of these threads that `pass`
    auto collect = [&](auto pass) {
      if (has_head && pass(to_f32(x[tid]))) offer(to_f32(x[tid]), tid);
      if (has_tail && pass(to_f32(x[tail_id]))) offer(to_f32(x[tail_id]), tail_id);
      for (int i = lane; i < total; i += 32) {
        const int n = i / each, v = v0 + warp * 32 + s_lane[warp][n] + (i - n * each) * kThreads;
        if (v >= v1) continue;
        float e[VE];
        if (!pass(open(vec[v], e, T()))) continue;
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (pass(e[j])) offer(e[j], head + v * VE + j);
      }
    };
    collect([&](float e) { return !(e < least); });
    __syncthreads();
    if (s_n > kCand) {
      // Many equal to `least` (masked rows with fewer than k others, rows of few values): those above it, then of the equal
      // ones the first that are needed, in the order of their ids.
      __syncthreads();
      if (tid == 0) s_n = 0;
      __syncthreads();
      collect([&](float e) { return e > least; });
      __syncthreads();
      int found = s_n;
      __syncthreads();
      if (found > kCand - 32 * VE - 2 * VE) {
        if (tid == 0) s_n = kCand + 1;
      } else if (warp == 0) {
        auto count = [&] {   // after the lanes' offers
          __syncwarp();
          found = *reinterpret_cast<volatile int *>(&s_n);
          __syncwarp();
        };
        if (has_head && to_f32(x[tid]) == least) offer(least, tid);
        count();
        for (int v = v0; v < v1 && found < p.k; v += 32) {
          float e[VE];
          if (v + lane < v1 && open(vec[v + lane], e, T()) >= least) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
              if (e[j] == least) offer(e[j], head + (v + lane) * VE + j);
          }
          count();
        }
        if (found < p.k && has_tail && to_f32(x[tail_id]) == least) offer(least, tail_id);
      }
      __syncthreads();
    }
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
          float e[VE];
          open(vec[v], e, T());
#pragma unroll
          for (int j = 0; j < VE; ++j) look(e[j], head + v * VE + j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine = max(mine, shfl_xor64(mine, o));
        __syncthreads();
        if (lane == 0) s_best[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mine = max(mine, s_best[w]);
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
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + 4), "f"(u.M) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + 8), "f"(u.z) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + 12), "f"(u.s) : "memory");
      }
    }
    __syncwarp();
    cluster_sync();
    if (part != 0) return;
    if (tid == 0) parts[0].sums = u;
    __syncthreads();
    u = join(PARTS, c, [&](int w) { return parts[w].sums; });
  } else {
    __syncthreads();
  }

  const float nan = __int_as_float(0x7fc00000), lz = logf(u.z);
  auto logprob = [&](float e) {
    if (u.m != u.m) return nan;
    if (u.m == -INFINITY) return -INFINITY;
    if (u.m == INFINITY) return e == INFINITY ? nan : -INFINITY;
    const float d = e - u.M;
    const float v = isinf(d) && !isinf(e) ? fmaf(__fmul_rn(0.5f * e - 0.5f * u.M, p.scale), 2.f, -lz)   // further apart than fp32 reaches
                                          : fmaf(d, p.scale, -lz);
    return v > 0.f ? 0.f : v;   // by rounding alone
  };
  if (tid < p.n_ids) p.logprob[asked] = id >= 0 && id < p.V ? logprob(logit) : nan;
  for (int i = tid + kThreads; i < p.n_ids; i += kThreads) {
    const int j = p.ids[row * p.n_ids + i];
    p.logprob[row * p.n_ids + i] = j >= 0 && j < p.V ? logprob(to_f32(x[j])) : nan;
  }
  if (tid == 0) {
    const bool finite = fabsf(u.m) < INFINITY;
    if (p.lse) p.lse[row] = finite ? fmaf(u.M, p.scale, lz) : u.m;
    const float h = fmaf(-kLn2, u.s / u.z, lz);
    if (p.entropy) p.entropy[row] = finite ? (h < 0.f ? 0.f : h) : (u.m == -INFINITY ? 0.f : nan);
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
  // A row's CTAs: as many as still run all at once, with at least 4096 elements each.  Rows of 131072 in bf16, 1, 2, 4 and 8 CTAs:
  // 1 row 12.7, 9.3, 7.5, 6.9 us; 64 rows 14.4, 11.3, 11.4, 11.9; 150 rows 20.9, 18.4, 16.0, 21.2; 320 rows 29.0, 23.5, 28.2,
  // 37.1; 600 rows 36.2, 40.9, 47.8, 62.8; one row of 32000 in fp32 7.2, 6.5, 5.8, 6.2.
  const int64_t slots = int64_t(num_sms()) * kResident;
  int n = 1;
  while (n < kMaxParts && T_ * 2 * n <= slots && p.V / (2 * n) >= 4096) n *= 2;
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
