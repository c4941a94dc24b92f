// Root-mean-square norm of rows with the residual's addition, and rows in 8 bits with a scale.
//
//   h = x + residual (fp32);  sum = RN(h);  r = 1 / sqrt(mean(h^2) + eps);  u = h w
//   y = RN(h r w);   q = rne(u * 127 / max|u|), scale = max|u| r / 127
//
// The factor r of a row is positive and common to it, so the 8-bit codes follow from u alone: the sum of squares and
// the largest magnitude come out of one pass over the row, with one exchange between its warps.  A row stays in its
// threads' registers between the loads and the stores, so memory sees every element once: the kernel is bound by it
// (2 + 2 + 2 + 1 bytes an element for 16-bit rows with a residual and 8-bit output).
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride, sum_stride, T;
  void *sum, *y;
  int8_t *q;
  float *scale;
  float eps, inv_d;
  int d, lanes, norm;   // lanes: threads of a row (a multiple of 32)
};

constexpr int kMaxD = 16384;

template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
  T v[V];
};
template <int V> struct alignas(V) Codes {
  int8_t v[V];
};

// Row-wide sum and maximum (as the bits of a non-negative float, so that NaN and infinity are the largest).  Every thread
// of the block takes part; the order of the additions is fixed.
__device__ __forceinline__ void row_reduce(float &ss, uint32_t &top, int lanes, float (*s_sum)[32], uint32_t (*s_top)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (lanes == 32) return;
  const int warp = threadIdx.x >> 5, n = lanes >> 5, first = warp / n * n;
  __syncthreads();   // the exchange before this one has been read
  if ((threadIdx.x & 31) == 0) {
    (*s_sum)[warp] = ss;
    (*s_top)[warp] = top;
  }
  __syncthreads();
  ss = 0.f;
  top = 0;
  for (int i = 0; i < n; ++i) {
    ss += (*s_sum)[first + i];
    top = max(top, (*s_top)[first + i]);
  }
}

// Most threads of a block: what the registers of a thread's elements allow without spills.
constexpr int most_threads(int V, int NV) { return V > 1 ? 1024 : (NV <= 8 ? 768 : 512); }

// A row per `lanes` threads, NV vectors of V elements a thread; short rows share a block.  The weight is read again from
// the L1 for the stores rather than kept in registers.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(most_threads(V, NV)) norm_kernel(const NormArgs p) {
  pdl_enter();
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  using P = Pack<T, V>;
  const int rows = blockDim.x / p.lanes, in = threadIdx.x / p.lanes, t = threadIdx.x - in * p.lanes;
  const int64_t row = int64_t(blockIdx.x) * rows + in;
  const int d = row < p.T ? p.d : 0;   // a row that is not there has no elements
  const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
  const T *residual = static_cast<const T *>(p.residual);
  const T *weight = static_cast<const T *>(p.weight);
  auto weight_of = [&](int at, int j) { return weight ? to_f32(weight[at + j]) : 1.f; };
  float h[NV][V];
  P a[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (t + i * p.lanes) * V;
    if (at < d) a[i] = *reinterpret_cast<const P *>(x + at);
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] = 0.f;
  }
  if (residual) {
    residual += row * p.residual_stride;
    P b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (t + i * p.lanes) * V;
      if (at < d) b[i] = *reinterpret_cast<const P *>(residual + at);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((t + i * p.lanes) * V < d) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = to_f32(a[i].v[j]) + to_f32(b[i].v[j]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((t + i * p.lanes) * V < d) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = to_f32(a[i].v[j]);
      }
  }
  if (p.sum) {   // may be the residual or x itself: this thread's elements of both have been read
    T *s = static_cast<T *>(p.sum) + row * p.sum_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (t + i * p.lanes) * V;
      if (at >= d) continue;
      P o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.v[j] = from_f32<T>(h[i][j]);
      *reinterpret_cast<P *>(s + at) = o;
    }
  }
  float ss, eps = p.eps, r = 1.f;
  uint32_t top;
  auto reduce = [&]() {
    ss = 0.f;
    top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (t + i * p.lanes) * V;
      if (at >= d) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ss = fmaf(h[i][j], h[i][j], ss);
        if (p.q) top = max(top, __float_as_uint(fabsf(h[i][j] * weight_of(at, j))));
      }
    }
    row_reduce(ss, top, p.lanes, &s_sum, &s_top);
  };
  reduce();
  if (p.norm) {
    // squares past fp32 (magnitudes above 1.8e19): the row again, 2^-64 times as large.  A block's rows go round together.
    if (__syncthreads_or(isinf(ss))) {
      if (isinf(ss)) {
        eps *= 0x1p-128f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) h[i][j] *= 0x1p-64f;
      }
      reduce();
    }
    r = rsqrtf(fmaf(ss, p.inv_d, eps));
  }
  if (p.y) {
    T *y = static_cast<T *>(p.y) + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (t + i * p.lanes) * V;
      if (at >= d) continue;
      P o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.v[j] = from_f32<T>(h[i][j] * r * weight_of(at, j));
      *reinterpret_cast<P *>(y + at) = o;
    }
  }
  if (p.q) {
    const float m = __uint_as_float(top);
    const bool fine = m <= 3.402823466e38f;   // neither infinite nor NaN
    // 127 / m overflows below 2^-121: small rows are brought up first (exact)
    const float up = m < 0x1p-60f ? 0x1p60f : 1.f;
    const float step = m > 0.f && fine ? __fdiv_rn(127.f, m * up) : 0.f;
    int8_t *q = p.q + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (t + i * p.lanes) * V;
      if (at >= d) continue;
      Codes<V> o;
#pragma unroll
      for (int j = 0; j < V; ++j)
        o.v[j] = fine ? int8_t(__float2int_rn(h[i][j] * weight_of(at, j) * up * step)) : int8_t(0);
      *reinterpret_cast<Codes<V> *>(q + at) = o;
    }
    if (t == 0 && d > 0) p.scale[row] = fine ? __fdiv_rn(m, 127.f) * r : __int_as_float(0x7fc00000);
  }
}

template <typename T, int V> int launch_rows(NormArgs p, cudaStream_t st) {
  const int vecs = (p.d + V - 1) / V;
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    p.lanes = int(cdiv(cdiv(vecs, NV), 32) * 32);
    // short rows share blocks of about 128 threads
    const int rows = p.lanes >= 128 ? 1 : 128 / p.lanes;
    launch_pdl(norm_kernel<T, V, NV>, dim3(unsigned(cdiv(p.T, rows))), dim3(unsigned(rows * p.lanes)), 0, st, p);
    return check_launch("rmsnorm");
  };
  // 8 elements a thread for few rows of few elements (more threads, less latency), 16 otherwise; single elements
  // (rows that do not start on 16 bytes) 8 or 32
  if constexpr (V == 1) {
    if (vecs <= 768 * 8) return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 32>{});
  } else {
    if (vecs <= 1024 * (8 / V) && p.T < num_sms()) return go(std::integral_constant<int, 8 / V>{});
    return go(std::integral_constant<int, 16 / V>{});
  }
}

template <typename T> int launch_norm(const NormArgs &p, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(T));
  auto whole = [](const void *q, int64_t stride) { return q == nullptr || (aligned16(q) && stride % V == 0); };
  if (p.d % V == 0 && whole(p.x, p.x_stride) && whole(p.residual, p.residual_stride) && whole(p.sum, p.sum_stride))
    return launch_rows<T, V>(p, st);
  return launch_rows<T, 1>(p, st);
}

int run_norm(const NormArgs &p, int dtype, cudaStream_t st) {
  return dtype == MOE_F16 ? launch_norm<__half>(p, st) : (dtype == MOE_BF16 ? launch_norm<__nv_bfloat16>(p, st) : launch_norm<float>(p, st));
}

bool on_element(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype_size(dtype) - 1)) == 0; }

int check_rows(int dtype, int64_t T, int64_t d) {
  MOE_REQUIRE(dtype == MOE_F16 || dtype == MOE_BF16 || dtype == MOE_F32, "bad dtype %d", dtype);
  MOE_REQUIRE(T >= 0 && T < (int64_t(1) << 31) && d >= 1, "T or d out of range");
  MOE_SUPPORT(d <= kMaxD, "rows of at most %d elements (d=%lld)", kMaxD, (long long)d);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_rmsnorm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, const void *weight,
                           int dtype, int64_t T, int64_t d, float eps, void *sum, int64_t sum_stride, void *y, int8_t *q,
                           float *q_scale, moe_stream_t stream) {
  MOE_TRY(check_rows(dtype, T, d));
  MOE_REQUIRE(eps >= 0.f && eps <= 3.402823466e38f, "eps must be finite and not negative");
  MOE_REQUIRE((x_stride >= d || T <= 1) && (residual == nullptr || residual_stride >= d || T <= 1) &&
                  (sum == nullptr || sum_stride >= d || T <= 1),
              "rows overlap");
  MOE_REQUIRE((q == nullptr) == (q_scale == nullptr), "q and q_scale come together");
  MOE_REQUIRE(y || q || sum || T == 0, "no output asked for");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(x && on_element(x, dtype) && on_element(residual, dtype) && on_element(sum, dtype),
              "x must be non-null; x, residual and sum start on an element");
  MOE_REQUIRE(aligned16(weight) && aligned16(y) && aligned16(q) && aligned16(q_scale), "pointers must be 16-byte aligned");
  MOE_REQUIRE(sum != x || sum_stride == x_stride || T == 1, "in place needs the same strides");
  MOE_REQUIRE(sum == nullptr || sum != residual || sum_stride == residual_stride || T == 1, "in place needs the same strides");
  NormArgs p{x, residual, weight, x_stride, residual_stride, sum_stride, T, sum, y, q, q_scale, eps, float(1.0 / double(d)),
             int(d), 0, 1};
  return run_norm(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_quantize_rows(const void *x, int64_t x_stride, int dtype, int64_t T, int64_t d, int8_t *q, float *q_scale,
                                 moe_stream_t stream) {
  MOE_TRY(check_rows(dtype, T, d));
  MOE_REQUIRE(x_stride >= d || T <= 1, "rows overlap");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(x && on_element(x, dtype) && q && q_scale, "null or misaligned pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(q_scale), "pointers must be 16-byte aligned");
  NormArgs p{x, nullptr, nullptr, x_stride, 0, 0, T, nullptr, nullptr, q, q_scale, 0.f, 0.f, int(d), 0, 0};
  return run_norm(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
