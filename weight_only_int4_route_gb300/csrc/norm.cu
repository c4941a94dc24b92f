// Root-mean-square norm of rows with the residual's addition, and rows in 8 bits with a scale.
//
//   h = x + residual (fp32);  sum = RN(h);  r = 1 / sqrt(mean(h^2) + eps);  u = h w
//   y = RN(h r w);   q = rne(u * 127 / max|u|), scale = max|u| r / 127
//
// The factor r of a row is positive and common to it, so the 8-bit codes follow from u alone: the sum of squares and
// the largest magnitude come out of one pass over the row, with one exchange between its warps.  A row stays in its
// threads' registers between the loads and the stores, so memory sees every element once: the kernel is bound by it
// (2 + 2 + 2 + 1 bytes an element for 16-bit rows with a residual and 8-bit output).  Measured on GB300: 8192 rows of 4096 in
// bf16, residual and 8-bit output, 40.1 us, 5.9 TB/s; 2501 rows of 2048 in f16, residual and 16-bit output, 6.9 us, 6.0 TB/s.
// Blocks that walk over rows with the next one's loads in flight were slower (82 us at the time of 67): registers, not
// loads, bounded the warps in flight.
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
  int vector_lanes;     // those that a row of this size has where it is read 16 bytes at a time
};

constexpr int kMaxD = 16384;
constexpr int kVectors = 4;   // 16-byte vectors of a thread

// V elements of a row: 16 bytes, or one.  Words, not arrays of elements: those cost a permute for every element that is read
// or put in (8192 rows of 4096 with residual and 8-bit output 60 us, 40 with words).
template <typename T, int V> struct Pack {
  uint32_t w[4];
  __device__ __forceinline__ void load(const T *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ void widen(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 two = __half22float2(u32_as_h2(w[i]));
        f[2 * i] = two.x, f[2 * i + 1] = two.y;
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void narrow(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else if constexpr (std::is_same<T, __half>::value) w[i] = h2_as_u32(__floats2half2_rn(f[2 * i], f[2 * i + 1]));
      else w[i] = h2_as_u32(__floats2bfloat162_rn(f[2 * i], f[2 * i + 1]));
    }
  }
  // the lowest bytes of the words
  static __device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&c)[V]) {
    uint32_t o[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      o[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(o[0], o[1]);
    else *reinterpret_cast<uint32_t *>(p) = o[0];
  }
};
template <typename T> struct Pack<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T *p) { w = *p; }
  __device__ __forceinline__ void store(T *p) const { *p = w; }
  __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = to_f32(w); }
  __device__ __forceinline__ void narrow(const float (&f)[1]) { w = from_f32<T>(f[0]); }
  static __device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&c)[1]) { *p = int8_t(c[0]); }
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Row-wide sum and maximum (NaN if one is), in an order that depends on the row's size alone.  A row of 32 threads is a
// warp's; a longer one is the block's, whose `turn`s use two places in turn, so that one barrier is enough.
struct Exchange {
  float sum[2][32], top[2][32];
};
__device__ __forceinline__ void row_reduce(float &ss, float &top, int lanes, Exchange &x, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (lanes == 32) return;
  const int warp = threadIdx.x >> 5, n = lanes >> 5;
  if ((threadIdx.x & 31) == 0) {
    x.sum[turn][warp] = ss;
    x.top[turn][warp] = top;
  }
  __syncthreads();
  ss = 0.f;
  top = 0.f;
  for (int i = 0; i < n; ++i) {
    ss += x.sum[turn][i];
    top = max_nan(top, x.top[turn][i]);
  }
  turn ^= 1;
}

// A row per `lanes` threads, NV vectors of V elements a thread; Q8: with 8-bit output.
// SV (with V = 1): rows that could be read 16 bytes, SV elements, at a time if they lay otherwise.  Their squares are added up in the
// order that they have there (from shared memory, in fp32), so a row's result does not depend on where it lies.  In bf16 with
// residual and 8-bit output: 8192 rows of 4096 at odd starts 117 us (16-byte starts 40), 5000 rows of 256 6.2 us (an
// order of their own 5.8).
template <typename T, int V, int NV, int MOST, bool Q8, int SV>
__global__ void __launch_bounds__(MOST) norm_kernel(const NormArgs p) {
  pdl_enter();
  __shared__ Exchange exchange;
  extern __shared__ __align__(16) float s_h[];
  using P = Pack<T, V>;
  const int rows = blockDim.x / p.lanes, t = int(threadIdx.x) % p.lanes;
  const int64_t row = int64_t(blockIdx.x) * rows + int(threadIdx.x) / p.lanes;
  if (row >= p.T) return;   // whole warps: no barrier is shared by several rows
  auto at = [&](int i) { return (t + i * p.lanes) * V; };
  const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
  P a[NV], b[NV], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {   // what is not there is 0, a weight 1
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 0.f;
    a[i].narrow(f);
    b[i].narrow(f);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 1.f;
    w[i].narrow(f);
    if (at(i) < p.d) a[i].load(x + at(i));
  }
  if (p.residual) {
    const T *y = static_cast<const T *>(p.residual) + row * p.residual_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at(i) < p.d) b[i].load(y + at(i));
  }
  if (p.weight) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at(i) < p.d) w[i].load(static_cast<const T *>(p.weight) + at(i));
  }
  float h[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[V];
    a[i].widen(h[i]);
    b[i].widen(f);
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] += f[j];
  }
  if (p.sum) {   // may be the residual or x itself: this thread's elements of both have been read
    T *s = static_cast<T *>(p.sum) + row * p.sum_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      P o;
      o.narrow(h[i]);
      if (at(i) < p.d) o.store(s + at(i));
    }
  }
  int turn = 0;
  float ss, top, eps = p.eps, r = 1.f;
  auto reduce = [&]() {   // elements that are not there are 0
    ss = top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      if (Q8) w[i].widen(f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (SV == 0) ss = fmaf(h[i][j], h[i][j], ss);
        if (Q8) top = max_nan(top, fabsf(h[i][j] * f[j]));
      }
    }
    if (SV > 0 && p.norm) {
      float *s = s_h + int(threadIdx.x) / p.lanes * p.d;
      __syncwarp();   // a second sum: the first one's values have been read (by other warps before row_reduce's barrier)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (at(i) < p.d) s[at(i)] = h[i][0];
      if (p.lanes == 32) __syncwarp();
      else __syncthreads();
      if (t < p.vector_lanes) {
        for (int k = t * SV; k < p.d; k += p.vector_lanes * SV) {
#pragma unroll
          for (int j = 0; j < SV; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(s + k + j);
            ss = fmaf(v.x, v.x, ss);
            ss = fmaf(v.y, v.y, ss);
            ss = fmaf(v.z, v.z, ss);
            ss = fmaf(v.w, v.w, ss);
          }
        }
      }
    }
    row_reduce(ss, top, p.lanes, exchange, turn);
  };
  reduce();
  if (p.norm) {
    // squares past fp32's range (magnitudes above 1.8e19), or below it with an eps that does not cover them: the row again, a power
    // of two times as large.  2^-72: 16384 squares of at most (2^128 2^-72)^2 are within range.  2^96: the
    // smallest subnormal number's square becomes 2^-106; these rows' elements are below 2^-41.
    const float by = isinf(ss) ? 0x1p-72f : (fmaf(ss, p.inv_d, eps) < 0x1p-96f ? 0x1p96f : 1.f);
    if (by != 1.f) {
      eps = eps * by * by;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] *= by;
      reduce();
    }
    r = rsqrtf(fmaf(ss, p.inv_d, eps));
  }
  if (p.y) {
    T *y = static_cast<T *>(p.y) + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      w[i].widen(f);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] *= h[i][j] * r;
      P o;
      o.narrow(f);
      if (at(i) < p.d) o.store(y + at(i));
    }
  }
  if (Q8) {
    const bool fine = top <= 3.402823466e38f;   // neither infinite nor NaN
    const float largest = top;
    float step = 0.f;
    const bool small = top < 0x1p-60f;
    if (small) {   // 127 / top overflows below 2^-121, products with the weight lose bits or all below 2^-126: the row is brought up first
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] *= 0x1p60f;
      reduce();
    }
    if (top > 0.f && fine) step = __fdiv_rn(127.f, top);
    int8_t *q = p.q + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[V];
      w[i].widen(f);
      uint32_t c[V];
      // adding 1.5 * 2^23 rounds to whole numbers, ties to even, and leaves their low 8 bits in the lowest byte
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = fine ? __float_as_uint(__fadd_rn(__fmul_rn(h[i][j] * f[j], step), 12582912.f)) : 0;
      if (at(i) < p.d) P::store_codes(q + at(i), c);
    }
    if (t == 0) {
      float scale = __fdiv_rn(largest, 127.f) * r;
      if (small && p.norm) scale = __fdiv_rn(top * r, 127.f) * 0x1p-60f;   // one rounding where the scale is subnormal
      p.scale[row] = !fine ? __int_as_float(0x7fc00000) : (top > 0.f ? scale : 0.f);
    }
  }
}

template <typename T, int V, int SV> int launch_rows(NormArgs p, cudaStream_t st) {
  const int vecs = (p.d + V - 1) / V;
  auto go = [&](auto nv, auto most) {
    constexpr int NV = decltype(nv)::value, MOST = decltype(most)::value;
    p.lanes = int(cdiv(cdiv(vecs, NV), 32) * 32);
    const int rows = p.lanes == 32 ? 4 : 1;
    auto kernel = p.q ? norm_kernel<T, V, NV, MOST, true, SV> : norm_kernel<T, V, NV, MOST, false, SV>;
    size_t smem = 0;
    if constexpr (SV > 0) {
      p.vector_lanes = int(cdiv(cdiv(p.d / SV, kVectors), 32) * 32);
      smem = size_t(rows) * p.d * sizeof(float);
      if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxD * sizeof(float))) != cudaSuccess)
        return check_launch("rmsnorm attribute");
    }
    launch_pdl(kernel, dim3(unsigned(cdiv(p.T, rows))), dim3(unsigned(rows * p.lanes)), smem, st, p);
    return check_launch("rmsnorm");
  };
  using std::integral_constant;
  if constexpr (V == 1) {   // rows that do not start on 16 bytes
    if (vecs <= 512 * 8) return go(integral_constant<int, 8>{}, integral_constant<int, 512>{});
    return go(integral_constant<int, 16>{}, integral_constant<int, 1024>{});
  } else {
    // 32 elements a thread (fp32: 16) whatever the number of rows: a row's sum has one order, its result is the same in every
    // batch.  8192 rows of 4096: 8, 16 and 32 elements a thread 70, 43 and 40 us; 8 rows 2.4 us with
    // 8 and 2.7 with 32.
    using Vectors = integral_constant<int, kVectors>;
    if (vecs <= 512 * kVectors) return go(Vectors{}, integral_constant<int, 512>{});
    if constexpr (V == 4) return go(Vectors{}, integral_constant<int, 1024>{});
    return set_error(MOE_ERR_UNSUPPORTED, "rows of at most %d elements", kMaxD);
  }
}

template <typename T> int launch_norm(const NormArgs &p, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(T));
  auto whole = [&](const void *q, int64_t stride) { return q == nullptr || (aligned16(q) && (stride % V == 0 || p.T == 1)); };
  if (p.d % V != 0) return launch_rows<T, 1, 0>(p, st);
  if (whole(p.x, p.x_stride) && whole(p.residual, p.residual_stride) && whole(p.sum, p.sum_stride)) return launch_rows<T, V, 0>(p, st);
  return launch_rows<T, 1, V>(p, st);
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
             int(d), 0, 1, 0};
  return run_norm(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_quantize_rows(const void *x, int64_t x_stride, int dtype, int64_t T, int64_t d, int8_t *q, float *q_scale,
                                 moe_stream_t stream) {
  MOE_TRY(check_rows(dtype, T, d));
  MOE_REQUIRE(x_stride >= d || T <= 1, "rows overlap");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(x && on_element(x, dtype) && q && q_scale, "null or misaligned pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(q_scale), "pointers must be 16-byte aligned");
  NormArgs p{x, nullptr, nullptr, x_stride, 0, 0, T, nullptr, nullptr, q, q_scale, 0.f, 0.f, int(d), 0, 0, 0};
  return run_norm(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
