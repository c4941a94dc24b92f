// Rotary positions: the table of cosines and sines, and the rotation of heads by it.
//
// A pair (a, b) of a head turns by its position's angle: (a cos - b sin, a sin + b cos); turning back
// (sin -> -sin) is the gradient.  The angles are formed and reduced in 64 bits when the table is made:
// position times frequency reaches 10^5 radians, where a 32-bit product is off by 10^-2.
//
// Measured on GB300: 40001 tokens x 16 heads of 128 in fp32 97 us, 7.0 TB/s (the measured copy rate);
// 8192 x 32 heads of 128 in f16, half of the head, interleaved, from a strided input 24 us, 5.7 TB/s.
#include "kv_internal.cuh"

namespace moe {

MOE_DEFINE_CHECK_WORD(rope)

namespace {

constexpr int kThreads = 256;

// One thread per (position, frequency); fp64, run once per model.
__global__ void __launch_bounds__(kThreads) rope_table_kernel(int64_t n_pos, int rot, double base, int scaling,
                                                              double factor, double original,
                                                              float *__restrict__ cos_sin) {
  pdl_enter();
  const int half = rot / 2;
  const int64_t total = n_pos * half;
  for (int64_t q = int64_t(blockIdx.x) * kThreads + threadIdx.x; q < total; q += int64_t(gridDim.x) * kThreads) {
    const int64_t p = q / half;
    const int i = int(q - p * half);
    const double pi2 = 6.283185307179586;
    double b = base, scale = 1.0;
    if (scaling == MOE_ROPE_NTK) b = base * pow(factor, double(rot) / double(rot - 2));
    double f = pow(b, -2.0 * i / double(rot));
    if (scaling == MOE_ROPE_LINEAR) f /= factor;
    if (scaling == MOE_ROPE_PARTS) {
      const double turns = original * f / pi2;
      const double g = fmin(fmax((turns - 1.0) / 31.0, 0.0), 1.0);
      f *= g + (1.0 - g) / factor;
      scale = 0.1 * log(factor) + 1.0;
    }
    double s, c;
    sincos(double(p) * f, &s, &c);
    cos_sin[p * rot + i] = float(c * scale);
    cos_sin[p * rot + half + i] = float(s * scale);
  }
}

// A thread owns one unit (a 16-byte vector, or a pair of them) of kHeads heads of one token: the angles
// are read once for them, and their loads are in flight together.  Consecutive threads own consecutive
// vectors of a head.  Bound by memory: nothing is read twice but the table, and it stays in the caches.
template <typename T, int V, int MODE, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_kernel(const T *x, int64_t xt, int64_t xh,
                                                        const int32_t *__restrict__ pos,
                                                        const float *__restrict__ cos_sin, int64_t n_pos, int64_t T_,
                                                        int heads, int rot, int units, int turned, int inverse,
                                                        T *out, int64_t ot, int64_t oh) {
  pdl_enter();
  const unsigned groups = unsigned(heads + kHeads - 1) / kHeads, per = groups * unsigned(units);
  // blocks take whole tokens' worth of threads in order; a token's index needs 64 bits in no launch (T < 2^31)
  const int64_t q = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = (q >> 32) == 0 ? int64_t(unsigned(q) / per) : q / per;
  if (t >= T_) return;
  const unsigned in = unsigned(q - t * per), group = in / unsigned(units);
  const int unit = int(in - group * unsigned(units)), h0 = int(group) * kHeads;
  const int p = __ldg(pos + t);   // first: the angles wait for it
  const T *src = x + t * xt + h0 * xh;
  RopeUnit<T, V, MODE> u[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (h0 + i < heads) u[i].load(src + i * xh, unit, turned, rot);
  Angles<V, MODE> g;
  if (unit < turned)
    load_angles<V, MODE>(g, cos_sin, n_pos, p, rot, unit, inverse, [] {
      if (MOE_CHECKED) check_fail(kCheckPos);
    });
  T *dst = out + t * ot + h0 * oh;
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (h0 + i < heads) u[i].store(dst + i * oh, unit, turned, rot, g);
}

unsigned grid_for(int64_t work) {
  const int64_t blocks = cdiv(work, kThreads), most = int64_t(num_sms()) * 16;
  return unsigned(blocks < most ? (blocks > 0 ? blocks : 1) : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_rope_table(int64_t n_pos, int64_t rot, double base, int scaling, double factor, int64_t original,
                              float *cos_sin, moe_stream_t stream) {
  MOE_REQUIRE(n_pos >= 0 && n_pos < (int64_t(1) << 31), "n_pos out of range");
  MOE_REQUIRE(rot >= 2 && rot % 2 == 0 && rot <= 4096, "rot must be even, 2 <= rot <= 4096 (rot=%lld)", (long long)rot);
  MOE_REQUIRE(base > 1.0 && base < 1e300, "base must be above 1");
  MOE_REQUIRE(scaling >= MOE_ROPE_PLAIN && scaling <= MOE_ROPE_PARTS, "bad rope scaling %d", scaling);
  MOE_REQUIRE(scaling == MOE_ROPE_PLAIN || (factor >= 1.0 && factor < 1e9), "factor must be at least 1");
  MOE_REQUIRE(scaling != MOE_ROPE_NTK || rot > 2, "NTK scaling needs rot > 2");
  MOE_REQUIRE(scaling != MOE_ROPE_PARTS || original >= 1, "PARTS scaling needs the trained context length");
  if (n_pos == 0) return MOE_OK;
  MOE_REQUIRE(cos_sin && aligned16(cos_sin), "cos_sin must be non-null and 16-byte aligned");
  launch_pdl(rope_table_kernel, dim3(grid_for(n_pos * (rot / 2))), dim3(kThreads), 0,
             reinterpret_cast<cudaStream_t>(stream), n_pos, int(rot), base, scaling, factor, double(original), cos_sin);
  return check_launch("rope_table");
}

extern "C" int moe_rope(const void *x, int dtype, int64_t T, int64_t heads, int64_t head_dim, int64_t x_token_stride,
                        int64_t x_head_stride, const int32_t *pos, const float *cos_sin, int64_t n_pos, int64_t rot,
                        int interleaved, int inverse, void *out, int64_t out_token_stride, int64_t out_head_stride,
                        moe_stream_t stream) {
  MOE_REQUIRE(dtype == MOE_F16 || dtype == MOE_BF16 || dtype == MOE_F32, "bad dtype %d", dtype);
  MOE_REQUIRE(T >= 0 && T < (int64_t(1) << 31) && heads >= 1 && heads < (int64_t(1) << 20), "T or heads out of range");
  MOE_REQUIRE(head_dim >= 8 && head_dim % 8 == 0 && head_dim <= 4096, "head_dim must be a multiple of 8, at most 4096 (%lld)",
              (long long)head_dim);
  MOE_REQUIRE(rot >= 2 && rot % 2 == 0 && rot <= head_dim, "rot must be even, 2 <= rot <= head_dim (rot=%lld)", (long long)rot);
  MOE_REQUIRE(n_pos >= 1 && n_pos < (int64_t(1) << 31), "n_pos out of range");
  const int64_t unit = 16 / int64_t(dtype_size(dtype));
  MOE_REQUIRE(x_token_stride >= 0 && x_head_stride >= 0 && out_token_stride >= 0 && out_head_stride >= 0 &&
                  x_token_stride % unit == 0 && x_head_stride % unit == 0 && out_token_stride % unit == 0 &&
                  out_head_stride % unit == 0,
              "strides must be non-negative multiples of 16 bytes");
  MOE_REQUIRE((out_head_stride >= head_dim || heads == 1) && (out_token_stride >= head_dim || T <= 1),
              "out's heads overlap");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(x && pos && cos_sin && out, "null pointer argument");
  MOE_REQUIRE(aligned16(x) && aligned16(pos) && aligned16(cos_sin) && aligned16(out), "pointers must be 16-byte aligned");
  MOE_REQUIRE(x != out || (x_token_stride == out_token_stride && x_head_stride == out_head_stride),
              "in place needs the same strides");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int V = rope_vec(int(dtype_size(dtype)), rot, interleaved);
  const int turned = int((interleaved ? rot : rot / 2) / V);
  // in place the untouched part needs no visit
  const int units = x == out ? turned : rope_units(V, int(head_dim), int(rot), interleaved);
  // several heads a thread (128 bytes of loads: a unit of the half layout is two vectors, of the interleaved one a
  // single one) once that leaves every SM half a load of threads; with fewer threads too little is in flight, with more
  // they spend themselves on indices.  Several and one, from a graph, 32 heads of 128 in bf16: 128 tokens 3.1 and 2.6 us in
  // either layout, 1024 4.1 and 4.6 (interleaved, half of the head 4.6 and 5.2), 4096 8.2 and 11.3 (10.2 and 15.9), 16384
  // 42 and 48 (48 and 60); 16 heads in f32 within 8 % from 512 tokens on, interleaved 4096 7.7 and 12.8.  They are even at
  // a fifth to a third of this bound: what lies between pays up to 2.5 us (a cache append of 48 heads 4).
  const bool many = T * heads * units >= int64_t(num_sms()) * 1024 * (interleaved ? 8 : 4);
  auto typed = [&](auto zero) -> int {
    using E = decltype(zero);
    return rope_dispatch<int(sizeof(E))>(interleaved ? kRopeInter : kRopeHalf, V, many, [&](auto mode, auto vec, auto per) -> int {
      const int64_t blocks = cdiv(T * cdiv(heads, int64_t(decltype(per)::value)) * units, kThreads);
      MOE_SUPPORT(blocks < (int64_t(1) << 31) && heads * units < (int64_t(1) << 31), "T * heads too large");
      launch_pdl(rope_kernel<E, decltype(vec)::value, decltype(mode)::value, decltype(per)::value>, dim3(unsigned(blocks)),
                 dim3(kThreads), 0, st, static_cast<const E *>(x), x_token_stride, x_head_stride, pos, cos_sin, n_pos, T,
                 int(heads), int(rot), units, turned, inverse, static_cast<E *>(out), out_token_stride, out_head_stride);
      return MOE_OK;
    });
  };
  MOE_TRY(dtype == MOE_F16 ? typed(__half{}) : (dtype == MOE_BF16 ? typed(__nv_bfloat16{}) : typed(float{})));
  return check_launch("rope");
}
