// Product of 8-bit integers with a scale for each token and each output channel:
//   out[m, n] = RN(((sum_k a[m, k] w[n, k]) a_scale[m]) w_scale[n] (+ bias[n]))
//
// The sum is exact in 32-bit integers, so its order and its split over warps and CTAs do not show: every form below gives the
// same bits.
#include <algorithm>
#include <atomic>

#include "linear8.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

// Rows of K bytes -> rows of `pitch` bytes, zeros behind: weights whose rows do not start on 16 bytes.  A thread per 16 bytes.
__global__ void __launch_bounds__(256) pad_rows_kernel(const int8_t *w, int64_t stride, int64_t rows, int K, int pitch, int8_t *out) {
  pdl_enter();
  const int per = pitch / 16;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
    const int64_t r = (i >> 32) == 0 ? int64_t(uint32_t(i) / uint32_t(per)) : i / per;
    const int k = int(i - r * per) * 16;
    const int8_t *src = w + r * stride + k;
    uint4 v = make_uint4(0, 0, 0, 0);
    int8_t *byte = reinterpret_cast<int8_t *>(&v);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (k + j < K) byte[j] = src[j];
    *reinterpret_cast<uint4 *>(out + r * pitch + k) = v;
  }
}

// ---- a few rows: the weights as a stream ------------------------------------------------------------------------------
//
// A CTA takes 16 CT channels and 8 MT rows over a range of K; its 8 warps take the range's pieces in turn and add their
// sums up in shared memory, the CTAs of a cluster (splits of K) theirs in the first one's.  The weights are the A operand
// of m16n8k16 (f16, fp32 accumulators), converted in registers from 16-byte loads: the order of a sum's terms is free, so a
// lane's 16 consecutive values stand for the slots that four MMAs want of it, and the rows' values, f16 in shared memory and
// read the same way, match.  (m16n8k32 on the integers themselves takes 128 cycles a sub-core on this chip: one row of 4096 x 6144
// 8.2 us, 16 rows 16.3 us.)  A warp's accumulators are emptied into the 32-bit integers after 1024 of K: up to there an
// fp32 sum of these products is exact.  Measured on GB300: one row of 6144 x 4096 7.2 us, 3.5 TB/s, of 32768 x 2048 17.6 us, 3.8 TB/s; a
// third of the first is launch, the rows' way to shared memory and the joining of the sums.
constexpr int kStreamThreads = 256, kStreamWarps = 8, kStreamSmem = 72 * 1024;

__device__ __forceinline__ uint4 load_stream(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// phase: K range whose rows' values fit the shared memory; split: K range of a CTA (both multiples of 256)
template <int MT, int CT>
__global__ void __launch_bounds__(kStreamThreads, 2) linear8_stream_kernel(const LinearArgs p, int splits, int split, int phase,
                                                                           int vector_rows) {
  pdl_enter();
  constexpr int kChunk = 256 / CT, kPieces = kChunk / 64;   // K of a step: 8 loads a lane
  extern __shared__ __align__(16) uint8_t s_rows[];         // 8 MT rows of phase f16 values + 16 bytes: no bank conflicts
  __shared__ int s_sum[8 * MT][16 * CT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int rank = splits > 1 ? int(cluster_rank()) : 0;
  const int n0 = int(blockIdx.x) / splits * (16 * CT);
  const int rows = int(p.M);
  const int kr = (p.K + 15) & ~15, k0 = rank * split, k1 = min(kr, k0 + split);
  const int pitch = 2 * phase + 16;
  for (int i = tid; i < 8 * MT * 16 * CT; i += kStreamThreads) (&s_sum[0][0])[i] = 0;
  if (splits > 1) {   // every CTA's sums are zero: waited for before the first one's are added to
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  }

  float c[CT][MT][4];
  auto clear = [&] {
#pragma unroll
    for (int u = 0; u < CT; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[u][t][i] = 0.f;
  };
  auto flush = [&] {
#pragma unroll
    for (int u = 0; u < CT; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (8 * t + 2 * q + (i & 1) < rows)
            atomicAdd(&s_sum[8 * t + 2 * q + (i & 1)][16 * u + g + 8 * (i >> 1)], __float2int_rn(c[u][t][i]));
  };
  clear();
  const int8_t *w = p.w + int64_t(n0 + g) * p.w_stride + 16 * q;
  uint4 r[2 * CT][kPieces];
  auto fetch = [&](int k, int end) {
#pragma unroll
    for (int i = 0; i < 2 * CT; ++i)
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        r[i][j] = n0 + g + 8 * i < p.N && k + 64 * j + 16 * q < end ? load_stream(w + 8 * i * p.w_stride + k + 64 * j) : make_uint4(0, 0, 0, 0);
  };
  for (int ph = k0; ph < k1; ph += phase) {
    const int end = min(k1, ph + phase);
    int k = ph + warp * kChunk;
    if (k < end) fetch(k, end);
    __syncthreads();   // the last phase's rows have been read; the sums are zero
    const int per = (end - ph) >> 4;
    for (int i = tid; i < per * rows; i += kStreamThreads) {
      const int m = i / per, at = (i - m * per) << 4;
      uint4 v = make_uint4(0, 0, 0, 0);
      const int8_t *src = p.a + m * p.a_stride + ph + at;
      if (vector_rows) {
        v = *reinterpret_cast<const uint4 *>(src);
      } else {
        int8_t *byte = reinterpret_cast<int8_t *>(&v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (ph + at + j < p.K) byte[j] = src[j];
      }
      uint32_t h[8];
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t two[2];
        i2f_int8(words[j] ^ 0x80808080u, two, __half());
        h[2 * j] = two[0];
        h[2 * j + 1] = two[1];
      }
      uint4 *dst = reinterpret_cast<uint4 *>(s_rows + m * pitch + 2 * at);
      dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
      dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
    __syncthreads();
    int steps = 0;
    while (k < end) {
      const uint8_t *rp = s_rows + 2 * (k - ph + 16 * q);
      // the pieces of this step that hold anything: what lies behind has not been written
      const int here = (end - k + 63) >> 6;
      uint4 now[2 * CT][kPieces];
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i)
#pragma unroll
        for (int j = 0; j < kPieces; ++j) now[i][j] = r[i][j];
      k += kStreamWarps * kChunk;
      if (k < end) fetch(k, end);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (j >= here) break;
        uint32_t a[2 * CT][8];
#pragma unroll
        for (int i = 0; i < 2 * CT; ++i) {
          const uint32_t words[4] = {now[i][j].x, now[i][j].y, now[i][j].z, now[i][j].w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t two[2];
            i2f_int8(words[s] ^ 0x80808080u, two, __half());
            a[i][2 * s] = two[0];
            a[i][2 * s + 1] = two[1];
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          // rows past the last one and values past a ragged end: zeros (f16 garbage could be NaN)
          const bool there = 8 * t + g < rows;
          const uint8_t *src = rp + (8 * t + g) * pitch + 128 * j;
          uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
          if (there && k - kStreamWarps * kChunk + 64 * j + 16 * q < end) {
            b0 = *reinterpret_cast<const uint4 *>(src);
            b1 = *reinterpret_cast<const uint4 *>(src + 16);
          }
#pragma unroll
          for (int u = 0; u < CT; ++u) {
            const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint32_t f[4] = {a[2 * u][2 * s], a[2 * u + 1][2 * s], a[2 * u][2 * s + 1], a[2 * u + 1][2 * s + 1]};
              mma16816(c[u][t], f, b[2 * s], b[2 * s + 1], __half());
            }
          }
        }
      }
      if (++steps == 1024 / kChunk) {
        flush();
        clear();
        steps = 0;
      }
    }
    if (steps) {
      flush();
      clear();
    }
  }
  __syncthreads();
  if (splits > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (rank != 0) {
      const uint32_t to = map_to_rank(&s_sum[0][0], 0);
      for (int i = tid; i < 16 * CT * rows; i += kStreamThreads)
        asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;\n" ::"r"(to + 4 * i), "r"((&s_sum[0][0])[i]) : "memory");
    }
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
  }
  for (int i = tid; i < 16 * CT * rows; i += kStreamThreads) {
    const int m = i / (16 * CT), at = i % (16 * CT), n = n0 + at;
    if (n < p.N)
      store_out(p.out, p.out_dtype, m * p.out_stride + n,
                scaled(s_sum[m][at], p.a_scale[m], p.w_scale[n], p.bias != nullptr, p.bias ? p.bias[n] : 0.f));
  }
}

template <int MT, int CT> int launch_stream(const LinearArgs &p, cudaStream_t st) {
  const int64_t tiles = cdiv(p.N, 16 * CT);
  const int kr = (p.K + 15) & ~15;
  // splits of K: as many as still run all at once, at least 512 of K each
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= 2 * num_sms() && kr / (2 * splits) >= 512) splits *= 2;
  const int split = int(cdiv(cdiv(kr, splits), 256) * 256);
  const int most = (kStreamSmem / (8 * MT) - 16) / 2 / 256 * 256;
  const int phase = std::min(split, most);
  const size_t smem = size_t(8 * MT) * (2 * phase + 16);
  const int vector_rows = p.K % 16 == 0 && p.a_stride % 16 == 0 && aligned16(p.a);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("linear_w8a8: cudaGetDevice");
  if (dev < 0 || dev >= 64) return set_error(MOE_ERR_UNSUPPORTED, "linear_w8a8: device index %d >= 64", dev);
  static std::atomic<bool> attr_set[64];
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(linear8_stream_kernel<MT, CT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem) != cudaSuccess)
      return check_launch("linear_w8a8 attribute");
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(tiles * splits));
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, linear8_stream_kernel<MT, CT>, p, splits, split, phase, vector_rows);
  return check_launch("linear_w8a8");
}

// Rows up to which the weights are streamed past all of them at once, whatever N and K.  24 rows there and on tcgen05: 4096 x 4096
// 15.7 and 11.6 us, 6144 x 4096 25.0 and 15.3, but 2048 x 2048 6.5 and 9.2: small weights would gain from the stream up to 24 rows.
// 16 rows 8.6, 13.4 and 5.2 there.
constexpr int64_t kStreamRows = 16;

// The workspace: the rows as f16 (many rows), then the weights' rows padded to 16 bytes (if they need it).
size_t padded_bytes(int64_t N, int64_t K) { return align256(size_t(N) * size_t((K + 15) & ~int64_t(15))); }
bool needs_padding(const int8_t *w, int64_t w_stride, int64_t K) { return K % 16 != 0 || w_stride % 16 != 0 || !aligned16(w); }

int check_sizes(int64_t M, int64_t N, int64_t K) {
  MOE_REQUIRE(M >= 0 && M < (int64_t(1) << 31) && N >= 0 && N < (int64_t(1) << 27), "M or N out of range");
  MOE_REQUIRE(K >= 1 && K <= 131071, "1 <= K <= 131071: longer sums do not fit 32 bits (K=%lld)", (long long)K);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_w8a8_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (check_sizes(M, N, K) != MOE_OK) return 0;
  return padded_bytes(N, K) + (M > kStreamRows ? linear8_tc_rows_bytes(M, K) : 0);
}

extern "C" int moe_linear_w8a8(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w, int64_t w_stride,
                               const float *w_scale, const float *bias, int64_t M, int64_t N, int64_t K, void *out,
                               int64_t out_stride, int out_dtype, void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_sizes(M, N, K));
  MOE_REQUIRE(out_dtype == MOE_F16 || out_dtype == MOE_BF16 || out_dtype == MOE_F32, "bad out_dtype %d", out_dtype);
  MOE_REQUIRE((a_stride >= K || M <= 1) && (w_stride >= K || N <= 1) && (out_stride >= N || M <= 1), "rows overlap");
  if (M == 0 || N == 0) return MOE_OK;
  MOE_REQUIRE(a && a_scale && w && w_scale && out, "null pointer argument");
  MOE_REQUIRE(aligned16(a_scale) && aligned16(w_scale) && aligned16(bias), "scales and bias must be 16-byte aligned");
  MOE_REQUIRE((reinterpret_cast<uintptr_t>(out) & (dtype_size(out_dtype) - 1)) == 0, "out must start on an element");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LinearArgs p{a, w, a_scale, w_scale, bias, out, M, a_stride, w_stride, out_stride, int(N), int(K), out_dtype};
  if (N == 1) p.w_stride = (K + 15) & ~int64_t(15);   // a single row's is not looked at
  const bool pad = needs_padding(w, p.w_stride, K), many = M > kStreamRows;
  const size_t rows_bytes = many ? linear8_tc_rows_bytes(M, K) : 0, need = rows_bytes + (pad ? padded_bytes(N, K) : 0);
  if (need > 0) {
    if (workspace_bytes < need) return set_error(MOE_ERR_WORKSPACE, "linear_w8a8 workspace %zu < %zu bytes", workspace_bytes, need);
    MOE_REQUIRE(workspace && aligned16(workspace), "workspace must be non-null and 16-byte aligned");
  }
  if (pad) {
    const int pitch = int((K + 15) & ~int64_t(15));
    int8_t *padded = static_cast<int8_t *>(workspace) + rows_bytes;
    const int64_t blocks = std::min<int64_t>(cdiv(N * (pitch / 16), 256), int64_t(num_sms()) * 32);
    launch_pdl(pad_rows_kernel, dim3(unsigned(blocks)), dim3(256), 0, st, w, p.w_stride, N, int(K), pitch, padded);
    MOE_TRY(check_launch("linear_w8a8 padding"));
    p.w = padded;
    p.w_stride = pitch;
  }
  if (many) return launch_linear8_tc(p, workspace, st);
  // 16 channels a CTA for few rows and channels, else 32 (the rows' values are read from shared memory half as often): 1 row
  // 4096 x 4096 5.2 and 5.5 us, 6144 x 4096 7.7 and 7.2, 32768 x 2048 21.1 and 17.6; 16 rows 10.3 and 8.6, 18.1 and 13.4,
  // 37.6 and 29.2
  if (M <= 8) return cdiv(N, 16) <= 2 * num_sms() ? launch_stream<1, 1>(p, st) : launch_stream<1, 2>(p, st);
  return launch_stream<2, 2>(p, st);
}
