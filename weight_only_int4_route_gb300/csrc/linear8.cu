// Product of 8-bit integers with a scale for each token and each output channel:
//   out[m, n] = RN(((sum_k a[m, k] w[n, k]) a_scale[m]) w_scale[n] (+ bias[n]))
//
// The sum is exact in 32-bit integers, so its order and its split over warps and CTAs do not show: every form below gives the
// same bits.
#include <algorithm>

#include "linear8.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

// Rows of K bytes -> rows of `pitch` bytes, zeros behind: weights whose rows do not start on 16 bytes.
__global__ void __launch_bounds__(256) pad_rows_kernel(const int8_t *w, int64_t stride, int64_t rows, int K, int pitch, int8_t *out) {
  pdl_enter();
  const int64_t total = rows * pitch;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / pitch;
    const int k = int(i - r * pitch);
    out[i] = k < K ? w[r * stride + k] : int8_t(0);
  }
}

// ---- a few rows: the weights as a stream ------------------------------------------------------------------------------
//
// A CTA takes 16 channels and 8 MT rows over a range of K; its 8 warps take the range's 256-wide pieces in turn and add their
// sums up in shared memory, the CTAs of a cluster (splits of K) theirs in the first one's.  The weights are the A operand
// of m16n8k32 (s8, s32 accumulators) straight from 16-byte loads: the order of a sum's terms is free, so a lane's
// four consecutive words stand for the four 4-wide slots that two MMAs want of it, and the rows' values, read from
// shared memory the same way, match.
constexpr int kStreamThreads = 256, kStreamWarps = 8, kChunk = 256;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_stream(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// phase: K range whose rows' values fit the shared memory; split: K range of a CTA (both multiples of kChunk)
template <int MT>
__global__ void __launch_bounds__(kStreamThreads) linear8_stream_kernel(const LinearArgs p, int splits, int split, int phase,
                                                                        int vector_rows) {
  pdl_enter();
  extern __shared__ __align__(16) int8_t s_rows[];   // 8 MT rows of phase + 64 bytes: two rows' pieces share no bank
  __shared__ int s_sum[8 * MT][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int rank = splits > 1 ? int(cluster_rank()) : 0;
  const int n0 = int(blockIdx.x) / splits * 16;
  const int64_t m0 = int64_t(blockIdx.y) * (8 * MT);
  const int rows = int(min(int64_t(8 * MT), p.M - m0));
  const int kr = (p.K + 15) & ~15, k0 = rank * split, k1 = min(kr, k0 + split);
  const int pitch = phase + 64;
  for (int i = tid; i < 8 * MT * 16; i += kStreamThreads) (&s_sum[0][0])[i] = 0;
  if (splits > 1) {   // every CTA's sums are zero: waited for before the first one's are added to
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  }

  int c[MT][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[t][i] = 0;
  const bool lo_there = n0 + g < p.N, hi_there = n0 + g + 8 < p.N;
  const int8_t *w_lo = p.w + int64_t(n0 + g) * p.w_stride, *w_hi = w_lo + 8 * p.w_stride;
  uint4 lo[4], hi[4];
  auto fetch = [&](int k, int end) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = k + 64 * j + 16 * q;
      lo[j] = lo_there && at < end ? load_stream(w_lo + at) : make_uint4(0, 0, 0, 0);
      hi[j] = hi_there && at < end ? load_stream(w_hi + at) : make_uint4(0, 0, 0, 0);
    }
  };
  for (int ph = k0; ph < k1; ph += phase) {
    const int end = min(k1, ph + phase);
    int k = ph + warp * kChunk;
    if (k < end) fetch(k, end);
    __syncthreads();   // the last phase's rows have been read
    if (vector_rows) {
      const int per = (end - ph) >> 4;
      for (int i = tid; i < per * 8 * MT; i += kStreamThreads) {
        const int r = i / per, at = (i - r * per) << 4;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) v = *reinterpret_cast<const uint4 *>(p.a + (m0 + r) * p.a_stride + ph + at);
        *reinterpret_cast<uint4 *>(s_rows + r * pitch + at) = v;
      }
    } else {
      const int per = end - ph;
      for (int i = tid; i < per * 8 * MT; i += kStreamThreads) {
        const int r = i / per, at = i - r * per;
        s_rows[r * pitch + at] = r < rows && ph + at < p.K ? p.a[(m0 + r) * p.a_stride + ph + at] : int8_t(0);
      }
    }
    __syncthreads();
    while (k < end) {
      uint4 wl[4], wh[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wl[j] = lo[j];
        wh[j] = hi[j];
      }
      const int8_t *rp = s_rows + g * pitch + (k - ph) + 16 * q;
      k += kStreamWarps * kChunk;
      if (k < end) fetch(k, end);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint4 b = *reinterpret_cast<const uint4 *>(rp + t * 8 * pitch + 64 * j);
          mma_s8(c[t], wl[j].x, wh[j].x, wl[j].y, wh[j].y, b.x, b.y);
          mma_s8(c[t], wl[j].z, wh[j].z, wl[j].w, wh[j].w, b.z, b.w);
        }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    atomicAdd(&s_sum[8 * t + 2 * q][g], c[t][0]);
    atomicAdd(&s_sum[8 * t + 2 * q + 1][g], c[t][1]);
    atomicAdd(&s_sum[8 * t + 2 * q][g + 8], c[t][2]);
    atomicAdd(&s_sum[8 * t + 2 * q + 1][g + 8], c[t][3]);
  }
  __syncthreads();
  if (splits > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (rank != 0) {
      const uint32_t to = map_to_rank(&s_sum[0][0], 0);
      for (int i = tid; i < 16 * rows; i += kStreamThreads)
        asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;\n" ::"r"(to + 4 * i), "r"((&s_sum[0][0])[i]) : "memory");
    }
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
  }
  for (int i = tid; i < 16 * rows; i += kStreamThreads) {
    const int r = i >> 4, n = n0 + (i & 15);
    if (n < p.N)
      store_out(p.out, p.out_dtype, (m0 + r) * p.out_stride + n, scaled(s_sum[r][i & 15], p.a_scale[m0 + r], p.w_scale[n], p.bias != nullptr, p.bias ? p.bias[n] : 0.f));
  }
}

template <int MT> int launch_stream(const LinearArgs &p, cudaStream_t st) {
  const int64_t tiles = cdiv(p.N, 16), chunks = cdiv(p.M, 8 * MT);
  const int kr = (p.K + 15) & ~15;
  // splits of K: two CTAs for every SM, at least 512 of K each
  int splits = 1;
  while (splits < 8 && tiles * chunks * splits < 2 * num_sms() && kr / (2 * splits) >= 512) splits *= 2;
  const int split = int(cdiv(cdiv(kr, splits), kChunk) * kChunk);
  const int most = 96 * 1024 / (8 * MT) - 64;
  const int phase = std::min(split, most / kChunk * kChunk);
  const size_t smem = size_t(8 * MT) * (phase + 64);
  const int vector_rows = p.K % 16 == 0 && p.a_stride % 16 == 0 && aligned16(p.a);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("linear_w8a8: cudaGetDevice");
  if (cudaFuncSetAttribute(linear8_stream_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024) != cudaSuccess)
    return check_launch("linear_w8a8 attribute");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(tiles * splits), unsigned(chunks));
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, linear8_stream_kernel<MT>, p, splits, split, phase, vector_rows);
  return check_launch("linear_w8a8");
}

// Rows up to which the weights are streamed past all of them at once.
constexpr int64_t kStreamRows = 32;

// The workspace: the weights' rows padded to 16 bytes (used if they need it), then the rows as f16 (many rows).
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
  const size_t need = (pad || many ? padded_bytes(N, K) : 0) + (many ? linear8_tc_rows_bytes(M, K) : 0);
  if (need > 0) {
    if (workspace_bytes < need) return set_error(MOE_ERR_WORKSPACE, "linear_w8a8 workspace %zu < %zu bytes", workspace_bytes, need);
    MOE_REQUIRE(workspace && aligned16(workspace), "workspace must be non-null and 16-byte aligned");
  }
  if (pad) {
    const int pitch = int((K + 15) & ~int64_t(15));
    int8_t *padded = static_cast<int8_t *>(workspace);
    const int64_t blocks = std::min<int64_t>(cdiv(N * pitch, 256), int64_t(num_sms()) * 32);
    launch_pdl(pad_rows_kernel, dim3(unsigned(blocks)), dim3(256), 0, st, w, p.w_stride, N, int(K), pitch, padded);
    MOE_TRY(check_launch("linear_w8a8 padding"));
    p.w = padded;
    p.w_stride = pitch;
  }
  if (many) return launch_linear8_tc(p, static_cast<char *>(workspace) + padded_bytes(N, K), st);
  if (M <= 8) return launch_stream<1>(p, st);
  if (M <= 16) return launch_stream<2>(p, st);
  return launch_stream<4>(p, st);
}
