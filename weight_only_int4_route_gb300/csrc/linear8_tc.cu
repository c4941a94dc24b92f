// Products of 8-bit integers for many rows, on the 16-bit tensor cores (tcgen05, accumulators in tensor memory).
//
// sm_103a has no 8-bit integer form of tcgen05.mma.  Every int8 is exact in f16, the product of two is at most 2^14, and 1024
// of them add up to at most 2^24: an fp32 accumulator over 1024 of K holds the integer sum exactly.  So K is cut into
// segments of 1024; the segments' accumulators alternate between two places in tensor memory, and the epilogue adds each to
// 32-bit integers while the tensor cores are at the next one.  The result is that of integer arithmetic, bit for bit.
//
// Orientation: D[128 channels x rows] = W[128 x K] . A^T[K x rows].
//   * W is the first operand: int8 tiles come by TMA, are converted in registers (one byte permute and one paired f16
//     subtraction for two values) and go straight into tensor memory.
//   * The rows are the second operand, read by the MMAs from shared memory.  They are converted once per call by a kernel of their
//     own into the workspace (3 bytes of traffic a value), not once per tile: shared memory is what bounds this kernel.
//     Per 128 of K it carries 32 KB of W (in and out) and 2 x 256 bytes a row (in and out), 256 + 4 n cycles at 128
//     bytes a cycle, beside 4 n cycles of MMAs: 1024 and 768 for the 192 rows a tile holds.  Converting the rows in
//     place would add 2 n and 1 n.
//   * Tensor memory: two accumulators of 192 columns, two W stages of 64.
//
// Warp roles (a CTA per SM, persistent over tiles):
//   warps 0-7    epilogue: warp w has lanes 32 (w % 4) and every other 32 columns;
//   warps 8-15   conversion, two groups of four warps; K block i belongs to group i % 2 and W stage i % 2;
//   warp 16, 17  copies of the rows (a ring of 3) and of W (a ring of 4: a multiple of the groups, so that a stage's
//                fills all go to one group and a wait by parity cannot be a phase ahead);
//   warp 18      MMAs, one thread.
// Few tiles: the CTAs of a cluster take a range of K each and add their integers up through distributed shared memory.
//
// Every wait is bounded (see tc_ptx.cuh); on expiry the CTA records a code, stops, drains its copies and MMAs, frees
// tensor memory and returns.
#include <algorithm>
#include <atomic>

#include "linear8.cuh"
#include "tc_ptx.cuh"

namespace moe {

__device__ int g_linear8_error = 0;

int linear8_error_take(int *out) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_linear8_error, sizeof(int)) != cudaSuccess) return check_launch("linear_w8a8 error read");
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_linear8_error, &zero, sizeof(int)) != cudaSuccess) return check_launch("linear_w8a8 error reset");
    *out = v;
  }
  return MOE_OK;
}

namespace {

constexpr int kEpiWarps = 8, kGroups = 2, kGroupWarps = 4;
constexpr int kConvWarp = kEpiWarps, kRowWarp = kConvWarp + kGroups * kGroupWarps, kWeightWarp = kRowWarp + 1, kMmaWarp = kRowWarp + 2;
constexpr int kTcThreads = (kRowWarp + 4) * 32;   // whole warpgroups: registers are dealt by them
constexpr int kEpiRegs = 152, kOtherRegs = 56;
constexpr int kBM = 128, kBN = 192, kBK = 128, kSegBlocks = 1024 / kBK;
constexpr int kRowStages = 3, kWStages = 4;
constexpr int kHalf = kBN * 128, kRowBytes = 2 * kHalf, kWBytes = kBM * kBK;
constexpr uint32_t kACol0 = 2 * kBN, kACols = kBK / 2;
static_assert(kWStages % kGroups == 0, "a W stage belongs to one group");
static_assert(2 * kBN + kGroups * (kBK / 2) <= 512, "tensor memory");
static_assert(kBN * kBM * 4 <= kRowStages * kRowBytes, "a tile's integers fit the rows' ring");
constexpr size_t kTcSmem = 1024 + kRowStages * kRowBytes + kWStages * kWBytes + 256;
static_assert(kTcSmem <= 232448, "shared memory");

enum : int { kErrFull = 51, kErrFree = 52, kErrReady = 53, kErrD = 54, kErrDrain = 55 };

struct TcArgs {
  LinearArgs p;
  int rows;          // of a tile, a multiple of 16
  int row_tiles, channel_blocks, blocks;   // blocks: 128-wide K blocks
  int splits, per;   // CTAs of a cluster, K blocks of each
};

struct Tile {
  int64_t row0;
  int ch0;
};
// Groups of 8 row tiles; inside, the row tiles of a channel block follow one another: CTAs that run together share W and rows in L2.
__device__ __forceinline__ Tile tile_at(const TcArgs &t, int i) {
  constexpr int kG = 8;
  const int group = i / (kG * t.channel_blocks), in = i - group * kG * t.channel_blocks;
  const int n = min(kG, t.row_tiles - group * kG);
  return {int64_t(group * kG + in % n) * t.rows, in / n * kBM};
}

template <typename OT>
__device__ __forceinline__ void store_columns(const LinearArgs &p, int64_t row0, int count, int ch, const int (&acc)[32], int lane) {
  const bool there = ch < p.N;
  const float sa = lane < count ? p.a_scale[row0 + lane] : 0.f, sw = there ? p.w_scale[ch] : 0.f;
  const float b = p.bias && there ? p.bias[ch] : 0.f;
  OT *o = static_cast<OT *>(p.out) + row0 * p.out_stride + ch;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float v = scaled(acc[j], __shfl_sync(0xffffffffu, sa, j), sw, p.bias != nullptr, b);
    if (there && j < count) o[j * p.out_stride] = from_f32<OT>(v);
  }
}

__global__ void __launch_bounds__(kTcThreads, 1)
    linear8_tc_kernel(const __grid_constant__ CUtensorMap map_rows, const __grid_constant__ CUtensorMap map_w, const TcArgs t) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  uint8_t *s_row = base, *s_w = s_row + kRowStages * kRowBytes;
  uint64_t *rfull = reinterpret_cast<uint64_t *>(s_w + kWStages * kWBytes), *done = rfull + kRowStages, *wfull = done + kRowStages,
           *wfree = wfull + kWStages, *ready = wfree + kWStages, *d_full = ready + kGroups, *d_empty = d_full + 2, *drain = d_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRowStages; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&done[s], 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wfree[s], kGroupWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ready[s], kGroupWarps);
      mbar_init(&d_full[s], 1);
      mbar_init(&d_empty[s], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_enter();   // what came before on the stream is complete from here on (see launch_pdl)

  const int rank = t.splits > 1 ? int(cluster_rank()) : 0;
  const int kb0 = rank * t.per, nkb = min(t.per, t.blocks - kb0);   // this CTA's K blocks: at least one
  const int segs = (nkb + kSegBlocks - 1) / kSegBlocks;
  const int tile0 = int(blockIdx.x) / t.splits, step = int(gridDim.x) / t.splits, tiles = t.row_tiles * t.channel_blocks;
  auto wait = [&](uint64_t *b, uint32_t parity, int code) { return mbar_wait(b, parity & 1, abort_flag, code, &g_linear8_error); };
  // a whole warp's wait: one that a lane gave up on has failed for all
  auto wait_warp = [&](uint64_t *b, uint32_t parity, int code) { return __all_sync(0xffffffffu, wait(b, parity, code)) != 0; };
  volatile int never = 0;

  if (warp < kEpiWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kEpiRegs));
    // ------------------------------------------------ epilogue
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + (uint32_t(q * 32) << 16);
    uint32_t seg = 0;
    bool ok = true;
    for (int i = tile0; ok && i < tiles; i += step) {
      const Tile tile = tile_at(t, i);
      int acc[3][32];
      for (int s = 0; s < segs; ++s, ++seg) {
        if (!(ok = wait_warp(&d_full[seg & 1], seg >> 1, kErrD))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int col = 32 * (2 * c + half);
          if (col >= t.rows) continue;
          float v[32];
          tc_ld32(lanes + (seg & 1) * kBN + uint32_t(col), v);
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = s == 0 ? __float2int_rn(v[j]) : acc[c][j] + __float2int_rn(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[seg & 1]);
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const int col = 32 * (2 * c + half);
        if (col >= t.rows) continue;
        if (t.splits > 1) {   // all of this CTA's MMAs are complete: the rows' ring is free
          int *sums = reinterpret_cast<int *>(s_row);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (col + j < t.rows) sums[(col + j) * kBM + q * 32 + lane] = acc[c][j];
        } else {
          const int64_t row0 = tile.row0 + col;
          const int count = int(min(int64_t(min(32, t.rows - col)), t.p.M - row0)), ch = tile.ch0 + q * 32 + lane;
          if (count <= 0) continue;
          if (t.p.out_dtype == MOE_F32) store_columns<float>(t.p, row0, count, ch, acc[c], lane);
          else if (t.p.out_dtype == MOE_F16) store_columns<__half>(t.p, row0, count, ch, acc[c], lane);
          else store_columns<__nv_bfloat16>(t.p, row0, count, ch, acc[c], lane);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp < kRowWarp) {
      // ------------------------------------------------ conversion into tensor memory
      const int q = warp & 3, group = (warp - kConvWarp) / kGroupWarps, r = q * 32 + lane;
      uint32_t it = 0;
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          if (int(it % kGroups) != group) continue;
          const uint32_t s = it % kWStages;
          // the tile's weights have landed; the MMAs that read this W stage last, those of block it - 2, are complete
          ok = wait_warp(&wfull[s], it / kWStages, kErrFull) &&
               (it < 2 || wait_warp(&done[(it - 2) % kRowStages], (it - 2) / kRowStages, kErrFree));
          if (!ok) break;
          tc_fence_after();
          const uint8_t *src = s_w + s * kWBytes + r * kBK;
          const uint32_t dst = tmem + (uint32_t(q * 32) << 16) + kACol0 + (it % kGroups) * kACols;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pr[16];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint4 w = *reinterpret_cast<const uint4 *>(src + 16 * ((2 * c + v) ^ (r & 7)));   // 128-byte swizzle
              const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t h[2];
                i2f_int8(words[j] ^ 0x80808080u, h, __half());
                pr[8 * v + 2 * j] = h[0];
                pr[8 * v + 2 * j + 1] = h[1];
              }
            }
            tc_st16(dst + uint32_t(16 * c), pr);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&wfree[s]);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[it % kGroups]);
        }
      }
    } else if (warp == kRowWarp && lane == 0) {
      // ------------------------------------------------ copies of the rows
      uint32_t it = 0;
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step) {
        const int row0 = int(tile_at(t, i).row0);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % kRowStages;
          if (!(ok = wait(&done[s], it / kRowStages + 1, kErrFree))) break;
          mbar_expect_tx(&rfull[s], uint32_t(t.rows) * 256);
          tma_load_2d(s_row + s * kRowBytes, &map_rows, (kb0 + kb) * kBK, row0, &rfull[s]);
          tma_load_2d(s_row + s * kRowBytes + kHalf, &map_rows, (kb0 + kb) * kBK + 64, row0, &rfull[s]);
        }
      }
      for (uint32_t n = it > kRowStages ? it - kRowStages : 0; n < it; ++n)
        mbar_wait(&rfull[n % kRowStages], (n / kRowStages) & 1, &never, kErrDrain, &g_linear8_error);
    } else if (warp == kWeightWarp && lane == 0) {
      // ------------------------------------------------ copies of W
      uint32_t it = 0;
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step) {
        const int ch0 = tile_at(t, i).ch0;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % kWStages;
          if (!(ok = wait(&wfree[s], it / kWStages + 1, kErrFree))) break;
          mbar_expect_tx(&wfull[s], kWBytes);
          tma_load_2d(s_w + s * kWBytes, &map_w, (kb0 + kb) * kBK, ch0, &wfull[s]);
        }
      }
      for (uint32_t n = it > kWStages ? it - kWStages : 0; n < it; ++n)
        mbar_wait(&wfull[n % kWStages], (n / kWStages) & 1, &never, kErrDrain, &g_linear8_error);
    } else if (warp == kMmaWarp && lane == 0) {
      // ------------------------------------------------ MMAs
      const uint32_t idesc = idesc_f16(0, kBM, t.rows);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t first = kb % kSegBlocks, s = it % kRowStages;
          if (first == 0 && !(ok = wait(&d_empty[seg & 1], (seg >> 1) + 1, kErrD))) break;
          if (!(ok = wait(&rfull[s], it / kRowStages, kErrFull) && wait(&ready[it % kGroups], it / kGroups, kErrReady))) break;
          tc_fence_after();
          tc_mma_kblock_ts<kHalf / 16, false>(tmem + (seg & 1) * kBN, tmem + kACol0 + (it % kGroups) * kACols,
                                              sw128_desc(su32(s_row + s * kRowBytes)), idesc, first);
          tc_commit(&done[s]);
          if (first == kSegBlocks - 1 || kb == nkb - 1) tc_commit(&d_full[seg++ & 1]);
        }
      }
      tc_commit(drain);
      mbar_wait(drain, 0, &never, kErrDrain, &g_linear8_error);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  if (t.splits == 1) return;
  // ---- the cluster's integers: each CTA adds up and stores every splits-th row of the tile
  __syncwarp();
  cluster_sync();
  if (*abort_flag == 0 && tile0 < tiles) {
    const Tile tile = tile_at(t, tile0);
    const int c = threadIdx.x & (kBM - 1), ch = tile.ch0 + c;
    const int count = int(min(int64_t(t.rows), t.p.M - tile.row0));
    const uint32_t sums = su32(s_row) + 4 * c;
    if (ch < t.p.N) {
      const float sw = t.p.w_scale[ch], b = t.p.bias ? t.p.bias[ch] : 0.f;
#pragma unroll 4
      for (int row = rank + t.splits * int(threadIdx.x / kBM); row < count; row += t.splits * (kTcThreads / kBM)) {
        int acc = 0;
        for (int r = 0; r < t.splits; ++r) {
          uint32_t from;
          int v;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(from) : "r"(sums + 4 * kBM * row), "r"(r));
          asm volatile("ld.shared::cluster.s32 %0, [%1];\n" : "=r"(v) : "r"(from) : "memory");
          acc += v;
        }
        store_out(t.p.out, t.p.out_dtype, (tile.row0 + row) * t.p.out_stride + ch,
                  scaled(acc, t.p.a_scale[tile.row0 + row], sw, t.p.bias != nullptr, b));
      }
    }
  }
  __syncwarp();
  cluster_sync();   // no CTA leaves while its integers are read
}

// int8 rows -> f16 rows of `pitch` values, zeros past K.
template <bool VEC>
__global__ void __launch_bounds__(256) expand_rows_kernel(const int8_t *__restrict__ a, int64_t stride, int64_t M, int K, int pitch,
                                                          __half *__restrict__ out) {
  pdl_enter();
  const int per = pitch / 16;
  const int64_t total = M * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per;
    const int k = int(i - r * per) * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    const int8_t *src = a + r * stride + k;
    if (VEC) {
      if (k < K) v = *reinterpret_cast<const uint4 *>(src);
    } else {
      int8_t *b = reinterpret_cast<int8_t *>(&v);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (k + j < K) b[j] = src[j];
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
    uint4 *dst = reinterpret_cast<uint4 *>(out + r * pitch + k);
    dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
    dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// Rows of a tile and CTAs of a cluster: the pair with the least time by the kernel's own cycle counts (shared memory and MMAs of a
// K block, 100 between blocks, a tile's start and end, the exchange of a cluster).
void plan(TcArgs &t, int64_t M, int sms) {
  const int64_t least = cdiv(M, kBN), most = std::max(least, std::min<int64_t>(cdiv(M, 64), least + 6));
  double best = 1e30;
  for (int64_t n = least; n <= most; ++n) {
    const int rows = int(cdiv(cdiv(M, n), 16) * 16);
    const int64_t tiles = cdiv(M, rows) * t.channel_blocks;
    const double block = std::max(256.0 + 4 * rows, 704.0) + 100;
    for (int s = 1; s <= 8; ++s) {
      if (s > 1 && tiles * s > sms) break;
      const int per = int(cdiv(t.blocks, s));
      if (cdiv(t.blocks, per) != s) continue;
      const double time = double(cdiv(tiles * s, sms)) * (per * block + 2000 + 8 * rows) + (s > 1 ? 2500 + 40 * rows / s : 0);
      if (time < best) {
        best = time;
        t.rows = rows;
        t.row_tiles = int(cdiv(M, rows));
        t.splits = s;
        t.per = per;
      }
    }
  }
}

}  // namespace

size_t linear8_tc_rows_bytes(int64_t M, int64_t K) { return align256(size_t(M) * size_t(cdiv(K, kBK) * kBK) * 2); }

int launch_linear8_tc(const LinearArgs &p, void *rows16, cudaStream_t st) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("linear_w8a8: cudaGetDevice");
  if (dev < 0 || dev >= 64) return set_error(MOE_ERR_UNSUPPORTED, "linear_w8a8: device index %d >= 64", dev);
  TcArgs t{};
  t.p = p;
  t.blocks = int(cdiv(p.K, kBK));
  t.channel_blocks = int(cdiv(p.N, kBM));
  plan(t, p.M, num_sms());
  const int pitch = t.blocks * kBK;
  CUtensorMap map_rows, map_w;
  {
    const cuuint64_t dims[2] = {cuuint64_t(pitch), cuuint64_t(p.M)}, strides[1] = {cuuint64_t(pitch) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(t.rows)}, es[2] = {1, 1};
    const CUresult r = enc(&map_rows, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows16, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(MOE_ERR_CUDA, "row tensor map encode failed (%d)", int(r));
  }
  {
    const cuuint64_t dims[2] = {cuuint64_t((p.K + 15) & ~15), cuuint64_t(p.N)}, strides[1] = {cuuint64_t(p.w_stride)};
    const cuuint32_t box[2] = {kBK, kBM}, es[2] = {1, 1};
    const CUresult r = enc(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(p.w), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(MOE_ERR_CUDA, "weight tensor map encode failed (%d)", int(r));
  }
  static std::atomic<bool> attr_set[64];
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(linear8_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmem)) != cudaSuccess)
      return check_launch("linear_w8a8 attribute");
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  const int64_t work = p.M * (pitch / 16);
  const dim3 blocks(unsigned(std::min<int64_t>(cdiv(work, 256), int64_t(num_sms()) * 32)));
  if (p.K % 16 == 0 && p.a_stride % 16 == 0 && aligned16(p.a))
    launch_pdl(expand_rows_kernel<true>, blocks, dim3(256), 0, st, p.a, p.a_stride, p.M, p.K, pitch, static_cast<__half *>(rows16));
  else
    launch_pdl(expand_rows_kernel<false>, blocks, dim3(256), 0, st, p.a, p.a_stride, p.M, p.K, pitch, static_cast<__half *>(rows16));
  MOE_TRY(check_launch("linear_w8a8 rows"));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(t.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  const int64_t tiles = int64_t(t.row_tiles) * t.channel_blocks;
  cfg.gridDim = dim3(unsigned(t.splits > 1 ? tiles * t.splits : std::min<int64_t>(tiles, num_sms())));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = t.splits > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, linear8_tc_kernel, map_rows, map_w, t);
  return check_launch("linear_w8a8");
}

}  // namespace moe
