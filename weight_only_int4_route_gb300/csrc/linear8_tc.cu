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
//   warp 18      MMAs, one thread;
//   warp 19      passes the arrival of a block's rows on to the barrier of its W stage: the MMA thread has one wait a block.
// Few tiles: the CTAs of a cluster take a range of K each and add their integers up through distributed shared memory.
//
// Measured on GB300: 8192 x 6144 x 4096 279 us with the rows' conversion (15 us), 1.48 PFLOP/s, 0.85 of the sustained 16-bit rate; a K
// block takes 1000 cycles, what shared memory needs.  300 x 6144 x 2048 17.4 us, 24 rows of 4096 x 4096 11.6 us: there a block takes
// the MMA thread's 850 cycles (8 issues of 65, a wait, a commit), and 6 us are launches, first copies and the outputs.
// Tried: W stages of half a K block, four of them (8192 rows 346 us at the time of 314: twice the waits and commits);
// waits that test without suspending (no change).
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
constexpr int kConvWarp = kEpiWarps, kRowWarp = kConvWarp + kGroups * kGroupWarps, kWeightWarp = kRowWarp + 1, kMmaWarp = kRowWarp + 2, kRelayWarp = kRowWarp + 3;
constexpr int kTcThreads = (kRowWarp + 4) * 32;   // whole warpgroups: registers are dealt by them
constexpr int kEpiRegs = 144, kOtherRegs = 64;   // 256 x 144 + 384 x 64 = 640 x 96, all there are
// CTAs of a cluster at most.  Clusters of 8 with this much shared memory do not all run at once (2048 x 2048, 24 rows: 12 us with 4,
// 21 with 8), and sizes that are no power of two leave SMs idle (3: 26 us where 2 took 18).
constexpr int kMaxSplits = 4;
constexpr int kBM = 128, kBN = 192, kBK = 128, kSegBlocks = 1024 / kBK;
constexpr int kRowStages = 3, kWStages = 4;
constexpr int kHalf = kBN * 128, kRowBytes = 2 * kHalf, kWBytes = kBM * kBK;
constexpr uint32_t kACol0 = 2 * kBN, kACols = kBK / 2;
static_assert(kWStages % kGroups == 0, "a W stage belongs to one group");
static_assert(2 * kBN + kGroups * (kBK / 2) <= 512, "tensor memory");
static_assert(kBN * kBM * 4 <= kRowStages * kRowBytes, "a tile's integers fit the rows' ring");
constexpr size_t kTcSmem = 1024 + kRowStages * kRowBytes + kWStages * kWBytes + 2 * 16 * kBM * 4 + 256;
static_assert(kTcSmem <= 232448, "shared memory");

enum : int { kErrFull = 51, kErrFree = 52, kErrReady = 53, kErrD = 54, kErrDrain = 55 };

struct TcArgs {
  LinearArgs p;
  int rows;          // of a tile, a multiple of 16
  int row_tiles, channel_blocks, blocks;   // blocks: 128-wide K blocks
  int splits, per;   // CTAs of a cluster, K blocks of each
  int vector;        // four results may be stored at once
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

// A row's four channels from ch on (those below n) from their integers.
struct FourScales {
  float w[4], b[4];
};
__device__ __forceinline__ void load_four(const LinearArgs &p, int ch, FourScales &f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.w[j] = ch + j < p.N ? p.w_scale[ch + j] : 0.f;
    f.b[j] = p.bias && ch + j < p.N ? p.bias[ch + j] : 0.f;
  }
}
__device__ __forceinline__ void store_four(const LinearArgs &p, bool vector, int64_t row, float sa, int ch, const int4 &acc,
                                           const FourScales &f) {
  const bool bias = p.bias != nullptr;
  const float v[4] = {scaled(acc.x, sa, f.w[0], bias, f.b[0]), scaled(acc.y, sa, f.w[1], bias, f.b[1]),
                      scaled(acc.z, sa, f.w[2], bias, f.b[2]), scaled(acc.w, sa, f.w[3], bias, f.b[3])};
  const int64_t at = row * p.out_stride + ch;
  if (vector && ch + 4 <= p.N) {
    if (p.out_dtype == MOE_F32) {
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 two;
      if (p.out_dtype == MOE_F16) two = make_uint2(h2_as_u32(__floats2half2_rn(v[0], v[1])), h2_as_u32(__floats2half2_rn(v[2], v[3])));
      else two = make_uint2(h2_as_u32(__floats2bfloat162_rn(v[0], v[1])), h2_as_u32(__floats2bfloat162_rn(v[2], v[3])));
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = two;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ch + j < p.N) store_out(p.out, p.out_dtype, at + j, v[j]);
  }
}

// Whether `ok` holds in all 128 threads that share barrier `id`.
__device__ __forceinline__ bool all_of_half(int id, bool ok) {
  int all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.s32 q, %1, 0;\n bar.red.and.pred p, %2, 128, q;\n selp.s32 %0, 1, 0, p;\n}\n"
               : "=r"(all)
               : "r"(int(ok)), "r"(id)
               : "memory");
  return all != 0;
}

__global__ void __launch_bounds__(kTcThreads, 1)
    linear8_tc_kernel(const __grid_constant__ CUtensorMap map_rows, const __grid_constant__ CUtensorMap map_w, const TcArgs t) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  uint8_t *s_row = base, *s_w = s_row + kRowStages * kRowBytes;
  int *s_stage = reinterpret_cast<int *>(s_w + kWStages * kWBytes);   // two halves' 16 rows
  uint64_t *rfull = reinterpret_cast<uint64_t *>(s_stage + 2 * 16 * kBM), *done = rfull + kRowStages, *wfull = done + kRowStages,
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
      mbar_init(&ready[s], kGroupWarps + 1);
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
      // what the outputs are scaled by, on its way early: four channels a lane, a row a lane of each 32
      const int ch = tile.ch0 + 4 * lane, count = int(min(int64_t(t.rows), t.p.M - tile.row0));
      FourScales f;
      float sa[3];
      if (t.splits == 1) {
        load_four(t.p, ch, f);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int row = 32 * (2 * c + half) + lane;
          sa[c] = row < count ? t.p.a_scale[tile.row0 + row] : 0.f;
        }
      }
      int acc[6][16];
#pragma unroll
      for (int c = 0; c < 6; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[c][j] = 0;
      for (int s = 0; s < segs; ++s, ++seg) {
        if (!(ok = wait_warp(&d_full[seg & 1], seg >> 1, kErrD))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 6; ++c) {
          const int col = 32 * (2 * (c >> 1) + half) + 16 * (c & 1);
          if (col >= t.rows) continue;
          uint32_t v[16];
          tc_ld16(lanes + (seg & 1) * kBN + uint32_t(col), v);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c][j] += __float2int_rn(__uint_as_float(v[j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[seg & 1]);
      }
      // The half's four warps pass the barriers below together or not at all: one warp's wait may have been given up on (the CTA
      // aborts) where another's has just been met, and the others would wait for it there without a limit.
      if (t.splits == 1) ok = all_of_half(1 + half, ok);
      if (!ok) break;
      // 16 rows at a time through shared memory, so that a warp stores whole rows of the tile; with splits all rows stay there
      // (all of this CTA's MMAs are complete: the rows' ring is free).  Loops, not unrolled code: fetching instructions that are
      // run once took 7500 cycles for 32 rows.
#pragma unroll 1
      for (int c = 0; c < 6; ++c) {
        const int col = 32 * (2 * (c >> 1) + half) + 16 * (c & 1);
        if (col >= t.rows) break;   // the same for the half's four warps
        int *to = (t.splits > 1 ? reinterpret_cast<int *>(s_row) + col * kBM : s_stage + half * (16 * kBM)) + q * 32 + lane;
        float scale = sa[0];
#pragma unroll
        for (int k = 0; k < 6; ++k)
          if (k == c) {
            scale = sa[k >> 1];
#pragma unroll
            for (int j = 0; j < 16; ++j) to[j * kBM] = acc[k][j];
          }
        if (t.splits > 1) continue;
        asm volatile("bar.sync %0, 128;\n" ::"r"(1 + half) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = q + 4 * i;
          const float row_scale = __shfl_sync(0xffffffffu, scale, 16 * (c & 1) + j);
          if (col + j < count && ch < t.p.N)
            store_four(t.p, t.vector, tile.row0 + col + j, row_scale, ch,
                       *reinterpret_cast<const int4 *>(s_stage + half * (16 * kBM) + j * kBM + 4 * lane), f);
        }
        asm volatile("bar.sync %0, 128;\n" ::"r"(1 + half) : "memory");
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
    } else if (warp == kRelayWarp && lane == 0) {
      // ------------------------------------------------ rows landed -> ready
      // Up to three blocks' rows land ahead of the conversion: one is passed on only when the MMAs two blocks before are complete,
      // or it would count in that block's phase of the barrier.  Rows land again only after their block's MMAs, which wait
      // for this: no phase can be missed.
      uint32_t it = 0;
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step)
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          ok = wait(&rfull[it % kRowStages], it / kRowStages, kErrFull) &&
               (it < 2 || wait(&done[(it - 2) % kRowStages], (it - 2) / kRowStages, kErrFree));
          if (!ok) break;
          mbar_arrive(&ready[it % kGroups]);
        }
    } else if (warp == kMmaWarp && lane == 0) {
      // ------------------------------------------------ MMAs
      // One thread's path bounds the kernel, so its state is kept in registers: shared-memory addresses, stages and parities
      // that are stepped, not divided out.
      const uint32_t idesc = idesc_f16(0, kBM, t.rows);
      const uint32_t b_done = su32(done), b_ready = su32(ready), b_dfull = su32(d_full), b_dempty = su32(d_empty);
      const uint64_t rows0 = sw128_desc(su32(s_row));
      uint32_t s = 0, w = 0, w_par = 0, d = 0, d_par = 1;
      auto wait_at = [&](uint32_t b, uint32_t parity, int code) { return mbar_wait_at(b, parity, abort_flag, code, &g_linear8_error); };
      bool ok = true;
      for (int i = tile0; ok && i < tiles; i += step) {
        for (int left = nkb; ok && left > 0;) {
          const int n = min(left, kSegBlocks);
          if (!(ok = wait_at(b_dempty + 8 * d, d_par, kErrD))) break;
          const uint32_t acc = tmem + d * kBN;
          for (int kb = 0; kb < n; ++kb) {
            if (!(ok = wait_at(b_ready + 8 * w, w_par, kErrReady))) break;
            tc_fence_after();
            tc_mma_kblock_ts<kHalf / 16, false>(acc, tmem + kACol0 + w * kACols, rows0 + s * (kRowBytes / 16), idesc, uint32_t(kb));
            tc_commit_at(b_done + 8 * s);
            if (++s == kRowStages) s = 0;
            w_par ^= w;
            w ^= 1;
          }
          if (!ok) break;
          tc_commit_at(b_dfull + 8 * d);
          d_par ^= d;
          d ^= 1;
          left -= n;
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
    const int ch = tile.ch0 + 4 * lane, count = int(min(int64_t(t.rows), t.p.M - tile.row0));
    const uint32_t sums = su32(s_row) + 16 * lane;
    if (ch < t.p.N) {
      FourScales f;
      load_four(t.p, ch, f);
      for (int row = rank + t.splits * warp; row < count; row += t.splits * (kTcThreads / 32)) {
        const float sa = t.p.a_scale[tile.row0 + row];
        int4 v[kMaxSplits], acc = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) {
          v[r] = make_int4(0, 0, 0, 0);
          if (r < t.splits) {
            uint32_t from;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(from) : "r"(sums + 4 * kBM * row), "r"(r));
            asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v[r].x), "=r"(v[r].y), "=r"(v[r].z), "=r"(v[r].w) : "r"(from));
          }
        }
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) acc.x += v[r].x, acc.y += v[r].y, acc.z += v[r].z, acc.w += v[r].w;
        store_four(t.p, t.vector, tile.row0 + row, sa, ch, acc, f);
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
    const int64_t r = (i >> 32) == 0 ? int64_t(uint32_t(i) / uint32_t(per)) : i / per;
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

// Rows of a tile and CTAs of a cluster: the pair with the least time by these cycle counts, fitted to measured times: a K block
// 256 + 4 rows (shared memory) and at least 950 (the MMA thread), a tile's start and end 40 a row, the exchange of a cluster 1300, with
// four CTAs 16 a row more.  Times of the pairs (row tiles / CTAs), the choice first: 2048 x 2048, 192 rows 2/4 12.2 us, 3/2
// 12.3, 1/4 13.2, 1/1 19.6; 6144 x 2048, 192 rows 1/2 15.4, 3/1 16.8; 4096 x 4096, 300 rows 2/2 20.6, 4/1 25.4, 2/1 28.4;
// 4096 x 4096, 1024 rows 8/1 45.2, 6/1 50.0; 6144 x 4096, 1024 rows 6/1 50.4, 8/1 62.4.
void plan(TcArgs &t, int64_t M, int sms) {
  const int64_t least = cdiv(M, kBN), most = std::max(least, std::min<int64_t>(cdiv(M, 64), least + 6));
  double best = 1e30;
  for (int64_t n = least; n <= most; ++n) {
    const int rows = int(cdiv(cdiv(M, n), 16) * 16);
    const int64_t tiles = cdiv(M, rows) * t.channel_blocks;
    const double block = std::max(256.0 + 4 * rows, 950.0);
    for (int s = 1; s <= kMaxSplits; s *= 2) {
      if (s > 1 && tiles * s > sms) break;
      const int per = int(cdiv(t.blocks, s));
      if (cdiv(t.blocks, per) != s) continue;
      const double time = double(cdiv(tiles * s, sms)) * per * block + 40.0 * rows + (s > 1 ? 1300 : 0) + (s > 2 ? 16.0 * rows : 0);
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
  const size_t es = dtype_size(p.out_dtype);
  t.vector = p.out_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & (4 * es - 1)) == 0;
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
