// Key and value absorption on the 5th-generation tensor cores: per call, H small
// GEMMs, each of one head's weights against the whole batch.
//
//   absorb_q:  q'[b,h,0:512] = q_nope[b,h,:] W_UK[h]   ([B x 128] x [128 x 512]),
//              q'[b,h,512:576] = q_rope[b,h,:]
//   absorb_o:  out[b,h,:] = bf16(out_latent[b,h,:]) W_UV[h]   ([B x 512] x [512 x 128])
// (glossary entry, "why absorb in decode": q^C (W^UK)^T and (sum_t p_t c_t) W^UV.)
//
// Both are HBM-bound (about 1 GFLOP against tens of MB at the largest workload), so
// they are written for streaming.  A work item is one head and a tile of up to 128
// batch rows (the MMA's M; rows past the batch are zero-filled by TMA on load and
// clipped by TMA on store); CTAs are persistent over items, one per SM.  Roles:
// warps 0-3 own the 128 TMEM lanes (epilogue, and for absorb_o the fp32 -> bf16
// conversion of A), warp 4 issues TMA loads, warp 5 allocates TMEM and issues the
// MMAs.  The accumulator is double-buffered in TMEM, so one tile's epilogue runs
// under the next tile's MMAs.  Every wait is bounded: on expiry the kernel records
// MLA_ERR_DEVICE_TIMEOUT, lets in-flight copies and MMAs finish, frees TMEM and
// returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 192;
constexpr int kRows = 128;                // batch rows per item (MMA M)
constexpr int kBox = kRows * 128;         // one [128 rows x 128 B] 128B-swizzled TMA box: 16 KB

// ---------------------------------------------------------------- helpers
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

struct Guard {
  int* err;
  volatile int* abort;
  uint64_t limit_ns;
};

// Bounded wait on an mbarrier phase; false on timeout (recorded) or abort.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, const Guard& g) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*g.abort) return false;
      const uint64_t t = now_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > g.limit_ns) {
        set_device_error(g.err, MLA_ERR_DEVICE_TIMEOUT);
        *g.abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ void drain_on(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = now_ns();
  while (!mbar_try_wait(bar, parity) && now_ns() - t0 < limit_ns) {
  }
}

// Tiled store of one box from shared memory (coordinates are never negative here).
__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most one committed bulk group still reading shared memory.
__device__ __forceinline__ void bulk_wait_read_1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bar_sync_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// 32 fp32 -> 16-byte chunks [q4] of bf16 (8 values each).
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
  return make_uint4(pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                    pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                    pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                    pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7])));
}

// ================================================================ absorb_q
// Item (head h, batch tile mt): A = q_nope[128 rows x 128 k] (two K-major boxes), then
// four n-tiles of 128: B = W_UK[h][128 k x 128 n] (two MN-major boxes), D = 128 x 128
// fp32 in TMEM, written out as bf16 through shared memory by TMA stores.
constexpr int kQA = 2 * kBox, kQB = 2 * kBox, kQO = 2 * kBox;  // 32 KB each
constexpr int kQBStages = 4;             // every n-tile of an item's weights in flight at once
constexpr int kQSmA = 0, kQSmB = kQA, kQSmO = kQSmB + kQBStages * kQB;
constexpr int kQSmem = kQSmO + 2 * kQO;  // 224 KB: A, B[4], out[2]
constexpr int kQNt = kDLatent / 128;     // n-tiles per item
constexpr uint32_t kQIdesc = idesc_bf16_f32(128, 128, 0, 1);

enum QBar { kQAFull = 0, kQAEmpty, kQBFull, kQBEmpty = kQBFull + kQBStages, kQDFull = kQBEmpty + kQBStages, kQDEmpty = kQDFull + 2, kQDone = kQDEmpty + 2, kQNumBars };

__global__ void __launch_bounds__(kThreads, 1)
    absorb_q_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_o, const __nv_bfloat16* __restrict__ q_rope,
                       __nv_bfloat16* __restrict__ q_out, int B, int H, int* err, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kQNumBars];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mtiles = (B + kRows - 1) / kRows;
  const int items = H * mtiles;

  if (tid == 0) {
    abort_s = 0;
    mbar_init(bar(kQAFull), 1);
    mbar_init(bar(kQAEmpty), 1);
    for (int i = 0; i < kQBStages; ++i) {
      mbar_init(bar(kQBFull + i), 1);
      mbar_init(bar(kQBEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kQDFull + i), 1);
      mbar_init(bar(kQDEmpty + i), 4);  // one arrival per epilogue warp
    }
    mbar_init(bar(kQDone), 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_o);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&tmem_s), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Launched as a programmatic dependent: the set-up above overlaps the previous grid,
  // whose writes (the inputs) are complete and visible after this wait.
  if (tid == 0) grid_dep_launch_dependents();
  grid_dep_wait();
  const uint32_t tmem = tmem_s;
  const Guard gd{err, &abort_s, limit_ns};

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      int it = 0, g = 0, ga = 0, gb = 0;  // items, n-tiles; loads issued into A and B
      bool ok = true;
      for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++it) {
        const int h = item % H, b0 = (item / H) * kRows;
        if (!wait_on(bar(kQAEmpty), (it & 1) ^ 1, gd)) { ok = false; break; }
        mbar_expect_tx(bar(kQAFull), kQA);
        tma_load_3d(sbase + kQSmA, &map_a, 0, h, b0, bar(kQAFull));
        tma_load_3d(sbase + kQSmA + kBox, &map_a, 64, h, b0, bar(kQAFull));
        ++ga;
        for (int j = 0; j < kQNt; ++j, ++g) {
          const int s = g % kQBStages;
          if (!wait_on(bar(kQBEmpty + s), ((g / kQBStages) & 1) ^ 1, gd)) { ok = false; break; }
          mbar_expect_tx(bar(kQBFull + s), kQB);
          tma_load_3d(sbase + kQSmB + s * kQB, &map_b, 128 * j, 0, h, bar(kQBFull + s));
          tma_load_3d(sbase + kQSmB + s * kQB + kBox, &map_b, 128 * j + 64, 0, h, bar(kQBFull + s));
          ++gb;
        }
      }
      // Every load issued lands before the CTA may exit (bounded).
      if (ga > 0) drain_on(bar(kQAFull), (ga - 1) & 1, limit_ns);
      for (int k = 0; k < kQBStages && k < gb; ++k) {
        const int l = gb - 1 - k;
        drain_on(bar(kQBFull + l % kQBStages), (l / kQBStages) & 1, limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      int it = 0, g = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++it) {
        if (!wait_on(bar(kQAFull), it & 1, gd)) { ok = false; break; }
        for (int j = 0; j < kQNt; ++j, ++g) {
          const int s = g % kQBStages, d = g & 1;
          if (!wait_on(bar(kQBFull + s), (g / kQBStages) & 1, gd) ||
              !wait_on(bar(kQDEmpty + d), ((g >> 1) & 1) ^ 1, gd)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ab = sbase + kQSmA, bb = sbase + kQSmB + s * kQB;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem + d * 128, desc_sw128(ab + (kk >> 2) * kBox + (kk & 3) * 32, 16, 1024),
                   desc_sw128(bb + kk * 2048, kBox, 1024), kQIdesc, kk > 0 ? 1u : 0u);
          mma_commit(bar(kQBEmpty + s));
          mma_commit(bar(kQDFull + d));
        }
        if (!ok) break;
        mma_commit(bar(kQAEmpty));
      }
      mma_commit(bar(kQDone));
      drain_on(bar(kQDone), 0, limit_ns);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue: thread = batch row
    // The four warps meet at named barriers, so none of them leaves the loops early:
    // after a failed wait they keep the same barrier sequence and skip the work.
    const int r = 32 * warp + lane;
    const uint32_t t_row = tmem + ((uint32_t)(32 * warp) << 16);
    int it = 0, g = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
      const int h = item % H, b0 = (item / H) * kRows;
      const int b = b0 + r;
      if (ok && b < B) {  // the rope half of q' is a copy
        const uint4* src = reinterpret_cast<const uint4*>(q_rope + ((size_t)b * H + h) * kDRope);
        uint4* dst = reinterpret_cast<uint4*>(q_out + ((size_t)b * H + h) * kDQK + kDLatent);
#pragma unroll
        for (int c = 0; c < 8; ++c) dst[c] = src[c];
      }
      for (int j = 0; j < kQNt; ++j, ++g) {
        const int d = g & 1;
        if (ok) ok = __all_sync(0xffffffffu, wait_on(bar(kQDFull + d), (g >> 1) & 1, gd));
        tc_fence_after();
        // Output buffer d was last stored from two n-tiles ago: that store has read it.
        if (tid == 0) bulk_wait_read_1();
        bar_sync_epilogue();
        if (ok) {
          uint8_t* ob = smem + kQSmO + d * kQO;
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 32 columns at a time
            uint32_t v[32];
            tmem_ld32(t_row + d * 128 + 32 * c, v);
            tmem_wait_ld();
            uint8_t* row = ob + (c >> 1) * kBox + r * 128;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const int chunk = (c & 1) * 4 + q4;
              *reinterpret_cast<uint4*>(row + ((chunk ^ (r & 7)) * 16)) = pack8(v + 8 * q4);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kQDEmpty + d));
          fence_proxy_async();
        }
        // Every epilogue warp agrees on ok here: a warp that failed set the abort flag,
        // and the store below is issued only if all four wrote their rows.
        bar_sync_epilogue();
        if (tid == 0 && !abort_s) {
          tma_store_3d(&map_o, sbase + kQSmO + d * kQO, 128 * j, h, b0);
          tma_store_3d(&map_o, sbase + kQSmO + d * kQO + kBox, 128 * j + 64, h, b0);
          bulk_commit();
        }
      }
    }
    if (tid == 0) bulk_wait_all();  // every store has completed before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ================================================================ absorb_o
// Item (head h, batch tile mt): K = 512 in eight chunks of 64.  Per chunk, TMA brings
// the fp32 out_latent rows [128 x 64] (two 128B-swizzled boxes of 32 floats) and the
// weights W_UV[h][64 k x 128 n] (two MN-major boxes); four converter warps round the
// fp32 rows to bf16 (nearest even) into the K-major A operand; the MMA warp adds the
// chunk's four K = 16 steps into D = 128 x 128 fp32 in TMEM.  The epilogue writes D
// through shared memory by TMA stores.  Warps 0-3 epilogue, 4-7 convert, 8 TMA, 9 MMA.
constexpr int kOThreads = 320;
constexpr int kOF = 2 * kBox, kOA = kBox, kOB = kBox, kOO = 4 * kBox;  // 32, 16, 16, 64 KB
constexpr int kOFStages = 2, kOStages = 3;
constexpr int kOSmF = 0, kOSmA = kOFStages * kOF, kOSmB = kOSmA + kOStages * kOA, kOSmO = kOSmB + kOStages * kOB;
constexpr int kOSmem = kOSmO + kOO;  // 224 KB
constexpr int kOChunks = kDLatent / 64;
constexpr uint32_t kOIdesc = idesc_bf16_f32(128, 128, 0, 1);

enum OBar {
  kOFFull = 0,
  kOFEmpty = kOFFull + kOFStages,
  kOBFull = kOFEmpty + kOFStages,
  kOABEmpty = kOBFull + kOStages,  // MMA done with A and B of a stage
  kOAReady = kOABEmpty + kOStages,
  kODFull = kOAReady + kOStages,
  kODEmpty = kODFull + 2,
  kODone = kODEmpty + 2,
  kONumBars
};

__global__ void __launch_bounds__(kOThreads, 1)
    absorb_o_tc_kernel(const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_o, int B, int H, int* err, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kONumBars];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = H * ((B + kRows - 1) / kRows);

  if (tid == 0) {
    abort_s = 0;
    for (int i = 0; i < kOFStages; ++i) {
      mbar_init(bar(kOFFull + i), 1);
      mbar_init(bar(kOFEmpty + i), 4);  // one arrival per converter warp
    }
    for (int i = 0; i < kOStages; ++i) {
      mbar_init(bar(kOBFull + i), 1);
      mbar_init(bar(kOABEmpty + i), 1);
      mbar_init(bar(kOAReady + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kODFull + i), 1);
      mbar_init(bar(kODEmpty + i), 4);
    }
    mbar_init(bar(kODone), 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_f);
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_o);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&tmem_s), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) grid_dep_launch_dependents();
  grid_dep_wait();  // as in absorb_q: the inputs are complete from here on
  const uint32_t tmem = tmem_s;
  const Guard gd{err, &abort_s, limit_ns};

  if (warp == 8) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      int gf = 0, gb = 0;  // fp32 A and weight chunks issued
      bool ok = true;
      for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
        const int h = item % H, b0 = (item / H) * kRows;
        for (int c = 0; c < kOChunks; ++c) {
          const int f = gf % kOFStages, s = gb % kOStages;
          if (!wait_on(bar(kOFEmpty + f), ((gf / kOFStages) & 1) ^ 1, gd)) { ok = false; break; }
          mbar_expect_tx(bar(kOFFull + f), kOF);
          tma_load_3d(sbase + kOSmF + f * kOF, &map_f, 64 * c, h, b0, bar(kOFFull + f));
          tma_load_3d(sbase + kOSmF + f * kOF + kBox, &map_f, 64 * c + 32, h, b0, bar(kOFFull + f));
          ++gf;
          if (!wait_on(bar(kOABEmpty + s), ((gb / kOStages) & 1) ^ 1, gd)) { ok = false; break; }
          mbar_expect_tx(bar(kOBFull + s), kOB);
          tma_load_3d(sbase + kOSmB + s * kOB, &map_w, 0, 64 * c, h, bar(kOBFull + s));
          tma_load_3d(sbase + kOSmB + s * kOB + kBox / 2, &map_w, 64, 64 * c, h, bar(kOBFull + s));
          ++gb;
        }
      }
      // Every load issued lands before the CTA may exit (bounded).
      for (int k = 0; k < kOFStages && k < gf; ++k) {
        const int l = gf - 1 - k;
        drain_on(bar(kOFFull + l % kOFStages), (l / kOFStages) & 1, limit_ns);
      }
      for (int k = 0; k < kOStages && k < gb; ++k) {
        const int l = gb - 1 - k;
        drain_on(bar(kOBFull + l % kOStages), (l / kOStages) & 1, limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      int it = 0, g = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++it) {
        const int d = it & 1;
        if (!wait_on(bar(kODEmpty + d), ((it >> 1) & 1) ^ 1, gd)) { ok = false; break; }
        for (int c = 0; c < kOChunks; ++c, ++g) {
          const int s = g % kOStages;
          if (!wait_on(bar(kOAReady + s), (g / kOStages) & 1, gd) || !wait_on(bar(kOBFull + s), (g / kOStages) & 1, gd)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ab = sbase + kOSmA + s * kOA, bb = sbase + kOSmB + s * kOB;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(tmem + d * 128, desc_sw128(ab + kk * 32, 16, 1024), desc_sw128(bb + kk * 2048, kBox / 2, 1024),
                   kOIdesc, (c > 0 || kk > 0) ? 1u : 0u);
          mma_commit(bar(kOABEmpty + s));
        }
        if (!ok) break;
        mma_commit(bar(kODFull + d));
      }
      mma_commit(bar(kODone));
      drain_on(bar(kODone), 0, limit_ns);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- fp32 -> bf16 A: thread = batch row
    const int r = tid - 128;
    int g = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
      for (int c = 0; c < kOChunks; ++c, ++g) {
        const int f = g % kOFStages, s = g % kOStages;
        if (!__all_sync(0xffffffffu, wait_on(bar(kOFFull + f), (g / kOFStages) & 1, gd) &&
                                         wait_on(bar(kOABEmpty + s), ((g / kOStages) & 1) ^ 1, gd))) {
          ok = false;
          break;
        }
        const uint8_t* frow = smem + kOSmF + f * kOF + r * 128;
        uint8_t* arow = smem + kOSmA + s * kOA + r * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // bf16 chunk q: k 8q..8q+7 = fp32 box q/4, chunks 2(q%4), 2(q%4)+1
          const uint8_t* fb = frow + (q >> 2) * kBox;
          const int c0 = 2 * (q & 3);
          const float4 x = *reinterpret_cast<const float4*>(fb + ((c0 ^ (r & 7)) * 16));
          const float4 y = *reinterpret_cast<const float4*>(fb + (((c0 + 1) ^ (r & 7)) * 16));
          *reinterpret_cast<uint4*>(arow + ((q ^ (r & 7)) * 16)) =
              make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kOFEmpty + f));
          mbar_arrive(bar(kOAReady + s));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue: thread = batch row
    // As in absorb_q, the four warps keep the same named-barrier sequence after a failure.
    const int r = 32 * warp + lane;
    const uint32_t t_row = tmem + ((uint32_t)(32 * warp) << 16);
    int it = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
      const int h = item % H, b0 = (item / H) * kRows;
      const int d = it & 1;
      if (ok) ok = __all_sync(0xffffffffu, wait_on(bar(kODFull + d), (it >> 1) & 1, gd));
      tc_fence_after();
      if (tid == 0) bulk_wait_all();  // the previous item's store has finished with the buffer
      bar_sync_epilogue();
      if (ok) {
        uint8_t* row = smem + kOSmO + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 32 columns = one box
          uint32_t v[32];
          tmem_ld32(t_row + d * 128 + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(row + c * kBox + ((q ^ (r & 7)) * 16)) =
                make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kODEmpty + d));
        fence_proxy_async();
      }
      bar_sync_epilogue();
      if (tid == 0 && !abort_s) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_store_3d(&map_o, sbase + kOSmO + c * kBox, 32 * c, h, b0);
        bulk_commit();
      }
    }
    if (tid == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ================================================================ absorb_o of a bf16 latent
// out[b,h,:] = x[b,h,:] W_UV[h] with x already bf16 (the window and shared-prefix decodes'
// output), taken transposed: D = out^T[128 v x N rows], A = W_UV[h]^T (MN-major boxes of
// [64 k x 64 v]), B = x (K-major, N batch rows).  Bound by HBM (W_UV and x once): with the
// batch as N, a short batch costs no padding, and chunks of 256 k (128 where the rows of x
// need the room) run through one ring across items, so one item's loads fly under the
// previous one's MMAs and stores.  A chunk is two TMA boxes, one of W_UV and one of x: a
// thread issues a box in 250 to 480 cycles whatever its size, and in boxes of 64 x 64 the
// calls took 4.7, 4.9 and 8.1 us for 5 x 16, 64 x 16 and 64 x 128 rows x heads, against 2.9,
// 3.5 and 7.4 (operands not in L2).  An item is a head, a tile of N batch rows (16 to 128)
// and, when there are too few heads to give every SM one, one half of the 128 v dims (kHalf:
// M = 64).
constexpr int kXThreads = 192;
constexpr int kXW = 16384;           // 64 k x 128 v of W_UV
constexpr int kXMaxStages = 5;
constexpr int kXSmem = 229376;
constexpr int kXBlocks = kDLatent / 64;
enum XBar { kXFull = 0, kXEmpty = kXFull + kXMaxStages, kXDFull = kXEmpty + kXMaxStages, kXDEmpty = kXDFull + 2, kXDone = kXDEmpty + 2, kXNumBars };

template <bool kHalf>
__global__ void __launch_bounds__(kXThreads, 1)
    absorb_o_bf16_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                         float* __restrict__ out, int B, int H, int N, int kc, int stages, int* err, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kXNumBars];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kParts = kHalf ? 2 : 1, kM = 128 / kParts;
  constexpr int kWBytes = kXW / kParts;
  const int stage_bytes = kc * (kWBytes + N * 128);  // kc blocks of 64 k
  const int items = H * kParts * ((B + N - 1) / N);

  if (tid == 0) {
    abort_s = 0;
    for (int i = 0; i < stages; ++i) {
      mbar_init(bar(kXFull + i), 1);
      mbar_init(bar(kXEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kXDFull + i), 1);
      mbar_init(bar(kXDEmpty + i), 4);
    }
    mbar_init(bar(kXDone), 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_s), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) grid_dep_launch_dependents();
  grid_dep_wait();
  const uint32_t tmem = tmem_s;
  const Guard gd{err, &abort_s, limit_ns};

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
        const int hp = item % (H * kParts), h = hp / kParts, v0 = kM * (hp % kParts), b0 = (item / (H * kParts)) * N;
        for (int c = 0; c < kXBlocks; c += kc) {
          if (!wait_on(bar(kXEmpty + s), phase ^ 1, gd)) { ok = false; break; }
          const uint32_t st = sbase + s * stage_bytes;
          mbar_expect_tx(bar(kXFull + s), stage_bytes);
          tma_load_4d(st, &map_w, 0, 64 * c, v0 / 64, h, bar(kXFull + s));
          tma_load_4d(st + kc * kWBytes, &map_x, 0, b0, c, h, bar(kXFull + s));
          ++issued;
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // Every load issued lands before the CTA may exit (bounded).
      for (int k = 1; k <= stages && k <= issued; ++k) {
        const int l = issued - k;
        drain_on(bar(kXFull + l % stages), (l / stages) & 1, limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    const uint32_t idesc = idesc_bf16_f32(kM, N, 1, 0);
    // W_UV: the two 64-v halves of a chunk lie kc blocks apart.
    constexpr uint64_t kKMajor = desc_sw128_const(16, 1024);
    const uint64_t mn_major = desc_sw128(0, kc * 8192, 1024);
    int s = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++it) {
      const int d = it & 1;
      ok = __all_sync(0xffffffffu, wait_on(bar(kXDEmpty + d), ((it >> 1) & 1) ^ 1, gd));
      for (int c = 0; ok && c < kXBlocks; c += kc) {
        ok = __all_sync(0xffffffffu, wait_on(bar(kXFull + s), phase, gd));
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = sbase + s * stage_bytes;
        for (int j = 0; j < kc; ++j)
          mma_x4_elect<128, 2>(tmem + d * 128, mn_major | desc_addr(st + j * 8192),
                               kKMajor | desc_addr(st + kc * kWBytes + j * N * 128), idesc, c + j > 0);
        mma_commit_elect(bar(kXEmpty + s));
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (ok) mma_commit_elect(bar(kXDFull + d));
    }
    mma_commit_elect(bar(kXDone));
    drain_on(bar(kXDone), 0, limit_ns);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue: lane = v
    // D's rows sit in lanes 0-127, or, for M = 64, in the lower 16 lanes of each quadrant.
    const int q = warp & 3;
    const int v = kHalf ? 16 * q + (lane & 15) : 32 * q + lane;
    const bool live = !kHalf || lane < 16;
    const uint32_t t_row = tmem + ((uint32_t)(32 * q) << 16);
    int it = 0;
    bool ok = true;  // no wait ran out: the outputs of this CTA's remaining items are NaN then
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
      const int hp = item % (H * kParts), h = hp / kParts, v0 = kM * (hp % kParts), b0 = (item / (H * kParts)) * N;
      const int d = it & 1;
      ok = ok && __all_sync(0xffffffffu, wait_on(bar(kXDFull + d), (it >> 1) & 1, gd));
      tc_fence_after();
      float* dst = out + ((size_t)b0 * H + h) * MLA_D_V + v0 + v;
      const int rows = min(N, B - b0);
      for (int c = 0; c < rows; c += 16) {
        uint32_t r[16];
        tmem_ld16(t_row + d * 128 + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (live && c + e < rows) dst[(size_t)(c + e) * H * MLA_D_V] = ok ? __uint_as_float(r[e]) : NAN;
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar(kXDEmpty + d));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// 3-D tiled map: dims innermost first (elements), strides of dims 1 and 2 in bytes.
bool map3d(CUtensorMap* m, CUtensorMapDataType t, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
           uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1, uint32_t b2, CUtensorMapSwizzle sw) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {s1, s2};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, t, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch as a programmatic dependent of the previous grid on the stream.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem, cudaStream_t stream,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int sm_count() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 1;
  }
  return n;
}

}  // namespace

cudaError_t launch_absorb_q(const __nv_bfloat16* q_nope, const __nv_bfloat16* q_rope, const __nv_bfloat16* w_uk,
                            __nv_bfloat16* q_out, int batch, int heads, int* err, cudaStream_t stream) {
  CUtensorMap ma, mb, mo;
  const uint64_t H = heads, Bn = batch;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!map3d(&ma, bf, q_nope, MLA_D_NOPE, H, Bn, MLA_D_NOPE * 2, H * MLA_D_NOPE * 2, 64, 1, kRows, sw) ||
      !map3d(&mb, bf, w_uk, kDLatent, MLA_D_NOPE, H, kDLatent * 2, (uint64_t)MLA_D_NOPE * kDLatent * 2, 64,
             MLA_D_NOPE, 1, sw) ||
      !map3d(&mo, bf, q_out, kDQK, H, Bn, kDQK * 2, H * kDQK * 2, 64, 1, kRows, sw))
    return cudaErrorInvalidValue;
  const int smem = kQSmem + 1024;
  static bool done[64] = {};
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(absorb_q_tc_kernel), smem, done);
  if (e != cudaSuccess) return e;
  const int items = heads * ((batch + kRows - 1) / kRows);
  const int grid = items < sm_count() ? items : sm_count();
  return launch_dependent(absorb_q_tc_kernel, grid, kThreads, smem, stream, ma, mb, mo, q_rope, q_out, batch, heads,
                          err, 2000ull * 1000000ull);
}

cudaError_t launch_absorb_o(const float* out_latent, const __nv_bfloat16* w_uv, float* out, int batch, int heads,
                            int* err, cudaStream_t stream) {
  CUtensorMap mf, mw, mo;
  const uint64_t H = heads, Bn = batch;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!map3d(&mf, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out_latent, kDLatent, H, Bn, kDLatent * 4, H * kDLatent * 4, 32, 1,
             kRows, sw) ||
      !map3d(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w_uv, MLA_D_V, kDLatent, H, MLA_D_V * 2,
             (uint64_t)kDLatent * MLA_D_V * 2, 64, 64, 1, sw) ||
      !map3d(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out, MLA_D_V, H, Bn, MLA_D_V * 4, H * MLA_D_V * 4, 32, 1, kRows, sw))
    return cudaErrorInvalidValue;
  const int smem = kOSmem + 1024;
  static bool done[64] = {};
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(absorb_o_tc_kernel), smem, done);
  if (e != cudaSuccess) return e;
  const int items = heads * ((batch + kRows - 1) / kRows);
  const int grid = items < sm_count() ? items : sm_count();
  return launch_dependent(absorb_o_tc_kernel, grid, kOThreads, smem, stream, mf, mw, mo, batch, heads, err,
                          2000ull * 1000000ull);
}

template <bool kHalf>
static cudaError_t launch_absorb_o_bf16_as(const CUtensorMap& mx, const CUtensorMap& mw, float* out, int batch, int heads,
                                           int rows, int kc, int* err, cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(absorb_o_bf16_kernel<kHalf>), kXSmem + 1024, done);
  if (e != cudaSuccess) return e;
  const int parts = kHalf ? 2 : 1;
  const int items = heads * parts * ((batch + rows - 1) / rows);
  const int stage = kc * (kXW / parts + rows * 128), fit = kXSmem / stage, stages = fit < kXMaxStages ? fit : kXMaxStages;
  return launch_dependent(absorb_o_bf16_kernel<kHalf>, items < sm_count() ? items : sm_count(), kXThreads, kXSmem + 1024,
                          stream, mx, mw, out, batch, heads, rows, kc, stages, err, 2000ull * 1000000ull);
}

cudaError_t launch_absorb_o_bf16(const __nv_bfloat16* out_latent, const __nv_bfloat16* w_uv, float* out, int batch,
                                 int heads, int* err, cudaStream_t stream) {
  CUtensorMap mx, mw;
  const uint64_t H = heads, Bn = batch;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int rows = batch <= 16 ? 16 : batch <= 32 ? 32 : batch <= 64 ? 64 : 128;
  // Half items when even they leave SMs without one: the loads of an item (128 KB of W_UV)
  // are then shared by two SMs.
  const int items = heads * ((batch + rows - 1) / rows);
  const bool half = 2 * items <= sm_count();
  // The longest chunk of which two fit.
  const int kc = 2 * 4 * ((half ? kXW / 2 : kXW) + rows * 128) <= kXSmem ? 4 : 2;
  // x as [8 blocks of 64 k][batch][64 k] of a head, W_UV as [2 halves of 64 v][512 k][64 v].
  const auto enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  auto map4d = [&](CUtensorMap* m, const __nv_bfloat16* p, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                   const cuuint32_t (&box)[4]) {
    return enc(m, bf, 4, const_cast<__nv_bfloat16*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map4d(&mx, out_latent, {64, Bn, 8, H}, {H * kDLatent * 2, 128, kDLatent * 2}, {64, (cuuint32_t)rows, (cuuint32_t)kc, 1}) ||
      !map4d(&mw, w_uv, {64, kDLatent, 2, H}, {MLA_D_V * 2, 128, (cuuint64_t)kDLatent * MLA_D_V * 2},
             {64, 64 * (cuuint32_t)kc, half ? 1u : 2u, 1}))
    return cudaErrorInvalidValue;
  return half ? launch_absorb_o_bf16_as<true>(mx, mw, out, batch, heads, rows, kc, err, stream)
              : launch_absorb_o_bf16_as<false>(mx, mw, out, batch, heads, rows, kc, err, stream);
}

}  // namespace mla
