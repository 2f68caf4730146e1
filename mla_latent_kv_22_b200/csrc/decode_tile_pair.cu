// Window and shared-prefix decode of row tiles above 64 rows: a CTA pair (a 2-CTA cluster)
// per worker, 128 query rows, two 64-token pages per step, all products pair-wide MMAs
// issued by CTA 0 with M = 128 rows, 64 in each CTA:
//     S[128 x 128]  = q'[128 x 576] . K^T   CTA r supplies page r of the step, all dims
//     O[128 x 512] += P[128 x 128] . V      two MMAs of N = 256 dims; CTA r supplies dims
//                                           [256r + 128j, +128) of both pages for MMA j
// A tile of 64 rows on one CTA was bound by shared-memory bandwidth: its M = 64 products read
// 4 KB for 32 cycles and 6 KB for 48 cycles of tensor work (32.2 and 48.2 cycles a MMA, 128
// bytes a cycle), ~3,500 cycles per 64 rows x 64 tokens with the loads on top.  The pair's
// products take 1,088 cycles for the same work (32.2 and 64.2 cycles a MMA), read 2 KB (4 KB
// where q' is in shared memory) per 32 cycles and 5 KB per 64 (P is taken from the collector
// the second time), and a page's rows serve twice as many queries: a step takes 2,400 to 2,800
// cycles of 2,176 of tensor work (at the 1.5 to 1.8 GHz that the power limit leaves under this
// load; 1.4 to 1.6 us).  Each CTA keeps the scores and outputs of its own rows, so the softmax
// needs nothing from the peer.  The value half that a CTA supplies is loaded apart from its
// score page (1.8 times the page's bytes, the second time from L2).
//
// Tensor memory (pair-wide M = 128: lane l < 64 holds row 64r + l and the first half of the
// N columns, lane l >= 64 row 64r + l - 64 and the second):
//   [0, 256)    O: block j, dims 128j.. in lanes 0-63 and 256 + 128j.. in lanes 64-127
//   [256, 320)  S of a step: page 0's tokens in lanes 0-63, page 1's in lanes 64-127
//   [320, 512)  q' dims [0, 384) as the A operand (each row in lanes h and h + 64)
// Shared memory per CTA: q' dims [384, 576) (24 KB), P (2 boxes [64 rows x 64 tokens]), two
// rope slots, three score slots (a half page, 256 dims) and two value slots (256 dims of a
// page), each filled by one TMA box of four 64-dim blocks.  Scores and values have rings of
// their own: a score slot is free as soon as its MMAs are done, 2,176 tensor cycles before
// the half that takes it over is needed; a value slot 1,664.  Few large boxes matter: one
// thread issues a box in 250 to 480 cycles whatever its size (measured, L2-resident pages:
// 16.5, 33 and 65 bytes a cycle and SM with boxes of 8, 16 and 32 KB).
//
// One buffer each for S and P is enough: while the softmax of step i runs, the tensor cores
// take the values of step i - 1 and the scores of step i + 1.
//
// Roles (384 threads; a 13th warp would leave 128 registers a thread, and the spills' traffic
// shares the path that bounds the products).  Warps 0-7: softmax, 4 threads per row (32 tokens
// each), and the epilogue.  Warp 8: q' and score loads.  Warp 9: score MMAs (CTA 0).  Warp 10:
// value loads, and zeroes their rows that no query sees.  Warp 11: tensor memory, value MMAs
// (CTA 0).  (The first warps also write the schedule's records, which the loads should not
// wait for.)
// The lazy running maximum, the roundings and the bounded waits are decode_tile.cu's.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "tile_tasks.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kRows = 128;
constexpr int kThreads = 384;
constexpr int kLoadK = 8, kScores = 9, kLoadV = 10, kValues = 11;  // warps; 0-7 are the softmax's
constexpr int kBox = 8192;            // [64 rows x 64 bf16], 128B swizzle
constexpr int kSlotBytes = 4 * kBox;  // a half page
constexpr int kKSlots = 3;
constexpr int kQTmemBoxes = 6, kQSmemBoxes = 3;
constexpr int kOffQ = 0;
constexpr int kOffP = kOffQ + kQSmemBoxes * kBox;
constexpr int kOffRope = kOffP + 2 * kBox;
constexpr int kOffK = kOffRope + 2 * kBox;
constexpr int kOffV = kOffK + kKSlots * kSlotBytes;
constexpr int kBytes = kOffV + 2 * kSlotBytes;
constexpr int kAlloc = kBytes + 1024;  // + alignment slack
static_assert(kAlloc + 5120 <= 232448, "dynamic + static shared memory above the per-CTA limit");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
static_assert(kColQ + 32 * kQTmemBoxes <= kTmemCols, "tensor-memory regions overlap");
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);  // A q' K-major, B rows K-major
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 256, 0, 1);  // A P K-major, B rows MN-major
constexpr uint16_t kBothCtas = 3;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

enum Bar {
  kFullK = 0,                  // [slot] CTA 0: both CTAs' halves landed
  kEmptyK = kFullK + kKSlots,  // [slot] both: the score MMAs have read it
  kFullV = kEmptyK + kKSlots,  // [page] CTA 0: both CTAs' values landed (and, if dirty, were cleaned)
  kEmptyV = kFullV + 2,        // [page] both: the value MMAs have read it
  kDirty = kEmptyV + 2,        // [page] own: values with unseen rows landed
  kQFull = kDirty + 2,         // CTA 0: q' of both CTAs landed in shared memory
  kQStage,                     // own: the rest of q' landed in two score slots
  kQReady,                     // CTA 0: the 16 softmax warps copied it to tensor memory
  kQEmpty,                     // both: the piece's last score MMA has read q'
  kSFull,                      // both: a step's scores are in S (and its rope slot is free)
  kSFree,                      // CTA 0: the 16 softmax warps have read them
  kPFull,                      // CTA 0: the 16 softmax warps wrote P (and rescaled O)
  kODone,                      // both: the value MMAs of a step are done
  kOFree,                      // CTA 0: the 16 softmax warps read O in the epilogue
  kGroup,                      // [2] the 4 softmax warps that share rows met
  kDrain = kGroup + 2,         // [2] either issuing warp's MMAs are all done
  kNumBars = kDrain + 2
};

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// What a wait needs besides its barrier, in shared memory: few registers across the kernel.
struct Ctl {
  int* err;
  uint64_t limit_ns;
  int abort;
  uint32_t peer_abort;  // the peer's abort flag (cluster address)
};

// Bounded wait on an mbarrier phase; false on timeout (recorded) or abort.  The first try is
// inlined, the rest is not (it would be at some thirty places).  CTA-scope acquire, since what
// crosses the pair is read by the tensor cores alone; kCluster: but for drop_s, whose words the
// peer's warps set and the value MMAs' warp reads.
template <bool kCluster>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  return kCluster ? mbar_try_wait(bar, parity) : mbar_try_wait_cta(bar, parity);
}
template <bool kCluster>
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, Ctl* c) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (phase_done<kCluster>(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*const_cast<volatile int*>(&c->abort)) return false;
      const uint64_t t = now_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > c->limit_ns) {
        set_device_error(c->err, MLA_ERR_DEVICE_TIMEOUT);
        *const_cast<volatile int*>(&c->abort) = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(c->peer_abort), "r"(1) : "memory");
        return false;
      }
    }
  }
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, Ctl* c) {
  return __all_sync(0xffffffffu, phase_done<kCluster>(bar, parity) || wait_long<kCluster>(bar, parity, c));
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = now_ns();
  while (!mbar_try_wait(bar, parity) && now_ns() - t0 < limit_ns) {
  }
}

// Arrive on a barrier of CTA 0.
__device__ __forceinline__ void arrive_cta0(uint32_t rank, uint32_t local_bar, uint32_t cluster_bar) {
  if (rank == 0) mbar_arrive(local_bar);
  else mbar_arrive_remote(cluster_bar);
}

// A warp's 128 dims of its 32 rows leave through its own part of the P buffer (64 bytes of
// 32 rows, the c-th half of each), 16 rows of 128 bytes at a time: 8 lanes then store 128
// contiguous bytes of one row.  `inv` is this lane's row's factor; `dst` is row 0 of the
// warp's 32, `live` how many of them are stored.
template <bool kDirect>
__device__ __forceinline__ void store_rows(uint32_t taddr, float inv, uint8_t* box, int c, int r32, int lane, int live, void* dst) {
  constexpr int kCols = kDirect ? 64 : 32;  // 128 bytes
  // The place of chunk e of staged row r: neither side meets a bank twice.
  auto cell = [&](int r, int e) -> uint4* {
    const int x = e ^ (r & 4), rr = (r & 3) | (x & 4) | ((r >> 2) << 3);
    return reinterpret_cast<uint4*>(box + (r32 + rr) * 128 + (((4 * c + (x & 3)) ^ (rr & 7)) * 16));
  };
#pragma unroll 1
  for (int cc = 0; cc < 128; cc += kCols) {
    uint32_t w[32];
    if constexpr (kDirect) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t r[32];
        tmem_ld32(taddr + cc + 32 * j, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[16 * j + e] = pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
      }
    } else {
      tmem_ld32(taddr + cc, w);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * inv);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (lane >> 4 == half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) *cell(lane & 15, e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 3), row = 16 * half + r;
        const uint4 v = *cell(r, lane & 7);
        if (row < live)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + ((size_t)row * kDLatent + cc) * (kDirect ? 2 : 4) + (lane & 7) * 16) = v;
      }
      __syncwarp();  // the staging area is rewritten by the next rows
    }
  }
}

// Zeroes the values that are not finite of a step's tokens, in both CTAs: bit j of lane w's
// word is token 32 w + j, in the four boxes of slot w / 2.  By a whole warp of CTA 0, with the
// values landed.
__device__ __noinline__ void drop_values(uint32_t v, uint32_t word, int lane) {
#pragma unroll 1
  for (int t = 0; t < 128; ++t) {
    if (!((__shfl_sync(0xffffffffu, word, t >> 5) >> (t & 31)) & 1u)) continue;
    // Four boxes of 128 bytes: 32 chunks of 16, one per lane and CTA.
    const uint32_t at = v + (t >> 6) * kSlotBytes + (lane >> 3) * kBox + (t & 63) * 128 + (lane & 7) * 16;
#pragma unroll 1
    for (int r = 0; r < 2; ++r) {
      const uint32_t ca = map_to_rank(at, r);
      uint4 x;
      asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(ca) : "memory");
      x = finite_chunk(x);
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ca), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  __syncwarp();
}

// kMixed: mixed_pages(a).   A copy of its own: the check costs up to 6% where it is not needed.
template <bool kShared, bool kMixed>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_tile_pair_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map,
                            const __grid_constant__ CUtensorMap q_map, const __grid_constant__ TileArgs a,
                            uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_base_s;
  __shared__ Ctl ctl_s;
  __shared__ uint32_t bad_s[16][4];  // [piece % 16] a bit for each row that a page id outside the cache spoils
  __shared__ RangeScratch range_s;
  __shared__ uint32_t drop_s[4][4];  // CTA 0: [step % 4][32 tokens] to be looked at (nonfinite_seen)
  __shared__ float mx_s[2][2][2][64];  // [step parity][page][column half][row]
  __shared__ float lsum_s[2][2][64];   // [page][column half][row]

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const int w = kShared ? pair : pair / a.groups;
  const int grp = kShared ? 0 : pair % a.groups;
  const int np = a.block_table ? a.num_pages : a.batch * a.max_blocks;

  if (tid == 0) {
    ctl_s = Ctl{a.err, limit_ns, 0, map_to_rank(smem_u32(&ctl_s.abort), rank ^ 1u)};
    for (int i = 0; i < 64; ++i) bad_s[i / 4][i % 4] = 0;
    for (int i = 0; i < 16; ++i) drop_s[i / 4][i % 4] = 0;
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(bar(kFullK + s), 1);   // CTA 0's producer arms it with both CTAs' bytes
      mbar_init(bar(kEmptyK + s), 1);  // MMA commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kFullV + i), 2);  // CTA 0's producer, twice, or the two cleaning warps
      mbar_init(bar(kEmptyV + i), 1);
      mbar_init(bar(kDirty + i), 1);
      mbar_init(bar(kGroup + i), 4);
      mbar_init(bar(kDrain + i), 1);
    }
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQStage), 1);
    mbar_init(bar(kQReady), 16);
    mbar_init(bar(kQEmpty), 1);
    mbar_init(bar(kSFull), 1);
    mbar_init(bar(kSFree), 16);
    mbar_init(bar(kPFull), 16);
    mbar_init(bar(kODone), 1);
    mbar_init(bar(kOFree), 16);
    fence_mbar_init();
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&rope_map);
    tma_prefetch_desc(&q_map);
  }
  if (warp == kValues) {
    tmem_alloc_pair(smem_u32(&tmem_base_s), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers and tensor memory of both CTAs ready before any remote access
  tc_fence_after();
  warm_params(a, tid);
  // Everything above overlaps the previous grid on the stream; from here on its writes
  // (the lengths, q', the tables, the cache) are visible.
  grid_dep_wait();
  derive_range(TaskLengths<kShared>{&a}, kShared ? a.tiles : a.batch, a.num_workers, a.min_pages,
               a.granule, a.whole_slack, a.piece_cost, a.task, a.err, w, range_s);
  const uint32_t tmem = tmem_base_s;
  Ctl* const ctl = &ctl_s;
  auto bar0 = [&](int i) { return map_to_rank(bar(i), 0); };

  if (warp == kLoadK) {
    // ------------------------------------------------------------ q' and score loads
    PieceLoads<kRows, kShared> ld(a, range_s.rg, grp, np, lane);
    int slot = 0, piece = 0, fills = 0, g = 0, stages = 0;
    uint32_t phase = 1;
    int withheld = -1;
    bool ok = true;
    while (ok && ld.next()) {
      const int steps = (ld.pc.pe - ld.pc.pa + 1) / 2;
      // q' dims [0, 384) pass through two score slots on their way to tensor memory, so that
      // they are here before the tensor memory is free; the rest needs its place free first.
      // (The first piece's pass through the value slots, idle until its first P, by the value
      // loads' warp: its scores then need not wait for a slot of theirs.  64 windows of 4,096
      // tokens, 128 heads: 76.5 -> 75.3 us; 16, 64 heads, two queries: 33.6 -> 33.2.)  The
      // stage before has landed first: after a first piece of one step a slot is free at once.
      const int qrow = ld.k.row0 + 64 * (int)rank;
      if (piece > 0 && !wait_all(bar(kQStage), (piece - 1) & 1, ctl)) { ok = false; break; }
      stages = piece + 1;
      for (int m = 0; m < 2 && piece > 0; ++m) {
        if (!wait_all(bar(kEmptyK + slot), phase, ctl)) { ok = false; break; }
        if (lane == 0) {
          if (m == 0) mbar_expect_tx(bar(kQStage), kQTmemBoxes * kBox);
          tma_load_3d(sbase + kOffK + slot * kSlotBytes, &q_map, 0, qrow, kQSmemBoxes * m, bar(kQStage));
          if (rank == 0) mbar_arrive(bar(kFullK + slot));  // the slot's phase passes without bytes
        }
        ++fills;
        if (++slot == kKSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
      if (!ok || !wait_all(bar(kQEmpty), (piece & 1) ^ 1, ctl)) break;
      if (lane == 0) {
        if (rank == 0) mbar_expect_tx(bar(kQFull), 2 * kQSmemBoxes * kBox);
        tma_load_3d_pair(sbase + kOffQ, &q_map, 0, qrow, kQTmemBoxes, bar0(kQFull));
      }
      for (int i = 0; i < steps && ok; ++i, ++g) {
        bool dirty;
        const int y = ld.row(ld.pc.pa + 2 * i + (int)rank, dirty, nullptr);  // bad pages: the value loads mark the rows
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          // The rope rides on the second half.  That half's slot was last held by the first
          // half of the step before, whose MMAs follow the last ones that read this rope slot.
          if (!wait_all(bar(kEmptyK + slot), phase, ctl)) { ok = false; break; }
          if (a.withhold_arrive && blockIdx.x == 0 && fills == 1) {
            withheld = slot;  // timeout test: this fill never completes
          } else if (lane == 0) {
            if (rank == 0) mbar_expect_tx(bar(kFullK + slot), 2 * (kSlotBytes + (m == 1 ? kBox : 0)));
            const uint32_t fb = bar0(kFullK + slot);
            tma_load_3d_pair(sbase + kOffK + slot * kSlotBytes, &kv_map, 0, y, 4 * m, fb);
            if (m == 1) tma_load_3d_pair(sbase + kOffRope + (g & 1) * kBox, &rope_map, 0, y, 8, fb);
          }
          ++fills;
          if (++slot == kKSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (i == 0) ld.look();
      }
      ++piece;
    }
    // Drain: the last fill of each slot lands before the CTA may exit (bounded).
    if (stages > 0) drain_wait(bar(kQStage), (stages - 1) & 1, limit_ns);
    if (rank == 0) {
      for (int j = 1; j <= kKSlots && j <= fills; ++j) {
        const int f = fills - j, s = f % kKSlots;
        if (s != withheld) drain_wait(bar(kFullK + s), (f / kKSlots) & 1, limit_ns);
      }
      if (piece > 0) drain_wait(bar(kQFull), (piece - 1) & 1, limit_ns);
    }
    __syncwarp();
  } else if (warp == kLoadV) {
    // ------------------------------------------------------------ value loads
    PieceLoads<kRows, kShared> ld(a, range_s.rg, grp, np, lane);
    int piece = 0, g = 0;
    uint32_t dirty_fills[2] = {0, 0};
    bool ok = true;
    const uint32_t full0 = bar0(kFullV);
    while (ok && ld.next()) {
      const int steps = (ld.pc.pe - ld.pc.pa + 1) / 2;
      // The marks eight pieces on are those of eight pieces back, long read: these loads are
      // at most a step ahead of the value MMAs.
      if (lane < 4) bad_s[(piece + 8) & 15][lane] = 0;
      __syncwarp();
      if (piece == 0 && lane == 0) {  // the first q' on its way to tensor memory
        mbar_expect_tx(bar(kQStage), kQTmemBoxes * kBox);
        for (int m = 0; m < 2; ++m)
          tma_load_3d(sbase + kOffV + m * kSlotBytes, &q_map, 0, ld.k.row0 + 64 * (int)rank, kQSmemBoxes * m, bar(kQStage));
      }
      for (int i = 0; i < steps && ok; ++i, ++g) {
        bool dirty[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int y = ld.row(ld.pc.pa + 2 * i + m, dirty[m], bad_s[piece & 15]);
          if (!wait_all(bar(kEmptyV + m), g & 1, ctl)) { ok = false; break; }  // first freed by the first q'
          if (lane == 0) {
            const uint32_t dst = sbase + kOffV + m * kSlotBytes;
            if (dirty[m]) {
              mbar_expect_tx(bar(kDirty + m), kSlotBytes);
              tma_load_3d(dst, &kv_map, 0, y, 4 * (int)rank, bar(kDirty + m));
            } else {
              if (rank == 0) {
                mbar_expect_tx(bar(kFullV + m), 2 * kSlotBytes);
                mbar_arrive(bar(kFullV + m));
              }
              tma_load_3d_pair(dst, &kv_map, 0, y, 4 * (int)rank, bar0(kFullV + m));
            }
          }
          dirty_fills[m] += dirty[m] ? 1u : 0u;
        }
        if (!ok) break;
        // Rows [h0, h1) and [e0, 64) of a dirty page are cleared here: the next step's loads
        // wait for this one's slots anyway.
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          if (!(m ? dirty[1] : dirty[0])) continue;
          int t0, e0;
          ld.page(ld.pc.pa + 2 * i + m, t0, e0);
          const int h0 = kShared ? 0 : max(ld.k.s.hole0 - t0, 0), h1 = kShared ? 0 : max(h0, min(ld.k.s.hole1 - t0, kPage));
          const int nrow = (h1 - h0) + (kPage - e0);
          if (!wait_all(bar(kDirty + m), ((m ? dirty_fills[1] : dirty_fills[0]) - 1) & 1, ctl)) { ok = false; break; }
          uint8_t* st = smem + kOffV + m * kSlotBytes;
#pragma unroll 1
          for (int idx = lane; idx < nrow * 8; idx += 32) {
            const int r = idx / 8, row = r < h1 - h0 ? h0 + r : e0 + (r - (h1 - h0));
#pragma unroll
            for (int box = 0; box < 4; ++box)
              *reinterpret_cast<uint4*>(st + box * kBox + row * 128 + (idx % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) arrive_cta0(rank, bar(kFullV + m), full0 + 8 * m);
        }
        if (i == 0) ld.look();
      }
      ++piece;
    }
    // Drain (bounded): the last clean fill of a slot completes CTA 0's phase, a dirty one this CTA's.
    for (int m = 0; m < 2; ++m) {
      if (dirty_fills[m] > 0) drain_wait(bar(kDirty + m), (dirty_fills[m] - 1) & 1, limit_ns);
      if (ok && g > 0 && rank == 0) drain_wait(bar(kFullV + m), (g - 1) & 1, limit_ns);
    }
    __syncwarp();
  } else if (warp == kScores) {
    // ------------------------------------------------------------ score MMAs
    if (rank == 0) {
      PieceIter<kShared> pi(range_s.rg);
      Piece pc;
      constexpr uint64_t kKMajor = desc_sw128_const(16, 1024);
      const uint64_t dq = kKMajor | desc_addr(sbase + kOffQ), drope = kKMajor | desc_addr(sbase + kOffRope);
      const uint64_t dk = kKMajor | desc_addr(sbase + kOffK);
      const uint32_t d = tmem + kColS;
      int slot = 0, piece = 0, g = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && pi.next(pc, a)) {
        const int steps = (pc.pe - pc.pa + 1) / 2;
        if (!wait_all(bar(kQFull), piece & 1, ctl) || !wait_all(bar(kQReady), piece & 1, ctl)) break;
        for (int m = 0; m < 2; ++m) {  // the two slots that q' passed through are free
          if (piece == 0) {
            mma_commit_pair_elect(bar(kEmptyV + m), kBothCtas);
            continue;
          }
          mma_commit_pair_elect(bar(kEmptyK + slot), kBothCtas);
          if (++slot == kKSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
        for (int i = 0; i < steps && ok; ++i, ++g) {
          if (g > 0 && !wait_all(bar(kSFree), (g - 1) & 1, ctl)) { ok = false; break; }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!wait_all(bar(kFullK + slot), phase, ctl)) { ok = false; break; }
            tc_fence_after();
            const uint64_t bk = dk + (uint64_t)(slot * (kSlotBytes >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int blk = 4 * m + j;
              if (blk < kQTmemBoxes)
                mma_pair_ts_x4_elect<2>(d, tmem + kColQ + 32 * blk, bk + (uint64_t)(j * (kBox >> 4)), kIdescS, blk ? 1u : 0u);
              else
                mma_pair_x4_elect<2, 2>(d, dq + (uint64_t)((blk - kQTmemBoxes) * (kBox >> 4)), bk + (uint64_t)(j * (kBox >> 4)),
                                        kIdescS, 1u);
            }
            mma_commit_pair_elect(bar(kEmptyK + slot), kBothCtas);
            if (++slot == kKSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          mma_pair_x4_elect<2, 2>(d, dq + (uint64_t)((8 - kQTmemBoxes) * (kBox >> 4)), drope + (uint64_t)((g & 1) * (kBox >> 4)),
                                  kIdescS, 1u);
          mma_commit_pair_elect(bar(kSFull), kBothCtas);
        }
        if (!ok) break;
        mma_commit_pair_elect(bar(kQEmpty), kBothCtas);
        ++piece;
      }
      // The MMAs issued are done before tensor memory is released (bounded).
      mma_commit_pair_elect(bar(kDrain), 1);
      drain_wait(bar(kDrain), 0, limit_ns);
    }
    __syncwarp();
  } else if (warp == kValues) {
    // ------------------------------------------------------------ value MMAs
    if (rank == 0) {
      PieceIter<kShared> pi(range_s.rg);
      Piece pc;
      constexpr uint64_t kKMajor = desc_sw128_const(16, 1024), kMNMajor = desc_sw128_const(kBox, 1024);
      const uint64_t dp = kKMajor | desc_addr(sbase + kOffP), dv = kMNMajor | desc_addr(sbase + kOffV);
        int piece = 0, g = 0;
      bool ok = true;
      while (ok && pi.next(pc, a)) {
        const int steps = (pc.pe - pc.pa + 1) / 2;
        for (int i = 0; i < steps && ok; ++i, ++g) {
          if (!wait_all<kMixed>(bar(kPFull), g & 1, ctl) ||
              (i == 0 && piece > 0 && !wait_all(bar(kOFree), (piece - 1) & 1, ctl))) {
            ok = false;
            break;
          }
          if constexpr (kMixed) {
            const uint32_t drop = reinterpret_cast<volatile uint32_t*>(drop_s[g & 3])[lane & 3];
            if (__any_sync(0xffffffffu, drop)) {
              if (lane < 4) drop_s[g & 3][lane] = 0;  // before the fences of drop_values: set again four steps on
              if (!wait_all(bar(kFullV), g & 1, ctl) || !wait_all(bar(kFullV + 1), g & 1, ctl)) { ok = false; break; }
              drop_values(sbase + kOffV, drop, lane);
            }
          }
          tc_fence_after();
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!wait_all(bar(kFullV + m), g & 1, ctl)) { ok = false; break; }
            tc_fence_after();
            const uint64_t ap = dp + (uint64_t)(m * (kBox >> 4)), bv = dv + (uint64_t)(m * (kSlotBytes >> 4));
            mma_pair_x4x2_elect<2, 128, 128, 2 * (kBox >> 4)>(tmem + kColO, ap, bv, kIdescO, i + m ? 1u : 0u);
            mma_commit_pair_elect(bar(kEmptyV + m), kBothCtas);
          }
          if (!ok) break;
          mma_commit_pair_elect(bar(kODone), kBothCtas);
        }
        ++piece;
      }
      mma_commit_pair_elect(bar(kDrain + 1), 1);
      drain_wait(bar(kDrain + 1), 0, limit_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    const int q = warp & 3;                     // TMEM lane quadrant
    const int c = warp >> 2;  // which 32 of a page's 64 tokens, and O block
    const int h = (32 * q + lane) & 63;         // row within this CTA
    const int hh = q >> 1;                      // page of the step held in this lane
    const int row = 64 * (int)rank + h;         // row of the tile
    const int r32 = 32 * (q & 1);               // the warp's first row within this CTA
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    const float scale2 = a.scale * kLog2e;
    const uint32_t grp_bar = bar(kGroup + (q & 1));
    int meets = 0;
    // The 4 warps holding the same rows (quadrants q and q ^ 2, both column halves) meet.
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(grp_bar);
      const bool r = wait_all(grp_bar, meets & 1, ctl);
      ++meets;
      return r;
    };
    const uint32_t sfree0 = bar0(kSFree), pfull0 = bar0(kPFull), ofree0 = bar0(kOFree), qready0 = bar0(kQReady);
    uint8_t* const pbox = smem + kOffP + hh * kBox;
    // q' dims [192c, 192c + 192) of this lane's row into tensor memory, from the slot that
    // holds them (three boxes of 64 dims).  Rows past the batch's are zeros; other rows
    // past the tile's feed rows of S that the masks hide.
    int qslot = 0, staged = 0;  // the ring position of the next piece's q', pieces staged
    auto stage_q = [&](const Piece& x, auto first) -> bool {
      if (!wait_all(bar(kQStage), staged & 1, ctl)) return false;
      const uint8_t* src = smem + (first.value ? kOffV + c * kSlotBytes : kOffK + (qslot + c) % kKSlots * kSlotBytes) + h * 128;
#pragma unroll
      for (int k4 = 0; k4 < 6; ++k4) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(src + (k4 >> 1) * kBox + (((4 * (k4 & 1) + e) ^ (h & 7)) * 16));
          v[4 * e] = x4.x;
          v[4 * e + 1] = x4.y;
          v[4 * e + 2] = x4.z;
          v[4 * e + 3] = x4.w;
        }
        tmem_st16(tmem + lane_addr + kColQ + 96 * c + 16 * k4, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0(rank, bar(kQReady), qready0);
      qslot = (qslot + (first.value ? 0 : 2) + 2 * ((x.pe - x.pa + 1) / 2)) % kKSlots;
      ++staged;
      return true;
    };
    PieceIter<kShared> pi(range_s.rg), pn(range_s.rg);  // pn runs one piece ahead
    Piece pc, nc;
    // A piece's task and what this row sees of it, looked up a piece ahead, under the epilogue.
    struct RowTask {
      Task t;
      RowSight sight;
    };
    auto row_task = [&](const Piece& x) {
      RowTask r{load_task<kRows, kShared>(a, x.t, grp), {}};
      r.sight = row_sight<kShared>(a, r.t, row);
      return r;
    };
    bool have_next = pn.next(nc, a);
    RowTask kn{};
    if (have_next) kn = row_task(nc);
    bool ok = !have_next || stage_q(nc, std::true_type{});
    int g = 0, piece = 0;
    while (ok && pi.next(pc, a)) {
      have_next = pn.next(nc, a);
      const RowTask k = kn;
      const int steps = (pc.pe - pc.pa + 1) / 2;
      PageRef ref{};  // lane l: list page pa + 32 (i / 16) + l
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < steps && ok; ++i) {
        const int gs = g + i, u = gs & 1;
        const int p = pc.pa + 2 * i + hh;
        if ((i & 15) == 0) ref = page_ref<kShared>(a, k.t, min(pc.pa + 2 * i + lane, pc.pe - 1));
        if (!wait_all(bar(kSFull), gs & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float y[32];
        {
          uint32_t r[32];
          tmem_ld32(tmem + lane_addr + kColS + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cta0(rank, bar(kSFree), sfree0);
        const int t0 = __shfl_sync(0xffffffffu, ref.page, 2 * (i & 15) + hh) * kPage + 32 * c;
        const int seq = kShared ? __shfl_sync(0xffffffffu, ref.seq, 2 * (i & 15) + hh) : 0;
        uint32_t see = 0;
        if (p < pc.pe) {
          if constexpr (kShared)
            see = seq < 0 ? below(k.sight.prefix_end - t0) : seq == k.sight.seq ? below(k.sight.end - t0) : 0u;
          else
            see = below(k.sight.end - t0) & (below(a.sinks - t0) | ~below(k.sight.from - t0));
        }
        const uint64_t s2 = f2_pack(scale2, scale2);
#pragma unroll
        for (int j = 0; j < 32; j += 2) f2_unpack(f2_mul(f2_pack(y[j], y[j + 1]), s2), y[j], y[j + 1]);
        bool dropped = false;
        if (kMixed && (a.s_q > 1 || seq >= 0)) {
          const uint32_t d = __reduce_or_sync(0xffffffffu, nonfinite_seen(y, see));
          dropped = d != 0;
          if (dropped && lane == 0) red_or_cluster(map_to_rank(smem_u32(&drop_s[gs & 3][2 * hh + c]), 0), d);
        }
        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = ((see >> j) & 1u) ? y[j] : -INFINITY;
        }
        float t3[10];
#pragma unroll
        for (int j = 0; j < 10; ++j) t3[j] = fmax3(y[3 * j], y[3 * j + 1], y[3 * j + 2]);
        float mp = fmaxf(y[30], y[31]);
#pragma unroll
        for (int j = 0; j < 10; j += 2) mp = fmax3(mp, t3[j], t3[j + 1]);
        mx_s[u][hh][c][h] = mp;
        if (!meet()) { ok = false; break; }
        const float m_new = fmaxf(m, fmaxf(fmaxf(mx_s[u][0][0][h], mx_s[u][0][1][h]), fmaxf(mx_s[u][1][0][h], mx_s[u][1][1][h])));
        const bool need = !(m_new <= m + kRescaleThreshold);  // also while m is -inf and a token is seen
        const float alpha = !need ? 1.f : (m == -INFINITY ? 0.f : fast_exp2(m - m_new));
        if (need) m = m_new;
        l *= alpha;
        const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen nothing holds only masked scores
        const uint64_t nm = f2_pack(-mm, -mm);
        uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float a0, a1, a2, a3;
          f2_unpack(f2_add(f2_pack(y[j], y[j + 1]), nm), a0, a1);
          f2_unpack(f2_add(f2_pack(y[j + 2], y[j + 3]), nm), a2, a3);
          a0 = fast_exp2(a0);
          a1 = fast_exp2(a1);
          a2 = fast_exp2(a2);
          a3 = fast_exp2(a3);
          acc0 = f2_add(acc0, f2_pack(a0, a1));
          acc1 = f2_add(acc1, f2_pack(a2, a3));
          pk[j / 2] = pack_bf16x2(a0, a1);
          pk[j / 2 + 1] = pack_bf16x2(a2, a3);
        }
        float s0, s1, s2_, s3;
        f2_unpack(acc0, s0, s1);
        f2_unpack(acc1, s2_, s3);
        l += (s0 + s1) + (s2_ + s3);
        // P and O belong to the step before until its value MMAs are done.
        if (gs > 0 && !wait_all(bar(kODone), (gs - 1) & 1, ctl)) { ok = false; break; }
        if (i > 0 && __any_sync(0xffffffffu, need)) {
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 128; cc += 16) {
            uint32_t r[16];
            const uint32_t ta = tmem + lane_addr + kColO + 128 * c + cc;
            tmem_ld16(ta, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(ta, r);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(pbox + h * 128 + (((4 * c + e) ^ (h & 7)) * 16)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (dropped) mbar_arrive_cluster(pfull0);  // with what it wrote to CTA 0
          else arrive_cta0(rank, bar(kPFull), pfull0);
        }
      }
      if (!ok) break;
      const int ge = g + steps - 1;
      lsum_s[hh][c][h] = l;
      // ---- the next piece's q' into tensor memory once this piece's last score MMA has
      // read the current one, so that its scores run under this epilogue
      if (have_next) {
        if (!wait_all(bar(kQEmpty), piece & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        if (!stage_q(nc, std::false_type{})) { ok = false; break; }
        kn = row_task(nc);
      }
      if (!meet()) { ok = false; break; }
      const float l_row = (lsum_s[0][0][h] + lsum_s[0][1][h]) + (lsum_s[1][0][h] + lsum_s[1][1][h]);
      if (!wait_all(bar(kODone), ge & 1, ctl)) { ok = false; break; }
      tc_fence_after();
      const bool bad = k.sight.bad || ((const_cast<volatile uint32_t&>(bad_s[piece & 15][row >> 5]) >> (row & 31)) & 1u);
      const bool none = l_row == 0.f;  // the row sees no token of the piece
      const float inv = bad ? NAN : (none ? 0.f : 1.f / l_row);
      const PieceOut to = piece_out<kRows, kShared>(a, k.t, pc, pi.rg, w, grp);
      if (hh == 0 && c == 0 && row < k.t.live) {
        const float v = bad ? NAN : (none ? -INFINITY : (m + __log2f(l_row)) * kLn2);
        (to.direct ? a.lse : a.part_lse)[to.row0 + row] = v;
      }
      const size_t at = (to.row0 + 64 * rank + r32) * kDLatent + 256 * hh + 128 * c;
      const int live = k.t.live - 64 * (int)rank - r32;
      if (to.direct)
        store_rows<true>(tmem + lane_addr + kColO + 128 * c, inv, pbox, c, r32, lane, live, a.out + at);
      else
        store_rows<false>(tmem + lane_addr + kColO + 128 * c, inv, pbox, c, r32, lane, live, a.part_o + at);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cta0(rank, bar(kOFree), ofree0);
      g += steps;
      ++piece;
    }
  }

  // ------------------------------------------------------------ teardown
  if (tid == 0) grid_dep_launch_dependents();  // the combine grid may launch (it waits for this grid's writes)
  tc_fence_before();
  __syncthreads();
  if (ctl_s.abort) {
    // A load whose barrier the peer never armed has no phase to wait for: give it time to land.
    const uint64_t t0 = now_ns();
    while (now_ns() - t0 < 100000) {
    }
  }
  cluster_sync();  // the peer's MMAs, loads and arrivals are done with this CTA
  if (warp == kValues) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  if (ctl_s.abort) spoil_pieces<kRows, kShared>(a, range_s.rg, w, grp);  // set in both CTAs
}

template <bool kShared, bool kMixed>
cudaError_t launch_pair(const TileArgs& a, cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(decode_tile_pair_kernel<kShared, kMixed>), kAlloc, done);
  if (e != cudaSuccess) return e;
  CUtensorMap kv_map, rope_map, q_map;
  if (!tile_maps(a, 64, kQSmemBoxes, &kv_map, &rope_map, &q_map)) return cudaErrorInvalidValue;
  const uint64_t limit_ns = (uint64_t)a.wait_limit * 1000000ull;
  return launch_dependent(decode_tile_pair_kernel<kShared, kMixed>, 2 * a.num_workers * (kShared ? 1 : a.groups), kThreads,
                          kAlloc, 0, stream, kv_map, rope_map, q_map, a, limit_ns);
}

}  // namespace

cudaError_t launch_decode_tile_pair(const TileArgs& a, cudaStream_t stream) {
  if (a.prefix_len) return mixed_pages<true>(a) ? launch_pair<true, true>(a, stream) : launch_pair<true, false>(a, stream);
  return mixed_pages<false>(a) ? launch_pair<false, true>(a, stream) : launch_pair<false, false>(a, stream);
}

}  // namespace mla
