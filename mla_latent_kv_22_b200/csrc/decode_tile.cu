// Sliding-window and shared-prefix decode: split-KV absorbed decode with one CTA per
// worker, a tile of N = 16 or 32 query rows and one 64-token page per step.  The pieces of
// split tiles are merged by a second grid, in short calls by the cluster that made them.
//
// A page is loaded once and feeds both products from the same shared memory:
//     S[64 x 64]    = q'[N x 576] . K^T       (M = 64 rows, N = 64 tokens, K = 576)
//     O^T[512 x N] += V^T[512 x 64] . P^T     (four M = 128 blocks of dims, N rows, K = 64)
// The second product is taken transposed: its accumulator is 4 N columns of tensor memory
// instead of 512, so two of them fit beside S, and the page's [64 tokens x 64 dims] boxes
// serve as the K-major B operand of the first and, read MN-major, as the A operand of the
// second.  Rows of S at or beyond N come from whatever shared memory follows q' and are
// never read.
//
// Every 64-token page costs 36 + 16 MMAs whatever the row count (32 and 39-40 cycles each,
// bound by shared memory's 128 bytes a cycle: 1,780 cycles) under the 3,300 that its 73.7 KB
// take from HBM at an SM's share of the copy rate; so few rows (a window decode on a
// tensor-parallel shard) run at the speed of the loads: 1,700 ns a page on all 148 SMs, 6.4
// TB/s.  More rows share pages in tiles of 128 on a CTA pair (decode_tile_pair.cu).
//
// Roles (384 threads).  Warps 0-3: softmax of the 16 rows in their TMEM quadrant (two threads
// per row, 32 tokens each).  Warps 4-7: store a piece's O, from one of two accumulators
// while the next piece runs in the other.  Warp 8: page loads (TMA), two 32 KB halves of 256
// latent dims per page into a ring, freed by the second product, and the rope dims into two
// 8 KB slots, freed by the first.  Warp 9: q' loads and the first product's MMAs.  Warp 10:
// zeroes the rows of a page that no query of the sequence sees (past its end, or between the
// sinks and the window), where a masked P of 0 would meet whatever the cache holds.  Warp 11:
// tensor memory and the second product's MMAs.  (One warp issuing both products was bound by
// its own instruction stream: 52 MMAs of ~35 cycles and 14 waits and commits of 70-110 a
// page; two warps, and one commit per half, overlap them.)  The first warps also write the
// schedule's records, which the loads should not wait for.
//
// The running maximum is lazy as in decode_pair.cu: O and the sum are rescaled only when a
// page's maximum exceeds the reference by more than 2^8.  Since O's lanes are dims, all
// four warps rescale for a row of any of them; they meet once per page.  P is rounded to
// bf16 (half a step: 2^-8 relative) for the tensor cores; scores, sums, O and the split partials stay
// fp32; out is rounded once to bf16.
//
// Every mbarrier wait is bounded by a time limit; on expiry the kernel records
// MLA_ERR_DEVICE_TIMEOUT, drains its work in flight, makes the rows of its pieces NaN and
// returns.  No trap.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include <algorithm>
#include <cmath>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "tile_tasks.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kLoad = 8, kScores = 9, kClean = 10, kValues = 11;  // warps; 0-3 softmax, 4-7 store
constexpr int kBox = 8192;            // [64 tokens x 64 bf16], 128B swizzle
constexpr int kSlotBytes = 4 * kBox;  // a ring slot: one half (256 latent dims) of a page
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;  // O^T: block m at column N m of its buffer; S: two buffers of 64 columns

// Shared memory for a row tile of N: q' (9 boxes of [N rows x 64 dims]; twice at 16 rows, so
// that a piece's q' loads under the one before, once at 32, where five ring slots leave no
// room), P ([N rows x 64 tokens], twice), two rope slots and the latent ring.
template <int N>
struct Layout {
  static constexpr int kQBox = N * 128;
  static constexpr int kQBufs = N == 16 ? 2 : 1;
  static constexpr int kPBufs = 2;
  static constexpr int kOBufs = 2;  // O^T accumulators: a piece's leaves under the next one's pages
  static constexpr int kSlots = 5;
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kQBufs * 9 * kQBox;
  static constexpr int kOffRope = kOffP + kPBufs * kQBox;
  static constexpr int kOffRing = kOffRope + 2 * kBox;
  static constexpr int kBytes = kOffRing + kSlots * kSlotBytes;
  static constexpr int kAlloc = kBytes + 1024;  // + alignment slack
  static_assert(N == 16 || N == 32, "row tile");
  // The first product reads 64 rows of every q' box; the last box's reach stays inside.
  static_assert((kQBufs * 9 - 1) * kQBox + 64 * 128 <= kBytes, "q' rows read outside the allocation");
  static_assert(kQBox % 1024 == 0 && kOffRope % 1024 == 0 && kOffRing % 1024 == 0, "1024-byte tiles");
  static_assert(kAlloc + 2048 <= 232448, "dynamic + static shared memory above the per-CTA limit");
  static_assert(4 * N * kOBufs <= 256 && kColS + 128 <= kTmemCols, "tensor-memory regions overlap");
};
constexpr int kMaxSlots = 5;

enum Bar {
  kFull = 0,                   // [slot] a half landed (and, if dirty, was cleaned)
  kEmpty = kFull + kMaxSlots,  // [slot] the second product has read it
  kDirty = kEmpty + kMaxSlots, // [slot] a half with unseen rows landed
  kQFull = kDirty + kMaxSlots, // [2] q' of a piece landed
  kQEmpty = kQFull + 2,        // [2] the piece's last first product has read q'
  kSFull = kQEmpty + 2,        // [2] scores of a page are in S (and its rope slot is free)
  kSFree = kSFull + 2,         // [2] the 4 softmax warps have read them
  kPFull = kSFree + 2,         // [2] the 4 softmax warps wrote P (and rescaled O)
  kODone = kPFull + 2,         // [2] the second product of a page is done
  kOFull = kODone + 2,         // [2] the last second product of a piece is done
  kOScale = kOFull + 2,        // [2] the 4 softmax warps wrote the piece's row factors
  kOFree = kOScale + 2,        // [2] the 4 storing warps have read O and the factors
  kMeet = kOFree + 2,          // the 4 softmax warps met
  kDrain,                      // [2] either issuing warp's MMAs are all done
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
};

// Bounded wait on an mbarrier phase; false on timeout (recorded) or abort.  The first try is
// inlined, the rest is not (it would be at some thirty places).
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, Ctl* c) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_cta(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*const_cast<volatile int*>(&c->abort)) return false;
      const uint64_t t = now_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > c->limit_ns) {
        set_device_error(c->err, MLA_ERR_DEVICE_TIMEOUT);
        *const_cast<volatile int*>(&c->abort) = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, Ctl* c) {
  return __all_sync(0xffffffffu, mbar_try_wait_cta(bar, parity) || wait_long(bar, parity, c));
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = now_ns();
  while (!mbar_try_wait_cta(bar, parity) && now_ns() - t0 < limit_ns) {
  }
}

// Lane 4g + i gives v[j] of row j and takes v[j] = row i of lane 4g + j.
__device__ __forceinline__ void transpose4(float (&v)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
  for (int p = 0; p < 4; p += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, b0 ? v[p] : v[p + 1], 1);
    if (b0) v[p] = got;
    else v[p + 1] = got;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float got = __shfl_xor_sync(0xffffffffu, b1 ? v[p] : v[p + 2], 2);
    if (b1) v[p] = got;
    else v[p + 2] = got;
  }
}

// One 16-column block of O^T leaves for out (bf16) or a partial (fp32): TMEM column e of
// `taddr` is row e, lanes are dims.  inv[e] is the row's factor, `live` the number of rows
// stored, ob / po the address of (row lane % 4, the lane quad's first dim).  Four lanes
// trade four rows of their dims for one row's four dims each, so that a store covers 128
// (fp32) or 64 (bf16) contiguous bytes of four rows.
template <bool kDirect>
__device__ __forceinline__ void store_o16(const uint32_t (&r)[16], const float* inv, int live, __nv_bfloat16* ob, float* po,
                                          int lane) {
  const int i = lane & 3;
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r[e + j]);
    transpose4(v, lane);
    const float f = inv[e + i];
    if (e + i < live) {
      if (kDirect)
        *reinterpret_cast<uint2*>(ob + e * kDLatent) = make_uint2(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f));
      else
        *reinterpret_cast<float4*>(po + e * kDLatent) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    }
  }
}

// All of a warp's O^T: four accumulators of N columns from `taddr` on, 128 dims apart, of
// which the warp holds 32 from dim0 on; rows below `live` are stored.  Four blocks of 16
// columns are read together.
template <int N, bool kDirect>
__device__ __forceinline__ void store_o(uint32_t taddr, const float* inv, int live, __nv_bfloat16* out, float* part, int dim0,
                                        int lane) {
  const size_t at = (size_t)(lane & 3) * kDLatent + dim0 + (lane & ~3);
#pragma unroll 1
  for (int n0 = 0; n0 < 4 * (N / 16); n0 += 4) {
    uint32_t r[4][16];
#pragma unroll
    for (int j = 0; j < 4; ++j) tmem_ld16(taddr + 16 * (n0 + j), r[j]);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j, m = n / (N / 16), r0 = 16 * (n % (N / 16));
      const size_t off = at + (size_t)r0 * kDLatent + 128 * m;
      store_o16<kDirect>(r[j], inv + r0, live - r0, out + off, part + off, lane);
    }
  }
}

// Zeroes the values that are not finite of a page's tokens (bit j of lanes 0-15's word is token j, of lanes
// 16-31's token 32 + j) in the four boxes of either half.  By a whole warp, between the page's
// scores and its second product.
__device__ __noinline__ void drop_values(uint8_t* h0, uint8_t* h1, uint32_t word, int lane) {
#pragma unroll 1
  for (int t = 0; t < 64; ++t) {
    if (!((__shfl_sync(0xffffffffu, word, t >> 1 & 16) >> (t & 31)) & 1u)) continue;
    const int at = (lane >> 3) * kBox + t * 128 + (lane & 7) * 16;  // 32 chunks of 16 bytes
    *reinterpret_cast<uint4*>(h0 + at) = finite_chunk(*reinterpret_cast<uint4*>(h0 + at));
    *reinterpret_cast<uint4*>(h1 + at) = finite_chunk(*reinterpret_cast<uint4*>(h1 + at));
  }
  fence_proxy_async();
  __syncwarp();
}

// ---------------------------------------------------------------- combine
// Merges the pieces of a row's task by their lse, in the order of their pages, and writes the
// rows that no piece holds.  Four warps take a row, 128 dims each, with four pieces' loads in
// flight, the first four before the weights are known.  Where there are few rows, each of
// kSplit = 4 such groups takes a quarter of the pieces, and the first adds them up in order
// (a call of 30 rows in 148 pieces 30.4 -> 21.5 us).
constexpr int kCombineThreads = 512;

template <int kSplit>
struct MergeScratch {
  float4 acc[kSplit][128];
  float wsum[kSplit][4];
};

// Row r of sequence b, row gr of the batch's, whose task's record is s.
template <bool kShared, int kSplit, int kLoads>
__device__ __forceinline__ void merge_row(const TileArgs& a, int gr, int b, int r, const SeqInfo s, int split,
                                          MergeScratch<kSplit>* sm) {
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) & 3, N = a.row_tile;
  bool nan = s.num_pieces < 0;
  if (kShared && bad_length(a.seqlens[b], a.max_blocks)) {
    set_device_error(a.err, MLA_ERR_DEVICE_BAD_PAGE);
    nan = true;
  }
  if (s.num_pieces == 1) return;  // written by the decode grid
  const int n = max(s.num_pieces, 0);
  // Storage row of piece k; a window's groups lie side by side, N rows each.
  const size_t stride = kShared ? N : (size_t)a.groups * N;
  const int r0 = kShared ? gr % N : r;
  auto at = [&](int k) -> size_t { return (size_t)(k == 0 ? s.first_slot : s.first_worker + k) * stride + r0; };
  // This group's pieces [ka, ke): whole rounds of loads.
  const int per = kSplit > 1 ? ((n + kLoads * kSplit - 1) / (kLoads * kSplit)) * kLoads : n, ka = split * per, ke = min(n, ka + per);
  float4 x[kLoads];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      x[j] = k0 + j < ke ? reinterpret_cast<const float4*>(a.part_o + at(k0 + j) * kDLatent)[32 * part + lane]
                         : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(ka);
  float L = -INFINITY;
#pragma unroll 1
  for (int k = lane; k < n; k += 32) {
    const float v = a.part_lse[at(k)];
    nan |= v != v;
    L = fmaxf(L, v);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, o));
  uint2* const out2 = reinterpret_cast<uint2*>(a.out + (size_t)gr * kDLatent) + 32 * part + lane;
  nan = __any_sync(0xffffffffu, nan);
  if (nan || L == -INFINITY) {  // alike in all groups of a row
    const uint32_t v = nan ? 0x7fff7fffu : 0u;
    if (split == 0) *out2 = make_uint2(v, v);
    if (split == 0 && part == 0 && lane == 0) a.lse[gr] = nan ? NAN : -INFINITY;
    return;
  }
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, wsum = 0.f, mine = 0.f;
#pragma unroll 1
  for (int k0 = ka; k0 < ke; k0 += kLoads) {
    if (k0 > ka) load(k0);
    const int i = (k0 - ka) & 31;
    if (i == 0) mine = k0 + lane < ke ? expf(a.part_lse[at(k0 + lane)] - L) : 0.f;  // the weights of 32 pieces
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const float wk = __shfl_sync(0xffffffffu, mine, i + j);  // 0 past the last piece
      wsum += wk;
      acc[0] += wk * x[j].x;
      acc[1] += wk * x[j].y;
      acc[2] += wk * x[j].z;
      acc[3] += wk * x[j].w;
    }
  }
  if (kSplit > 1) {
    sm->acc[split][32 * part + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (lane == 0) sm->wsum[split][part] = wsum;
    __syncthreads();
    if (split == 0) {
#pragma unroll
      for (int g = 1; g < kSplit; ++g) {
        const float4 y = sm->acc[g][32 * part + lane];
        acc[0] += y.x;
        acc[1] += y.y;
        acc[2] += y.z;
        acc[3] += y.w;
        wsum += sm->wsum[g][part];
      }
    }
    __syncthreads();
  }
  if (split == 0) {
    const float inv = 1.f / wsum;
    *out2 = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    if (part == 0 && lane == 0) a.lse[gr] = L + logf(wsum);
  }
}

template <bool kShared, int kSplit>
__global__ void __launch_bounds__(kCombineThreads, 3) combine_tile_kernel(const __grid_constant__ TileArgs a) {
  constexpr int kRows = kCombineThreads / (128 * kSplit);  // rows at a time
  __shared__ MergeScratch<kSplit> scratch;
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int group = threadIdx.x >> 7, R = a.batch * a.rows;
#pragma unroll 1
  for (int gr = blockIdx.x * kRows + (kSplit > 1 ? 0 : group); gr < R; gr += gridDim.x * kRows) {
    const int b = gr / a.rows;
    merge_row<kShared, kSplit, 4>(a, gr, b, gr - b * a.rows, a.task[kShared ? gr / a.row_tile : b], kSplit > 1 ? group : 0, &scratch);
  }
}

// ---------------------------------------------------------------- teams
// A short call: a cluster of 8 or 16 CTAs (the team) per row tile shares out the tile's pages
// evenly and merges its pieces itself, behind a barrier of the cluster instead of in a second
// grid.  Such a call is a chain of latencies (lengths, table, page, the two products, store,
// merge); the team takes the second grid's start and the exchange over the batch's lengths
// out of it, and its launch off the host (9.7 -> 5.9 us a call).  us, split schedule / team of
// 8 / of 16: 16 heads over a window of 512 10.6 / 10.9 / 10.0, of 64 11.8 / 9.4 / 9.5; 2 such
// windows of 512 11.5 / 11.1 / 10.0, 14 of them 13.4 / 11.9 / -; 7 sequences of 16 heads behind
// 1,000 tokens 14.0 / 13.7 / 13.4.  (Pieces left in shared memory and read across the cluster
// took 10.4 for 9.7: every CTA has to stay until its peers have read.)

// The team's record of tile (t, grp), and this CTA's range of its pages.
template <bool kShared>
static __device__ __noinline__ void team_range(const TileArgs& a, int t, int rank, volatile WorkerRange& rg, SeqInfo& s) {
  const TaskLengths<kShared> len{&a};
  const bool bad = len.bad(t);
  const int n = task_pages<kShared>(a, t), q = max((n + a.team - 1) / a.team, a.min_pages), pa = rank * q, pe = min(pa + q, n);
  if (threadIdx.x == 0) {
    if (bad && rank == 0) set_device_error(a.err, MLA_ERR_DEVICE_BAD_PAGE);
    const int b = pa < pe ? t : -1;
    rg.b0 = rg.b1 = b;
    rg.p0 = pa;
    rg.p1 = pe;
    s = SeqInfo{a.team * t, bad ? -1 : (n + q - 1) / q, a.team * t};
  }
  __syncthreads();
}

// The team's rows, three per CTA at a time, with all pieces of a row in flight.
template <int N, bool kShared>
static __device__ __noinline__ void team_merge(const TileArgs& a, int t, int grp, int rank, const SeqInfo& s) {
  const Task k = load_task<N, kShared>(a, t, grp);
#pragma unroll 1
  for (int row = rank + a.team * (threadIdx.x >> 7); row < k.live; row += a.team * (kThreads / 128)) {
    const int gr = k.row0 + row, b = gr / a.rows;
    merge_row<kShared, 1, 16>(a, gr, b, gr - b * a.rows, s, 0, static_cast<MergeScratch<1>*>(nullptr));
  }
}

template <int N, bool kShared, bool kTeam>
__global__ void __launch_bounds__(kThreads, 1)
    decode_tile_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map,
                       const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ TileArgs a, uint64_t limit_ns) {
  using Lay = Layout<N>;
  constexpr int kSlots = Lay::kSlots;
  constexpr uint32_t kIdescS = idesc_bf16_f32(64, 64, 0, 0);   // A q' K-major, B rows K-major
  constexpr uint32_t kIdescO = idesc_bf16_f32(128, N, 1, 0);   // A rows MN-major, B P K-major
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_base_s;
  __shared__ Ctl ctl_s;
  constexpr int kWords = (N + 31) / 32;
  __shared__ uint32_t bad_s[16][kWords];  // [piece % 16] a bit for each row that a page id outside the cache spoils
  __shared__ RangeScratch range_s;
  __shared__ SeqInfo team_s;
  // Rescale factors and whether a warp has any.  Four pages deep: a warp may be three pages
  // ahead of another across the end of a piece, where they do not meet.
  constexpr int kAhead = 2 * Lay::kPBufs;
  __shared__ float al_s[kAhead][N];       // [page % kAhead][row]
  __shared__ int need_s[kAhead][4];       // [page % kAhead][warp]
  __shared__ float inv_s[Lay::kOBufs][N];  // [O buffer][row] 1 / l

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = kTeam ? blockIdx.x / a.team : blockIdx.x, rank = kTeam ? blockIdx.x % a.team : 0;
  const int w = (kShared ? unit : unit / a.groups) * (kTeam ? a.team : 1) + rank;
  const int grp = kShared ? 0 : unit % a.groups;
  const int np = a.block_table ? a.num_pages : a.batch * a.max_blocks;

  if (tid == 0) {
    ctl_s = Ctl{a.err, limit_ns, 0};
    for (int i = 0; i < 16 * kWords; ++i) bad_s[i / kWords][i % kWords] = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(kFull + s), 1);   // the producer, or the cleaning warp
      mbar_init(bar(kEmpty + s), 1);  // MMA commit
      mbar_init(bar(kDirty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kQFull + i), 1);
      mbar_init(bar(kQEmpty + i), 1);
      mbar_init(bar(kDrain + i), 1);
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 4);
      mbar_init(bar(kPFull + i), 4);
      mbar_init(bar(kODone + i), 1);
      mbar_init(bar(kOFull + i), 1);
      mbar_init(bar(kOScale + i), 4);
      mbar_init(bar(kOFree + i), 4);
    }
    mbar_init(bar(kMeet), 4);
    fence_mbar_init();
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&rope_map);
    tma_prefetch_desc(&q_map);
  }
  if (warp == kValues) {
    tmem_alloc(smem_u32(&tmem_base_s), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  warm_params(a, tid);
  // Everything above overlaps the previous grid on the stream; from here on its writes
  // (the lengths, q', the tables, the cache) are visible.
  grid_dep_wait();
  if constexpr (kTeam)
    team_range<kShared>(a, w / a.team, rank, range_s.rg, team_s);
  else
    derive_range(TaskLengths<kShared>{&a}, kShared ? a.tiles : a.batch, a.num_workers, a.min_pages,
                 a.granule, a.whole_slack, a.piece_cost, a.task, a.err, w, range_s);
  const uint32_t tmem = tmem_base_s;
  Ctl* const ctl = &ctl_s;

  if (warp == kLoad) {
    // ------------------------------------------------------------ page loads
    PieceLoads<N, kShared> ld(a, range_s.rg, grp, np, lane);
    int slot = 0, piece = 0, fills = 0, g = 0;
    uint32_t phase = 1;               // parity of the "empty" phase to wait for
    uint32_t dpar = 0;                // [slot] parity of the slot's next dirty fill
    uint32_t was_dirty = 0, was = 0;  // [slot] the last fill was dirty; there was one
    uint32_t lpar = 0;                // [slot] parity of the last fill's phase
    int withheld = -1;
    bool ok = true;
    while (ok && ld.next()) {
      // The marks eight pieces on are those of eight pieces back, long read: five ring slots
      // hold halves of at most three pieces whose second product is not done.
      if (lane < kWords) bad_s[(piece + 8) & 15][lane] = 0;
      __syncwarp();
      for (int p = ld.pc.pa; p < ld.pc.pe && ok; ++p, ++g) {
        bool dirty;
        const int y = ld.row(p, dirty, bad_s[piece & 15]);
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          // The page's rope rides on its second half, whose ring slot (of five) was last held
          // by the first half of the page two before: with its second product done, that
          // page's scores are, and its rope slot is free.
          if (!wait_all(bar(kEmpty + slot), phase, ctl)) { ok = false; break; }
          const uint32_t bit = 1u << slot;
          if (a.withhold_arrive && blockIdx.x == 0 && fills == 1) {
            withheld = slot;  // timeout test: this fill never completes
          } else if (lane == 0) {
            const uint32_t b = bar((dirty ? kDirty : kFull) + slot);
            mbar_expect_tx(b, kSlotBytes + (m == 1 ? kBox : 0));
            tma_load_3d(sbase + Lay::kOffRing + slot * kSlotBytes, &kv_map, 0, y, 4 * m, b);
            if (m == 1) tma_load_3d(sbase + Lay::kOffRope + (g & 1) * kBox, &rope_map, 0, y, 8, b);
          }
          if (dirty) {
            lpar = (lpar & ~bit) | (dpar & bit);
            dpar ^= bit;
            was_dirty |= bit;
          } else {
            lpar = (lpar & ~bit) | ((phase ^ 1u) ? bit : 0u);
            was_dirty &= ~bit;
          }
          was |= bit;
          ++fills;
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (p == min(ld.pc.pa + 1, ld.pc.pe - 1)) ld.look();
      }
      ++piece;
    }
    // Drain: every load issued lands before the CTA may exit (bounded).
    if (lane == 0) {
      for (int s = 0; s < kSlots; ++s)
        if (((was >> s) & 1u) && s != withheld)
          drain_wait(bar((((was_dirty >> s) & 1u) ? kDirty : kFull) + s), (lpar >> s) & 1u, limit_ns);
    }
    __syncwarp();
  } else if (warp == kScores) {
    // ------------------------------------------------------------ q' loads, scores
    PieceIter<kShared> pi(range_s.rg), pq(range_s.rg);  // pq: the next piece whose q' is loaded
    Piece pc, qc;
    // Descriptors: a K-major step of 16 dims is 32 bytes.
    constexpr uint64_t kKMajor = desc_sw128_const(16, 1024);
    const uint64_t dq0 = kKMajor | desc_addr(sbase + Lay::kOffQ);
    const uint64_t drope = kKMajor | desc_addr(sbase + Lay::kOffRope);
    const uint32_t ring = desc_addr(sbase + Lay::kOffRing);
    constexpr int kQBufs = Lay::kQBufs;
    int slot = 0, piece = 0, loaded = 0, g = 0;
    uint32_t phase = 0;
    bool ok = true, more = true;
    // q' of the next piece into its buffer, once the piece that used it is done with it.
    auto load_q = [&]() -> bool {
      if (!more || !(more = pq.next(qc, a))) return true;
      const int qb = loaded % kQBufs;
      if (!wait_all(bar(kQEmpty + qb), ((loaded / kQBufs) & 1) ^ 1, ctl)) return false;
      if (lane == 0) {
        mbar_expect_tx(bar(kQFull + qb), 9 * Lay::kQBox);
        tma_load_3d(sbase + Lay::kOffQ + qb * 9 * Lay::kQBox, &q_map, 0, load_task<N, kShared>(a, qc.t, grp).row0, 0,
                    bar(kQFull + qb));
      }
      ++loaded;
      __syncwarp();
      return true;
    };
    ok = load_q();
    while (ok && pi.next(pc, a)) {
      const int n = pc.pe - pc.pa;
      const int qb = piece % kQBufs;
      if (!wait_all(bar(kQFull + qb), (piece / kQBufs) & 1, ctl)) { ok = false; break; }
      const uint64_t dq = dq0 + (uint64_t)(qb * (9 * Lay::kQBox >> 4));
      for (int i = 0; i < n && ok; ++i, ++g) {
        if (!wait_all(bar(kSFree + (g & 1)), ((g >> 1) & 1) ^ 1, ctl)) { ok = false; break; }
        const uint32_t d = tmem + kColS + 64 * (g & 1);
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          if (!wait_all(bar(kFull + slot), phase, ctl)) { ok = false; break; }
          tc_fence_after();
          const uint64_t bk = kKMajor | (ring + slot * (kSlotBytes >> 4));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_x4_elect<2, 2>(d, dq + (uint64_t)((4 * m + j) * (Lay::kQBox >> 4)), bk + (uint64_t)(j * (kBox >> 4)), kIdescS,
                               m + j ? 1u : 0u);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_x4_elect<2, 2>(d, dq + 8 * (Lay::kQBox >> 4), drope + (g & 1) * (kBox >> 4), kIdescS, 1u);
        mma_commit_elect(bar(kSFull + (g & 1)));
        if (kQBufs == 2 && i == 0) ok = load_q();
      }
      if (!ok) break;
      mma_commit_elect(bar(kQEmpty + qb));
      if (kQBufs == 1) ok = load_q();
      ++piece;
    }
    // The MMAs issued are done before tensor memory is released, q' has landed (bounded).
    mma_commit_elect(bar(kDrain));
    drain_wait(bar(kDrain), 0, limit_ns);
    for (int j = 1; j <= kQBufs && j <= loaded; ++j)
      drain_wait(bar(kQFull + (loaded - j) % kQBufs), ((loaded - j) / kQBufs) & 1, limit_ns);
    __syncwarp();
  } else if (warp == kClean) {
    // ------------------------------------------------------------ rows in no query's sight
    PieceIter<kShared> pi(range_s.rg);
    Piece pc;
    int slot = 0;
    uint32_t dpar = 0;
    bool ok = true;
    while (ok && pi.next(pc, a)) {
      const Task k = load_task<N, kShared>(a, pc.t, grp);
      for (int p0 = pc.pa; p0 < pc.pe && ok; p0 += 32) {
        const int np0 = min(32, pc.pe - p0);
        const PageRef ref = page_ref<kShared>(a, k, min(p0 + lane, pc.pe - 1));
        uint32_t dirty = __ballot_sync(0xffffffffu, lane < np0 && page_dirty<kShared>(k, ref));
        int done = 0;  // pages of the 32 passed
        for (; dirty && ok; dirty &= dirty - 1) {
          const int j = __ffs(dirty) - 1;
          slot = (slot + 2 * (j - done)) % kSlots;
          done = j + 1;
          const int t0 = __shfl_sync(0xffffffffu, ref.page, j) * kPage;
          // Rows [h0, h1) and [e0, 64) of the page.
          const int h0 = kShared ? 0 : max(k.s.hole0 - t0, 0), h1 = kShared ? 0 : max(h0, min(k.s.hole1 - t0, kPage));
          const int e0 = __shfl_sync(0xffffffffu, ref.valid_rows(), j);
          const int nrow = (h1 - h0) + (kPage - e0);
          for (int m = 0; m < 2; ++m) {
            if (!wait_all(bar(kDirty + slot), (dpar >> slot) & 1u, ctl)) { ok = false; break; }
            dpar ^= 1u << slot;
            uint8_t* st = smem + Lay::kOffRing + slot * kSlotBytes;
#pragma unroll 1
            for (int idx = lane; idx < nrow * 8; idx += 32) {
              const int r = idx / 8, row = r < h1 - h0 ? h0 + r : e0 + (r - (h1 - h0));
#pragma unroll
              for (int box = 0; box < 4; ++box)
                *reinterpret_cast<uint4*>(st + box * kBox + row * 128 + (idx % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kFull + slot));
            if (++slot == kSlots) slot = 0;
          }
        }
        slot = (slot + 2 * (np0 - done)) % kSlots;
      }
    }
  } else if (warp == kValues) {
    // ------------------------------------------------------------ O^T += V^T P^T
    // An MN-major step of 16 tokens is 2048 bytes; two 64-dim boxes side by side are the
    // MN-major halves of 128 dims.
    PieceIter<kShared> pi(range_s.rg);
    Piece pc;
    constexpr uint64_t kKMajor = desc_sw128_const(16, 1024), kMNMajor = desc_sw128_const(kBox, 1024);
    const uint64_t dp = kKMajor | desc_addr(sbase + Lay::kOffP);
    const uint32_t ring = desc_addr(sbase + Lay::kOffRing);
    constexpr int kOBufs = Lay::kOBufs;
    int slot = 0, piece = 0, g = 0;
    bool ok = true;
    while (ok && pi.next(pc, a)) {
      const int n = pc.pe - pc.pa, ob = piece % kOBufs;
      const uint32_t o = tmem + kColO + 4 * N * ob;
      for (int i = 0; i < n; ++i, ++g) {
        if (!wait_all(bar(kPFull + (g & 1)), (g >> 1) & 1, ctl) ||
            (i == 0 && piece >= kOBufs && !wait_all(bar(kOFree + ob), (piece / kOBufs - 1) & 1, ctl))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bp = dp + (uint64_t)((g % Lay::kPBufs) * (Lay::kQBox >> 4));
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          const uint64_t av = kMNMajor | (ring + slot * (kSlotBytes >> 4));
          mma_x4_elect<128, 2>(o + N * 2 * m, av, bp, kIdescO, i ? 1u : 0u);
          mma_x4_elect<128, 2>(o + N * (2 * m + 1), av + 2 * (kBox >> 4), bp, kIdescO, i ? 1u : 0u);
          mma_commit_elect(bar(kEmpty + slot));
          if (++slot == kSlots) slot = 0;
        }
        mma_commit_elect(bar(kODone + (g & 1)));
      }
      if (!ok) break;
      mma_commit_elect(bar(kOFull + ob));
      ++piece;
    }
    mma_commit_elect(bar(kDrain + 1));
    drain_wait(bar(kDrain + 1), 0, limit_ns);
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ softmax
    const int q = warp & 3;               // TMEM lane quadrant
    const int half = lane >> 4;           // which 32 of the page's 64 tokens
    const int row = 16 * q + (lane & 15); // row of the tile
    const bool holds = 16 * q < N;        // warps beyond the tile only rescale O
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    const float scale2 = a.scale * kLog2e;
    int meets = 0;
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kMeet));
      const bool r = wait_all(bar(kMeet), meets & 1, ctl);
      ++meets;
      return r;
    };
    const bool mixed = mixed_pages<kShared>(a);
    uint8_t* const prow = smem + Lay::kOffP + (row < N ? row : 0) * 128;
    constexpr int kOBufs = Lay::kOBufs;
    PieceIter<kShared> pi(range_s.rg);
    Piece pc;
    int g = 0, piece = 0;
    bool ok = true;
    while (ok && pi.next(pc, a)) {
      const Task k = load_task<N, kShared>(a, pc.t, grp);
      const int n = pc.pe - pc.pa, ob = piece % kOBufs;
      const uint32_t o = tmem + lane_addr + kColO + 4 * N * ob;
      const RowSight sight = row_sight<kShared>(a, k, row);
      PageRef ref{};  // lane l: list page pa + 32 (i / 32) + l
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n && ok; ++i) {
        const int gs = g + i, u = gs & 1;
        if ((i & 31) == 0) ref = page_ref<kShared>(a, k, min(pc.pa + i + lane, pc.pe - 1));
        float y[32];
        float mp = -INFINITY;
        if (!wait_all(bar(kSFull + u), (gs >> 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        if (holds) {
          uint32_t r[32];
          tmem_ld16x2_32<32>(tmem + lane_addr + kColS + 64 * u, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + u));
        if (holds) {
          const int t0 = __shfl_sync(0xffffffffu, ref.page, i & 31) * kPage + 32 * half;
          const int seq = kShared ? __shfl_sync(0xffffffffu, ref.seq, i & 31) : 0;
          uint32_t see;
          if constexpr (kShared)
            see = seq < 0 ? below(sight.prefix_end - t0) : seq == sight.seq ? below(sight.end - t0) : 0u;
          else
            see = below(sight.end - t0) & (below(a.sinks - t0) | ~below(sight.from - t0));
          const uint64_t s2 = f2_pack(scale2, scale2);
#pragma unroll
          for (int j = 0; j < 32; j += 2) f2_unpack(f2_mul(f2_pack(y[j], y[j + 1]), s2), y[j], y[j + 1]);
          if (mixed && (a.s_q > 1 || seq >= 0)) {
            // The page's values are here (its scores are), and the second product waits for P.
            const uint32_t d = nonfinite_seen(y, see);
            const uint32_t d0 = __reduce_or_sync(0xffffffffu, half ? 0u : d), d1 = __reduce_or_sync(0xffffffffu, half ? d : 0u);
            if (d0 | d1) {
              uint8_t* const ring = smem + Lay::kOffRing;
              drop_values(ring + 2 * gs % kSlots * kSlotBytes, ring + (2 * gs + 1) % kSlots * kSlotBytes, half ? d1 : d0, lane);
            }
          }
          if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = ((see >> j) & 1u) ? y[j] : -INFINITY;
          }
          float t3[10];
#pragma unroll
          for (int j = 0; j < 10; ++j) t3[j] = fmax3(y[3 * j], y[3 * j + 1], y[3 * j + 2]);
          mp = fmaxf(y[30], y[31]);
#pragma unroll
          for (int j = 0; j < 10; j += 2) mp = fmax3(mp, t3[j], t3[j + 1]);
          mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, 16));
        }
        const float m_new = fmaxf(m, mp);
        const bool need = !(m_new <= m + kRescaleThreshold);  // also while m is -inf and a token is seen
        const float alpha = !need ? 1.f : (m == -INFINITY ? 0.f : fast_exp2(m - m_new));
        if (need) m = m_new;
        if (i > 0) {
          // O^T's lanes are dims: a row's rescale concerns every warp.
          const int s4 = gs & (kAhead - 1);
          if (half == 0 && holds) al_s[s4][row] = alpha;
          const bool any = __any_sync(0xffffffffu, need);
          if (lane == 0) need_s[s4][q] = any;
          if (!meet()) { ok = false; break; }
          if (need_s[s4][0] | need_s[s4][1] | need_s[s4][2] | need_s[s4][3]) {
            if (!wait_all(bar(kODone + (u ^ 1)), ((gs - 1) >> 1) & 1, ctl)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 4 * N; cc += 16) {
              uint32_t r[16];
              tmem_ld16(o + cc, r);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * al_s[s4][(cc & (N - 1)) + e]);
              tmem_st16(o + cc, r);
            }
            tmem_wait_st();
          }
        }
        // The page that last used this P buffer must have been read before it is rewritten.
        if (!wait_all(bar(kODone + u), ((gs >> 1) & 1) ^ 1, ctl)) { ok = false; break; }
        if (holds) {
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
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(prow + (u % Lay::kPBufs) * Lay::kQBox + (((4 * half + c) ^ (row & 7)) * 16)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + u));
      }
      if (!ok) break;
      // ---- the piece's row factors for the storing warps, and lse
      const bool bad =
          sight.bad || (holds && ((const_cast<volatile uint32_t&>(bad_s[piece & 15][row >> 5]) >> (row & 31)) & 1u));
      const float l_row = l + __shfl_xor_sync(0xffffffffu, l, 16);
      const bool none = l_row == 0.f;  // the row sees no token of the piece
      if (piece >= kOBufs && !wait_all(bar(kOFree + ob), (piece / kOBufs - 1) & 1, ctl)) break;
      if (half == 0 && holds) inv_s[ob][row] = bad ? NAN : (none ? 0.f : 1.f / l_row);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOScale + ob));
      if (holds && half == 0 && row < k.live) {
        const PieceOut to = piece_out<N, kShared>(a, k, pc, pi.rg, w, grp);
        const float v = bad ? NAN : (none ? -INFINITY : (m + __log2f(l_row)) * kLn2);
        (to.direct ? a.lse : a.part_lse)[to.row0 + row] = v;
      }
      g += n;
      ++piece;
    }
  } else {
    // ------------------------------------------------------------ O / l leaves
    constexpr int kOBufs = Lay::kOBufs;
    const int q = warp & 3;
    PieceIter<kShared> pi(range_s.rg);
    Piece pc;
    int piece = 0;
    while (pi.next(pc, a)) {
      const Task k = load_task<N, kShared>(a, pc.t, grp);
      const PieceOut to = piece_out<N, kShared>(a, k, pc, pi.rg, w, grp);
      const int ob = piece % kOBufs, par = (piece / kOBufs) & 1;
      const uint32_t o = tmem + ((uint32_t)(32 * q) << 16) + kColO + 4 * N * ob;
      if (!wait_all(bar(kOScale + ob), par, ctl) || !wait_all(bar(kOFull + ob), par, ctl)) break;
      tc_fence_after();
      if (to.direct)
        store_o<N, true>(o, inv_s[ob], k.live, a.out + to.row0 * kDLatent, nullptr, 32 * q, lane);
      else
        store_o<N, false>(o, inv_s[ob], k.live, nullptr, a.part_o + to.row0 * kDLatent, 32 * q, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOFree + ob));
      ++piece;
    }
  }

  // ------------------------------------------------------------ teardown
  if (tid == 0) grid_dep_launch_dependents();  // the combine grid may launch (it waits for this grid's writes)
  tc_fence_before();
  __syncthreads();
  if (warp == kValues) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (ctl_s.abort) spoil_pieces<N, kShared>(a, range_s.rg, w, grp);
  if constexpr (kTeam) {
    __syncwarp();
    cluster_sync();  // the team's partials are written
    team_merge<N, kShared>(a, w / a.team, grp, rank, team_s);
  }
}

template <bool kShared, int kSplit>
cudaError_t launch_combine_tile(const TileArgs& a, int grid, cudaStream_t stream) {
  return launch_dependent(combine_tile_kernel<kShared, kSplit>, grid, kCombineThreads, 0, 0, stream, a);
}

template <int N, bool kShared, bool kTeam>
cudaError_t launch_tile(const TileArgs& a, cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(decode_tile_kernel<N, kShared, kTeam>), Layout<N>::kAlloc, done);
  if (e != cudaSuccess) return e;
  CUtensorMap kv_map, rope_map, q_map;
  if (!tile_maps(a, N, 9, &kv_map, &rope_map, &q_map)) return cudaErrorInvalidValue;
  const uint64_t limit_ns = (uint64_t)a.wait_limit * 1000000ull;
  return launch_dependent(decode_tile_kernel<N, kShared, kTeam>, kShared ? a.num_workers : a.num_workers * a.groups, kThreads,
                          Layout<N>::kAlloc, a.team, stream, kv_map, rope_map, q_map, a, limit_ns);
}

template <int N, bool kShared>
cudaError_t launch_tile(const TileArgs& a, cudaStream_t stream) {
  return a.team ? launch_tile<N, kShared, true>(a, stream) : launch_tile<N, kShared, false>(a, stream);
}

}  // namespace

namespace {

constexpr int kRowTiles[] = {16, 32, 128};

// How many teams of `size` CTAs run at once on the current device (a cluster's CTAs share a GPC,
// and GPCs differ in size: 15 of 8 and 7 of 16 where this was measured).
int teams_at_once(int size) {
  static std::atomic<int> known[64][2];  // + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const auto allow_wide = [](auto fn) {  // clusters above the portable 8
    return cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  };
  std::atomic<int>& k = known[dev][size > 8];
  if (k.load() == 0) {
    const auto kernel = decode_tile_kernel<16, false, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Layout<16>::kAlloc;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<16>::kAlloc) != cudaSuccess ||
        !allow_wide(kernel) || !allow_wide(decode_tile_kernel<16, true, true>) || !allow_wide(decode_tile_kernel<32, false, true>) ||
        !allow_wide(decode_tile_kernel<32, true, true>) ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      n = 0;
      cudaGetLastError();  // no teams, then
    }
    k.store(n + 1);
  }
  return k.load() - 1;
}

// The most pages of a tile of n rows that the window or the tables allow.
long long most_pages(const TileArgs& a, int n) {
  if (a.prefix_len) {
    const int seqs = a.rows % n == 0 ? 1 : n % a.rows == 0 ? n / a.rows : (n - 1) / a.rows + 2;
    return a.prefix_blocks + (long long)a.max_blocks * std::min(seqs, a.batch);
  }
  const long long w = ((long long)a.window + a.s_q - 1) / kPage + 2 + ((long long)a.sinks + kPage - 1) / kPage;
  return std::min<long long>(a.max_blocks, w);
}

// CTAs per team for tiles of n rows, or 0: teams that run at once, with so few pages each that
// they end before the split schedule would, which has all SMs but two grids (a call of one
// tile: 1 page, of up to 6: 2, of more: 3; us split / team: a window of 960 for 16 heads 11.2 /
// 11.3 at 2 pages each, two of them 11.9 / 11.4; 7 sequences behind 2,000 tokens 15.4 / 14.8 at
// 3, 3 of them 13.8 / 14.2).  A schedule knob means the split schedule.
int team_size(const TileArgs& a, int n) {
  if (n > 32 || knob_value(MLA_KNOB_NUM_WORKERS) || knob_value(MLA_KNOB_MIN_PAGES) || knob_value(MLA_KNOB_SPLIT_POLICY) ||
      knob_value(MLA_KNOB_PIECE_COST))
    return 0;
  const long long tiles = a.prefix_len ? ((long long)a.batch * a.rows + n - 1) / n : (long long)a.batch * ((a.rows + n - 1) / n);
  const long long pages = most_pages(a, n), most = tiles == 1 ? 1 : tiles <= 6 ? 2 : 3;
  for (int size : {16, 8})
    if (pages <= size * most && tiles * size <= a.sm_count && tiles <= teams_at_once(size)) return size;
  return 0;
}

// The sizes that follow from a row tile, and the workspace (see plan_tile).
size_t lay_out(TileArgs* a, int row_tile, int sm_count, int forced_workers, void* base) {
  const bool shared = a->prefix_len != nullptr;
  a->sm_count = sm_count;
  a->row_tile = row_tile;
  a->groups = (a->rows + row_tile - 1) / row_tile;
  a->tiles = shared ? (int)(((long long)a->batch * a->rows + row_tile - 1) / row_tile) : 0;
  const int workers = row_tile == 128 ? sm_count / 2 : sm_count;
  a->num_workers = std::max(1, shared ? workers : workers / a->groups);
  if (forced_workers > 0) a->num_workers = forced_workers;
  const size_t tasks = shared ? a->tiles : a->batch;
  const size_t rows = (size_t)2 * a->num_workers * (shared ? 1 : a->groups) * row_tile;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? static_cast<char*>(base) + off : nullptr;
    off += (bytes + 255) & ~size_t(255);
    return p;
  };
  a->task = reinterpret_cast<SeqInfo*>(take(tasks * sizeof(SeqInfo)));
  a->part_lse = reinterpret_cast<float*>(take(rows * sizeof(float)));
  a->part_o = reinterpret_cast<float*>(take(rows * kDLatent * sizeof(float)));
  a->team = base ? team_size(*a, row_tile) : 0;  // no more partials than of the split schedule's workers
  if (a->team) a->num_workers = a->team * (shared ? a->tiles : a->batch);
  return off;
}

// Estimated us of a call in tiles of kRowTiles[i] rows: a call's own, and a page's per worker,
// fitted to 39 shapes of the split schedule (us at 16 / 32 / 128 rows a tile: a window of 512 for
// 128 heads 11.6 / 11.7 / 15.5, 64 windows of 1,024 for 64 heads 58 / 37 / 27; 7 sequences of 16
// heads behind 1,000 tokens 13.4 / 14.2 / 17.5, 16 behind 16,000 44 / 32 / 25; tiles of 64 rows on
// one CTA were best nowhere).  The pages are those that the window or the prefix's table allow,
// and, behind a shared prefix, `own` of each sequence.
double tile_time(const TileArgs& a, int i, int sm_count, double own) {
  constexpr double fixed[] = {10.2, 10.8, 14.3}, page[] = {1.5, 1.7, 0.8};
  const int n = kRowTiles[i];
  double pages;
  if (a.prefix_len)
    pages = (double)(((long long)a.batch * a.rows + n - 1) / n) * a.prefix_blocks + own * a.batch * (1 + (a.rows - 1) / n);
  else
    pages = (double)a.batch * most_pages(a, n) * ((a.rows + n - 1) / n);
  return fixed[i] + page[i] * std::max(2.0, pages / (n == 128 ? sm_count / 2 : sm_count));
}

// The row tile with the least estimated time.  A narrow tile costs more per row and page, but
// spreads the fixed parts of a short call (above all the partials' stores, at 32 bytes a cycle
// and SM) over more SMs.  The host does not know the lengths, and a server's tables may be as
// wide as its longest allowed sequence: behind a shared prefix the tile that serves both few own
// pages (4 a sequence) and many (half the table) is taken, by the sum of its times over the best
// ones.  (By half the table alone, 2,048 columns swamped the prefix: 64 sequences of 16 heads
// with up to 200 tokens behind 4,096 took 46.9 us in 16-row tiles for 27 in 128-row ones, 32 with
// up to 300 behind 4,000 33.5 for 24.  By the estimate over 20,000 drawn shapes with 2,048
// columns, the choice costs at most 1.2 times the best one's time, 4.6 times by half the table.)
int pick_row_tile(const TileArgs& a, int sm_count) {
  const int forced = knob_value(MLA_KNOB_ROW_TILE);
  for (int n : kRowTiles)
    if (forced == n) return n;
  if ((a.prefix_len ? (long long)a.batch * a.rows : a.rows) <= 16) return 16;
  double loss[3] = {};
  const double many = 0.5 * a.max_blocks;
  for (double own : {std::min(4.0, many), many}) {
    double t[3];
    for (int i = 0; i < 3; ++i) t[i] = tile_time(a, i, sm_count, own);
    const double best = *std::min_element(t, t + 3);
    for (int i = 0; i < 3; ++i) loss[i] += t[i] / best;
  }
  return kRowTiles[std::min_element(loss, loss + 3) - loss];
}

}  // namespace

size_t plan_tile(TileArgs* a, int sm_count, int forced_workers, void* base) {
  return lay_out(a, pick_row_tile(*a, sm_count), sm_count, forced_workers, base);
}

size_t tile_bytes(TileArgs a, int sm_count, int forced_workers) {
  const int forced = knob_value(MLA_KNOB_ROW_TILE);
  const bool few = (a.prefix_len ? (long long)a.batch * a.rows : a.rows) <= 16;  // never better in a wider tile
  size_t most = 0;
  for (int n : kRowTiles)
    if (n == 16 || n == forced || !few) most = std::max(most, lay_out(&a, n, sm_count, forced_workers, nullptr));
  return most;
}

void tile_schedule(TileArgs* a) {
  const int mp = knob_value(MLA_KNOB_MIN_PAGES), pc = knob_value(MLA_KNOB_PIECE_COST);
  const int policy = knob_value(MLA_KNOB_SPLIT_POLICY);
  a->granule = a->row_tile == 128 ? 2 : 1;  // pages per step
  a->min_pages = mp > 0 ? mp : a->team ? 1 : 2;
  // A piece costs a pair as much as 10 of its pages, a single CTA, whose stores overlap, as much
  // as one (graph-replayed us at 4 / 7 / 10 / 13 pages: pair, 64 sequences of 128 heads sharing 8,192 tokens
  // 161 / 137 / 146 / 154, 32 sharing 2,000 44 / 37 / 36 / 38; single, at 0 / 1 / 2 / 3, 16
  // heads over 256 windows of 1,021 67.3 / 67.2 / 68.3 / 69.2, over 200 of 4,096 143 / 142 /
  // 148 / 152, 8 sequences of 8 heads behind 4,000 tokens 16.1 / 15.0 / 15.0 / 15.0).
  a->piece_cost = pc > 0 ? std::min(pc - 1, kMaxPieceCost) : a->row_tile == 128 ? 10 : 1;
  // Sequences (or tiles) run whole when splitting them would save less than it costs: to a
  // pair, of R rows in all, 10 + R / 512 pages (a piece more per worker, fp32 partials and
  // their merge; whole / split us: 64 windows of 65 pages for 128 heads 75 / 86, of 1 to 34
  // pages 47 / 53; 16 windows of 66 pages for two queries of 64 heads 59 / 37).
  const int slack = a->row_tile == 128 ? 10 + a->batch * a->rows / 512 : 2;
  a->whole_slack = knob_value(MLA_KNOB_NUM_WORKERS) > 0 || policy == 1 ? -1 : policy == 2 ? 1 << 30 : slack;
}

cudaError_t launch_decode_tile(const TileArgs& a, cudaStream_t stream) {
  const bool shared = a.prefix_len != nullptr;
  cudaError_t e;
  if (a.row_tile == 128) e = launch_decode_tile_pair(a, stream);
  else if (shared) e = a.row_tile == 16 ? launch_tile<16, true>(a, stream) : launch_tile<32, true>(a, stream);
  else e = a.row_tile == 16 ? launch_tile<16, false>(a, stream) : launch_tile<32, false>(a, stream);
  if (e != cudaSuccess || a.team) return e;
  // As many CTAs as run at once; each takes rows until they are done.
  const int R = a.batch * a.rows;
  if (R <= 2 * a.sm_count)
    return shared ? launch_combine_tile<true, 4>(a, R, stream) : launch_combine_tile<false, 4>(a, R, stream);
  const int grid = std::min((R + 3) / 4, 3 * a.sm_count);
  return shared ? launch_combine_tile<true, 1>(a, grid, stream) : launch_combine_tile<false, 1>(a, grid, stream);
}

}  // namespace mla
