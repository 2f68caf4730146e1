// The tasks of a window or shared-prefix decode (TileArgs in mla_internal.h): their lengths
// for the split schedule, their pages, rows and masks, and the launch, shared by
// decode_tile.cu (one CTA per worker) and decode_tile_pair.cu (a CTA pair).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "worker_range.cuh"

namespace mla {

// Brings a launch's parameters into the constant cache while the previous grid ends.
__device__ __forceinline__ void warm_params(const TileArgs& a, int tid) {
  if (tid < (int)(sizeof(TileArgs) / 4)) {
    const int v = reinterpret_cast<const int*>(&a)[tid];
    asm volatile("" ::"r"(v));
  }
}

// ---------------------------------------------------------------- tasks
// The pages of a task: page p of its list is page real(p) of its table; the first `ns`
// hold the sinks, the rest run from the window's first page to the last.
struct Span {
  int T, n, ns, skip;
  int hole0, hole1;  // tokens [hole0, hole1) are in no query's sight (between sinks and window)
  __device__ __forceinline__ int real(int p) const { return p < ns ? p : p + skip; }
};

__device__ __forceinline__ Span window_span(const TileArgs& a, int T) {
  Span s{T, 0, 0, 0, 0, 0};
  if (T <= 0 || T > a.max_blocks * kPage) return s;
  const int first = max(0, T - a.s_q - a.window + 1);
  const int sinks = min(a.sinks, T);
  s.ns = (sinks + kPage - 1) / kPage;
  s.skip = max(0, first / kPage - s.ns);
  s.n = (T + kPage - 1) / kPage - s.skip;
  s.hole0 = sinks;
  s.hole1 = first;
  return s;
}

template <bool kShared>
struct TaskLengths {
  const TileArgs* a;
  __device__ __forceinline__ int raw(int t) const {
    if (!kShared) return a->seqlens[t];
    return t < a->tiles ? *a->prefix_len : a->seqlens[(t - a->tiles) / a->groups];
  }
  __device__ __forceinline__ int cap(int t) const { return kShared && t < a->tiles ? a->prefix_blocks : a->max_blocks; }
  __device__ __forceinline__ bool bad(int t) const {
    const int T = raw(t);
    return T < 0 || T > cap(t) * kPage;
  }
  __device__ __forceinline__ int pages(int t) const {
    const int T = raw(t);
    if (!kShared) return window_span(*a, T).n;
    return (T < 0 || T > cap(t) * kPage) ? 0 : (T + kPage - 1) / kPage;
  }
};

struct Task {
  Span s;
  const int32_t* table;  // null: page = base + real
  int base;
  int row0, live;  // first query row of the whole batch's, rows of the tile
  int srow;        // row0 within its sequence (window, own tokens)
};

template <int N, bool kShared>
__device__ __forceinline__ Task load_task(const TileArgs& a, int t, int g) {
  Task k;
  k.base = 0;
  if (kShared && t < a.tiles) {
    const int T = *a.prefix_len;
    k.s = Span{T, (T + kPage - 1) / kPage, (T + kPage - 1) / kPage, 0, 0, 0};
    k.table = a.prefix_table;
    k.row0 = t * N;
    k.live = min(N, a.batch * a.rows - k.row0);
    k.srow = 0;
    return k;
  }
  const int b = kShared ? (t - a.tiles) / a.groups : t;
  if (kShared) g = (t - a.tiles) % a.groups;
  const int T = a.seqlens[b];
  k.s = kShared ? Span{T, (T + kPage - 1) / kPage, (T + kPage - 1) / kPage, 0, 0, 0} : window_span(a, T);
  k.table = a.block_table ? a.block_table + (size_t)b * a.max_blocks : nullptr;
  k.base = b * a.max_blocks;
  k.srow = g * N;
  k.row0 = b * a.rows + k.srow;
  k.live = min(N, a.rows - k.srow);
  return k;
}

struct Piece {
  int t, pa, pe;
};

// Iterates the pieces of a worker's range in schedule order.
template <bool kShared>
struct PieceIter {
  WorkerRange rg;
  int t;
  __device__ explicit PieceIter(const volatile WorkerRange& r) : rg{r.b0, r.p0, r.b1, r.p1}, t(r.b0) {}
  __device__ bool next(Piece& pc, const TileArgs& a) {
    if (rg.b0 < 0) return false;
    const TaskLengths<kShared> len{&a};
    while (t <= rg.b1) {
      const int cur = t++;
      const int pa = cur == rg.b0 ? rg.p0 : 0;
      const int pe = cur == rg.b1 ? rg.p1 : len.pages(cur);
      if (pa < pe) {
        pc = {cur, pa, pe};
        return true;
      }
    }
    return false;
  }
};

// Where a piece's results go: out / lse (direct), or a partial's storage; row0 is the row of
// either that the tile's row 0 takes.
struct PieceOut {
  bool direct;
  size_t row0;
};

template <int N, bool kShared>
__device__ __forceinline__ PieceOut piece_out(const TileArgs& a, const Task& k, const Piece& pc, const WorkerRange& rg, int w,
                                              int grp) {
  if (pc.pa == 0 && pc.pe == k.s.n) {
    if (!kShared) return {true, (size_t)k.row0};
    return {false, (size_t)2 * a.num_workers * N + (pc.t < a.tiles ? 0 : a.batch * a.rows) + k.row0};
  }
  const size_t slot = pc.t == rg.b0 ? w : a.num_workers + w;
  return {false, (kShared ? slot : slot * a.groups + grp) * N};
}

// A loading warp's walk over its worker's pages.  The next piece's task and first page ids
// are read (look) while the current piece loads, so that a piece starts without waiting for
// its table.
template <int N, bool kShared>
struct PieceLoads {
  const TileArgs& a;
  const int grp, np, lane;
  PieceIter<kShared> it;
  Piece pc, nc;
  Task k, nk;
  int ids, nids, at;  // lane l holds the id of list page at + l
  bool have, fresh, bad;

  __device__ PieceLoads(const TileArgs& args, const volatile WorkerRange& rg, int g, int num_pages, int l)
      : a(args), grp(g), np(num_pages), lane(l), it(rg) {
    look();
  }
  __device__ __forceinline__ int id(const Task& t, const Piece& p, int pp) const {
    return pp < p.pe ? (t.table ? t.table[t.s.real(pp)] : t.base + t.s.real(pp)) : 0;
  }
  __device__ __forceinline__ void look() {
    have = it.next(nc, a);
    if (!have) return;
    nk = load_task<N, kShared>(a, nc.t, grp);
    nids = id(nk, nc, nc.pa + lane);
  }
  // The piece looked up last becomes the current one.
  __device__ __forceinline__ bool next() {
    if (!have) return false;
    pc = nc;
    k = nk;
    ids = nids;
    at = pc.pa;
    fresh = true;
    bad = have = false;
    return true;
  }
  // First row of list page p; a page id outside the cache gives the row that reads zeros,
  // the error, and `bad` for the rest of the piece.
  __device__ __forceinline__ int row(int p) {
    if (p >= pc.pe) return np * kPage;
    if (p >= at + 32) {
      at = p;
      ids = id(k, pc, p + lane);
      fresh = true;
    }
    if (fresh) {
      fresh = false;
      if (__any_sync(0xffffffffu, (unsigned)ids >= (unsigned)np)) {
        if ((unsigned)ids >= (unsigned)np) set_device_error(a.err, MLA_ERR_DEVICE_BAD_PAGE);
        bad = true;
      }
    }
    const int v = __shfl_sync(0xffffffffu, ids, p - at);
    return (unsigned)v < (unsigned)np ? v * kPage : np * kPage;
  }
};

// Whether some row of table page `real` is in no query's sight.
__device__ __forceinline__ bool page_dirty(const Span& s, int real) {
  const int t0 = real * kPage;
  return s.T < t0 + kPage || (max(s.hole0, t0) < min(s.hole1, t0 + kPage));
}

// Bits [0, x) of a word.
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

// A launch as a programmatic dependent of the grid before it on the stream.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem, cudaStream_t stream,
                             const Args&... args) {
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

// The cache and q' as [9 blocks of 64 dims][rows][64 dims]: one box takes several blocks of
// the same rows (a half page: 4, its rope: 1, q': q_blocks of q_rows rows), each landing as a
// 128B-swizzled tile.  Every box starts at the beginning of a block.
inline bool tile_maps(const TileArgs& a, int q_rows, int q_blocks, CUtensorMap* kv_map, CUtensorMap* rope_map, CUtensorMap* q_map) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  const cuuint64_t strides[2] = {(cuuint64_t)kDQK * 2, 128};
  const cuuint64_t kv_rows = (cuuint64_t)(a.block_table ? a.num_pages : a.batch * a.max_blocks) * kPage;
  auto map = [&](CUtensorMap* m, const __nv_bfloat16* p, cuuint64_t rows, cuuint32_t box_rows, cuuint32_t box_blocks) {
    const cuuint64_t dims[3] = {64, rows, 9};
    const cuuint32_t box[3] = {64, box_rows, box_blocks};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return map(kv_map, a.kv, kv_rows, kPage, 4) && map(rope_map, a.kv, kv_rows, kPage, 1) &&
         map(q_map, a.q, (cuuint64_t)a.batch * a.rows, q_rows, q_blocks);
}

}  // namespace mla
