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
// Window: a task is a sequence; page p of its list is page real(p) of its table; the first
// `ns` hold the sinks, the rest run from the window's first page to the last.
// Shared prefix: a task is a tile of query rows of the whole batch; its list holds the
// prefix's pages, then the own pages of each sequence that has rows in the tile (a page of
// one sequence is hidden from the others' rows).
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

__device__ __forceinline__ bool bad_length(int T, int blocks) { return T < 0 || T > blocks * kPage; }
__device__ __forceinline__ int own_pages(const TileArgs& a, int b) { return seq_pages(a.seqlens, a.max_blocks, b); }
__device__ __forceinline__ int prefix_pages(const TileArgs& a) { return seq_pages(a.prefix_len, a.prefix_blocks, 0); }
// The first and last sequence with rows in a tile of the batch.
__device__ __forceinline__ int tile_seq0(const TileArgs& a, int t) { return t * a.row_tile / a.rows; }
__device__ __forceinline__ int tile_seq1(const TileArgs& a, int t) { return (min((t + 1) * a.row_tile, a.batch * a.rows) - 1) / a.rows; }

static __device__ __noinline__ int tile_pages(const TileArgs& a, int t);

template <bool kShared>
struct TaskLengths {
  const TileArgs* a;
  __device__ __forceinline__ bool bad(int t) const {
    return kShared ? bad_length(*a->prefix_len, a->prefix_blocks) : bad_length(a->seqlens[t], a->max_blocks);
  }
  __device__ __forceinline__ int pages(int t) const {
    if constexpr (!kShared) return window_span(*a, a->seqlens[t]).n;
    if (bad(t)) return 0;
    int n = prefix_pages(*a);
    const int b1 = tile_seq1(*a, t);
#pragma unroll 8
    for (int b = tile_seq0(*a, t); b <= b1; ++b) n += own_pages(*a, b);
    return n;
  }
  // pages(thread) for thread < tasks, else 0, by whole warps: a few tiles of many sequences
  // (one of 128 took 11 us by one thread) are counted by a warp each.
  __device__ __forceinline__ int mine(int thread, int tasks) const {
    if (kShared && a->row_tile > 8 * a->rows * tasks) {
      int n = 0;
      for (int j = 0; j < 32 && (thread & ~31) + j < tasks; ++j) {
        const int v = tile_pages(*a, (thread & ~31) + j);
        if ((thread & 31) == j) n = v;
      }
      return n;
    }
    return thread < tasks ? pages(thread) : 0;
  }
};

// Pages of a task, taken by a whole warp together.  (Not inlined, like page_ref_shared: twelve
// warps run six roles, and seldom-run code in their loops costs instruction cache.)
static __device__ __noinline__ int tile_pages(const TileArgs& a, int t) {
  if (bad_length(*a.prefix_len, a.prefix_blocks)) return 0;
  int n = 0;
  const int b1 = tile_seq1(a, t);
#pragma unroll 1
  for (int b = tile_seq0(a, t) + (threadIdx.x & 31); b <= b1; b += 32) n += own_pages(a, b);
  return prefix_pages(a) + __reduce_add_sync(0xffffffffu, n);
}
template <bool kShared>
__device__ __forceinline__ int task_pages(const TileArgs& a, int t) {
  if constexpr (kShared) return tile_pages(a, t);
  else return window_span(a, a.seqlens[t]).n;
}

struct Task {
  // Window: the sequence's span, T and the hole as far as the tile's queries see; shared: the
  // prefix's T (as far as they see) and n alone.
  Span s;
  int b0, b1;      // the sequence; shared: the first and last with rows in the tile
  int row0, live;  // first query row of the whole batch's, rows of the tile
  int srow;        // window: row0 within its sequence
  int cut;         // shared: the last tokens of b1 that none of its queries in the tile sees
};

template <int N, bool kShared>
__device__ __forceinline__ Task load_task(const TileArgs& a, int t, int g) {
  Task k;
  if constexpr (kShared) {
    k.b0 = tile_seq0(a, t);
    k.b1 = tile_seq1(a, t);
    k.row0 = t * N;
    k.live = min(N, a.batch * a.rows - k.row0);
    k.srow = 0;
    k.cut = a.s_q - 1 - (k.row0 + k.live - 1 - k.b1 * a.rows) / a.heads;
    const int P = *a.prefix_len;
    // Every sequence but the last has its last query in the tile, which sees the whole prefix.
    k.s = Span{k.b0 < k.b1 ? P : P + min(a.seqlens[k.b1] - k.cut, 0), prefix_pages(a), 0, 0, 0, 0};
  } else {
    k.srow = g * N;
    k.row0 = t * a.rows + k.srow;
    k.live = min(N, a.rows - k.srow);
    k.s = window_span(a, a.seqlens[t]);
    const int end = k.s.T - a.s_q + 1;  // of query 0
    k.s.hole1 = max(0, end + k.srow / a.heads - a.window);
    k.s.T = end + (k.srow + k.live - 1) / a.heads;
    k.b0 = k.b1 = t;
    k.cut = 0;
  }
  return k;
}

// A page of a task's list: its sequence (-1: the prefix), its index in that table, and the
// tokens of the sequence (or prefix) as far as the tile's queries see.
struct PageRef {
  int seq, page, T;
  __device__ __forceinline__ int valid_rows() const { return min(max(T - page * kPage, 0), kPage); }
};

// Page q of the own pages of sequences b0..b1 for every lane of a warp (each its own q; q < 0:
// page q + prefix of the prefix, whose length is T).
static __device__ __noinline__ PageRef page_ref_shared(const TileArgs& a, int q, int prefix, int T0, int b0, int b1, int cut) {
  const int lane = threadIdx.x & 31;
  PageRef r{-1, q + prefix, T0};
  bool open = q >= 0;
  // 32 sequences at a time: the ends of their pages in the list, and each lane's search.
#pragma unroll 1
  for (; b0 <= b1 && __any_sync(0xffffffffu, open); b0 += 32) {
    const int b = b0 + lane;
    const int T = b <= b1 ? a.seqlens[b] : 0;
    const int n = bad_length(T, a.max_blocks) ? 0 : (T + kPage - 1) / kPage;
    int end = n;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const int total = __shfl_sync(0xffffffffu, end, 31);
    int j = 0;  // the first sequence whose end is above q
#pragma unroll 1
    for (int o = 16; o; o >>= 1)
      if (__shfl_sync(0xffffffffu, end, j + o - 1) <= q) j += o;
    const int first = __shfl_sync(0xffffffffu, end - n, j), Tj = __shfl_sync(0xffffffffu, T, j);
    if (open && q < total) {
      r = PageRef{b0 + j, q - first, Tj - (b0 + j == b1 ? cut : 0)};
      open = false;
    }
    q -= total;
  }
  return r;
}
// Page p of a task's list for every lane of a warp (each its own p, inside the list).
template <bool kShared>
__device__ __forceinline__ PageRef page_ref(const TileArgs& a, const Task& k, int p) {
  if constexpr (kShared) return page_ref_shared(a, p - k.s.n, k.s.n, k.s.T, k.b0, k.b1, k.cut);
  else return {k.b0, k.s.real(p), k.s.T};
}

// What row `row` of a task's tile sees: tokens t < end of its sequence's own (window: all)
// tokens with t < sinks or t >= from; of a shared prefix the tokens t < prefix_end.  `seq` is
// the row's sequence, and `bad` says that its length is invalid.
struct RowSight {
  int seq, end, from, prefix_end;
  bool bad;
};

template <bool kShared>
__device__ __forceinline__ RowSight row_sight(const TileArgs& a, const Task& k, int row) {
  RowSight r{-2, -1, 0, -1, false};  // a row past the tile's sees nothing
  if (row >= k.live) return r;
  r.seq = kShared ? (k.row0 + row) / a.rows : k.b0;
  const int T = a.seqlens[r.seq];
  r.end = T - a.s_q + 1 + (k.row0 + row - r.seq * a.rows) / a.heads;
  if constexpr (kShared) {
    r.bad = bad_length(T, a.max_blocks);
    r.prefix_end = *a.prefix_len + min(r.end, 0);
  } else {
    r.from = r.end - a.window;
  }
  return r;
}

struct Piece {
  int t, pa, pe;
  int n;  // pages of the whole task
};

// Iterates the pieces of a worker's range in schedule order (by a whole warp).
template <bool kShared>
struct PieceIter {
  WorkerRange rg;
  int t;
  __device__ explicit PieceIter(const volatile WorkerRange& r) : rg{r.b0, r.p0, r.b1, r.p1}, t(r.b0) {}
  __device__ __forceinline__ bool next(Piece& pc, const TileArgs& a) {
    if (rg.b0 < 0) return false;
#pragma unroll 1
    while (t <= rg.b1) {
      const int cur = t++, n = task_pages<kShared>(a, cur);
      const int pa = cur == rg.b0 ? rg.p0 : 0;
      const int pe = cur == rg.b1 ? rg.p1 : n;
      if (pa < pe) {
        pc = {cur, pa, pe, n};
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
  if (pc.pa == 0 && pc.pe == pc.n) return {true, (size_t)k.row0};
  const size_t slot = pc.t == rg.b0 ? w : a.num_workers + w;
  return {false, (kShared ? slot : slot * a.groups + grp) * N};
}

// NaN for the rows of all pieces of a worker, one of whose waits ran out: written where the
// piece's results go, or, for a partial, as the lse by which the merge makes its rows NaN.  By the
// whole CTA, when nothing of it writes any more.
template <int N, bool kShared>
static __device__ __noinline__ void spoil_pieces(const TileArgs& a, const volatile WorkerRange& rg, int w, int grp) {
  const int lane = threadIdx.x & 31;
  PieceIter<kShared> it(rg);
  Piece pc;
#pragma unroll 1
  while (it.next(pc, a)) {
    const Task k = load_task<N, kShared>(a, pc.t, grp);
    const PieceOut to = piece_out<N, kShared>(a, k, pc, it.rg, w, grp);
#pragma unroll 1
    for (int row = threadIdx.x >> 5; row < k.live; row += blockDim.x >> 5) {
      if (lane == 0) (to.direct ? a.lse : a.part_lse)[to.row0 + row] = NAN;
      if (to.direct) {
        uint4* o = reinterpret_cast<uint4*>(a.out + (to.row0 + row) * kDLatent) + lane;
        o[0] = o[32] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      }
    }
  }
}

// Whether some row of a page is in no query's sight.
template <bool kShared>
__device__ __forceinline__ bool page_dirty(const Task& k, const PageRef& r) {
  const int t0 = r.page * kPage;
  return r.T < t0 + kPage || (!kShared && max(k.s.hole0, t0) < min(k.s.hole1, t0 + kPage));
}

// Sets bits [r0, r1) of `words` words.
static __device__ __noinline__ void mark_rows(uint32_t* bits, int words, int r0, int r1) {
#pragma unroll 1
  for (int i = 0; i < words; ++i) {
    const int lo = max(r0 - 32 * i, 0), hi = min(r1 - 32 * i, 32);
    if (lo < hi) atomicOr(bits + i, (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u));
  }
}

// A loading warp's walk over its worker's pages, 32 of the list at a time.  The next piece's
// task and first pages are looked up while the current piece loads, so that a piece starts
// without waiting for its table.
template <int N, bool kShared>
struct PieceLoads {
  static constexpr int kWords = (N + 31) / 32;
  const TileArgs& a;
  const int grp, np, lane;
  PieceIter<kShared> it;
  Piece pc, nc;
  Task k, nk;
  int id, nid, at;     // lane l holds the page id of list page at + l,
  PageRef ref, nref;   // and where it stands
  bool have, fresh;

  __device__ PieceLoads(const TileArgs& args, const volatile WorkerRange& rg, int g, int num_pages, int l)
      : a(args), grp(g), np(num_pages), lane(l), it(rg) {
    look();
  }
  __device__ __forceinline__ void read(const Task& t, const Piece& p, int p0, int& id_, PageRef& r) const {
    r = page_ref<kShared>(a, t, min(p0 + lane, p.pe - 1));
    if (kShared && r.seq < 0) id_ = a.prefix_table[r.page];
    else id_ = a.block_table ? a.block_table[(size_t)r.seq * a.max_blocks + r.page] : r.seq * a.max_blocks + r.page;
  }
  __device__ __forceinline__ void look() {
    have = it.next(nc, a);
    if (!have) return;
    nk = load_task<N, kShared>(a, nc.t, grp);
    read(nk, nc, nc.pa, nid, nref);
  }
  // The piece looked up last becomes the current one.
  __device__ __forceinline__ bool next() {
    if (!have) return false;
    pc = nc;
    k = nk;
    id = nid;
    ref = nref;
    at = pc.pa;
    fresh = true;
    have = false;
    return true;
  }
  // First row of list page p and whether the page is dirty; pages past the piece and page
  // ids outside the cache give the row that reads zeros, the latter also the error and, in
  // `bad` (a bit per row of the tile), the rows that see the page.
  __device__ __forceinline__ int row(int p, bool& dirty, uint32_t* bad) {
    dirty = false;
    if (p >= pc.pe) return np * kPage;
    if (p >= at + 32) {
      at = p;
      read(k, pc, p, id, ref);
      fresh = true;
    }
    if (fresh) {
      fresh = false;
      if ((unsigned)id >= (unsigned)np) {
        set_device_error(a.err, MLA_ERR_DEVICE_BAD_PAGE);
        if (bad) {
          const bool all = !kShared || ref.seq < 0;
          mark_rows(bad, kWords, all ? 0 : max(ref.seq * a.rows - k.row0, 0), all ? N : min((ref.seq + 1) * a.rows - k.row0, N));
        }
      }
      __syncwarp();
    }
    dirty = __shfl_sync(0xffffffffu, (int)page_dirty<kShared>(k, ref), p - at) != 0;
    const int v = __shfl_sync(0xffffffffu, id, p - at);
    return (unsigned)v < (unsigned)np ? v * kPage : np * kPage;
  }
  // The first token and the valid rows of list page p, whose row() was just asked for.
  __device__ __forceinline__ void page(int p, int& t0, int& rows) const {
    t0 = __shfl_sync(0xffffffffu, ref.page, p - at) * kPage;
    rows = __shfl_sync(0xffffffffu, ref.valid_rows(), p - at);
  }
};

// Whether a call has pages that some rows of a tile see and others do not: several queries, or
// tiles that hold rows of several sequences.  A hidden token's P is 0 for the rows that do not
// see it, which its values survive only if they are finite: see nonfinite_seen.
template <bool kShared>
__host__ __device__ __forceinline__ bool mixed_pages(const TileArgs& a) {
  return a.s_q > 1 || (kShared && a.rows % a.row_tile != 0);
}

// The tokens (bits) whose score is not finite in a row that sees them: a value that is not
// finite makes its token's score so in every row.  (So does a query: the values themselves
// are looked at, by finite_chunk, before they are taken as zeros.  The rows that see such a
// token have no finite result anyway, or, at a score of -inf, weigh it by 0.)
__device__ __forceinline__ uint32_t nonfinite_seen(const float (&y)[32], uint32_t see) {
  uint64_t z = f2_pack(0.f, 0.f);
  const uint64_t zero = z;
#pragma unroll
  for (int j = 0; j < 32; j += 2) z = f2_fma(f2_pack(y[j], y[j + 1]), zero, z);
  float z0, z1;
  f2_unpack(z, z0, z1);
  uint32_t bits = 0;
  if (z0 + z1 != 0.f) {  // NaN: some score is not finite
#pragma unroll
    for (int j = 0; j < 32; ++j) bits |= isfinite(y[j]) ? 0u : 1u << j;
  }
  return bits & see;
}

// A chunk of eight bf16 values with zeros for those that are not finite.
__device__ __forceinline__ uint4 finite_chunk(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bits [0, x) of a word.
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

// A launch as a programmatic dependent of the grid before it on the stream, in clusters of
// `cluster` CTAs (0: the kernel's own).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem, int cluster, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
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
