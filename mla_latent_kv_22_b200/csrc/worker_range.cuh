// The split schedule, derived inside the decode grid: every CTA computes its worker's
// page range from the sequence lengths (the same arithmetic in every CTA), so no
// separate grid has to run, and be waited for, before the first page load.
//
// The sequences are laid end to end, each as `piece_cost` units of fixed cost followed by
// its pages (an empty sequence takes no units); with W units in all and P workers, worker
// w takes the pages inside units [w q, min((w+1) q, W)), q = max(ceil(W / P), min_pages)
// rounded up to the kernel's page granule.  A piece costs its worker a q' staging, a
// pipeline fill and an epilogue besides its pages, so charging each sequence for one
// evens out workers that hold several short pieces against workers that hold one long
// one (a worker's range also pays at most once for continuing a sequence, the same for
// every worker).  piece_cost = 0 is a split by pages alone.  When there are no more
// sequences than workers and the longest is at most whole_slack pages above the pages-only
// share ceil(pages / P), every sequence instead runs whole on worker b (nearly uniform
// lengths run faster unsplit: a split sequence pays for a piece boundary in its workers
// and for the combine).  CTA c also writes the sequence records (SeqInfo) of the
// sequences b = c, c + gridDim.x, ... that the combine grid reads, and reports their
// invalid lengths.
#pragma once

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

// Pages of sequence b; an invalid length (negative, or beyond the block table) has none.
__device__ __forceinline__ int seq_pages(const int32_t* seqlens, int max_blocks, int b) {
  const int T = seqlens[b];
  return (T < 0 || T > max_blocks * kPage) ? 0 : (T + kPage - 1) / kPage;
}

struct RangeScratch {
  int4 warp_tot[32];  // per warp: pages, units, longest sequence
  int carry;                                    // units before the current pass of the scan
  int total, total_units, maxp;
  WorkerRange rg;
};

// The lengths a schedule is made of, for a batch of plain sequences: pages(b) is the
// page count of sequence b (0 when its length is invalid), bad(b) whether it is invalid.
struct SeqLengths {
  const int32_t* seqlens;
  int max_blocks;
  __device__ __forceinline__ int pages(int b) const { return seq_pages(seqlens, max_blocks, b); }
  // pages(thread) for thread < B, else 0 (called by every thread of the CTA).
  __device__ __forceinline__ int mine(int thread, int B) const { return thread < B ? pages(thread) : 0; }
  __device__ __forceinline__ bool bad(int b) const {
    const int T = seqlens[b];
    return T < 0 || T > max_blocks * kPage;
  }
};

// Called by every thread of the CTA (block-uniform control flow, blockDim.x a multiple
// of 32) with the call's lengths, their number B, worker count P and schedule knobs;
// writes this CTA's share of the records `seq`, and on return rs.rg holds worker w's
// range (b0 < 0: no work).  Not inlined: it runs once per CTA and keeps its registers
// out of the kernel's main loops.
template <class Lengths>
static __device__ __noinline__ void derive_range(const Lengths len, int B, int P, int min_pages, int granule,
                                                 int whole_slack, int piece_cost, SeqInfo* seq, int* err, int w,
                                                 RangeScratch& rs) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  auto owns = [&](int b) { return b % (int)gridDim.x == (int)blockIdx.x; };
  auto units = [&](int n) { return n > 0 ? n + piece_cost : 0; };  // a sequence's share of the layout

  auto share = [&](int total) {
    int q = (total + P - 1) / P;
    if (q < min_pages) q = min_pages;
    if (q < 1) q = 1;
    return (q + granule - 1) & -granule;  // a power of two
  };
  // Sequence b with n pages whose first unit is st occupies units [st, st + units(n)); its
  // pages sit at [pos, pos + n), pos = st + piece_cost, and the next non-empty sequence's
  // pages start at st + units(n) + piece_cost.  With W units in all, worker w's first piece
  // is the sequence whose pages meet its [g0, g1) with st <= g0 (no earlier pages in the
  // range), and its last piece the one whose pages meet it with g1 <= the next sequence's
  // first page: each is written by exactly one thread.
  auto place = [&](int b, int n, int st, int W, long long g0, long long g1) {
    const int pos = st + (n > 0 ? piece_cost : 0);  // its first page in the layout
    if (n > 0 && g0 < W && max(g0, (long long)pos) < min(g1, (long long)pos + n)) {
      if (g0 >= st) {
        rs.rg.b0 = b;
        rs.rg.p0 = (int)(max(g0, (long long)pos) - pos);
      }
      if (g1 <= (long long)pos + n + piece_cost) {
        rs.rg.b1 = b;
        rs.rg.p1 = (int)(min(g1, (long long)pos + n) - pos);
      }
    }
  };
  // Its record, with q units per worker.
  auto record = [&](int b, int n, bool bad, int st, int q) {
    if (bad) set_device_error(err, MLA_ERR_DEVICE_BAD_PAGE);
    const int pos = st + (n > 0 ? piece_cost : 0);
    SeqInfo si;
    si.first_worker = pos / q;
    si.num_pieces = bad ? -1 : (n > 0 ? (pos + n - 1) / q - pos / q + 1 : 0);
    // The first piece is its worker's first piece iff no earlier pages fall in that
    // worker's units (its range starts at or after st); every later piece starts its
    // worker's range.
    si.first_slot = si.first_worker * q >= st ? si.first_worker : P + si.first_worker;
    seq[b] = si;
  };

  // 0. As many threads as sequences: one read of the lengths, one exchange between warps
  // (2.0 -> 1.1 us at one sequence and 256, most of it the read).
  if (B <= (int)blockDim.x) {
    const int n = len.mine(tid, B);
    const bool bad = tid < B && len.bad(tid);
    const int u = units(n);
    int x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int wsum = __reduce_add_sync(0xffffffffu, n), wmax = __reduce_max_sync(0xffffffffu, n);
    if (lane == 31) rs.warp_tot[warp] = make_int4(wsum, x, wmax, 0);
    if (tid == 0) rs.rg = WorkerRange{-1, 0, -1, 0};
    __syncthreads();
    const int4 t = lane < nw ? rs.warp_tot[lane] : make_int4(0, 0, 0, 0);
    const int total = __reduce_add_sync(0xffffffffu, t.x), W = __reduce_add_sync(0xffffffffu, t.y);
    const int maxp = __reduce_max_sync(0xffffffffu, t.z);
    const int st = __reduce_add_sync(0xffffffffu, lane < warp ? t.y : 0) + x - u;  // the sequence's first unit
    const int q = share(W);
    const bool whole = whole_slack >= 0 && B <= P && maxp <= share(total) + whole_slack;
    if (whole) {
      if (tid == w && n > 0) rs.rg = WorkerRange{w, 0, w, n};
    } else {
      const long long g0 = (long long)w * q;
      place(tid, n, st, W, g0, min(g0 + q, (long long)W));
    }
    __syncthreads();
    // The records are for the next grid: nothing here waits for them.
    if (tid < B && owns(tid)) {
      if (!whole) {
        record(tid, n, bad, st, q);
      } else {
        if (bad) set_device_error(err, MLA_ERR_DEVICE_BAD_PAGE);
        seq[tid] = SeqInfo{tid, bad ? -1 : (n > 0 ? 1 : 0), tid};
      }
    }
    return;
  }

  // 1. Total pages, total units and the longest sequence.
  long long sum = 0, wsum = 0;
  int mx = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    const int n = len.pages(b);
    sum += n;
    wsum += units(n);
    mx = max(mx, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) {
    rs.warp_tot[warp] = make_int4((int)sum, (int)wsum, mx, 0);
  }
  if (tid == 0) {
    rs.carry = 0;
    rs.rg = WorkerRange{-1, 0, -1, 0};
  }
  __syncthreads();
  if (tid == 0) {
    int s = 0, u = 0, m = 0;
    for (int i = 0; i < nw; ++i) {
      s += rs.warp_tot[i].x;
      u += rs.warp_tot[i].y;
      m = max(m, rs.warp_tot[i].z);
    }
    rs.total = s;
    rs.total_units = u;
    rs.maxp = m;
  }
  __syncthreads();
  if (whole_slack >= 0 && B <= P && rs.maxp <= share(rs.total) + whole_slack) {
    // 2a. One whole sequence per worker.
    if (tid == 0 && w < B) {
      const int n = len.pages(w);
      if (n > 0) rs.rg = WorkerRange{w, 0, w, n};
    }
    for (int b = tid; b < B; b += blockDim.x) {
      if (!owns(b)) continue;
      const bool bad = len.bad(b);
      if (bad) set_device_error(err, MLA_ERR_DEVICE_BAD_PAGE);
      seq[b] = SeqInfo{b, bad ? -1 : (len.pages(b) > 0 ? 1 : 0), b};
    }
    __syncthreads();
    return;
  }

  // 2b. Exclusive prefix sum of units, blockDim.x sequences per pass.
  const int W = rs.total_units;
  const int q = share(W);
  const long long g0 = (long long)w * q, g1 = min(g0 + q, (long long)W);
  for (int base = 0; base < B; base += blockDim.x) {
    const int b = base + tid;
    const int n = b < B ? len.pages(b) : 0;
    const int u = units(n);
    int x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) rs.warp_tot[warp].x = x;
    __syncthreads();
    int before = rs.carry;
    for (int i = 0; i < warp; ++i) before += rs.warp_tot[i].x;
    const int st = before + x - u;  // first unit of sequence b
    if (b < B) {
      place(b, n, st, W, g0, g1);
      if (owns(b)) record(b, n, len.bad(b), st, q);
    }
    __syncthreads();
    if (tid == blockDim.x - 1) rs.carry = st + u;
    __syncthreads();
  }
}

// The schedule of a batch of plain sequences.
static __device__ __forceinline__ void derive_worker_range(const int32_t* seqlens, int B, int max_blocks, int P,
                                                           int min_pages, int granule, int whole_slack, int piece_cost,
                                                           SeqInfo* seq, int* err, int w, RangeScratch& rs) {
  derive_range(SeqLengths{seqlens, max_blocks}, B, P, min_pages, granule, whole_slack, piece_cost, seq, err, w, rs);
}

}  // namespace mla
