// Cache append with position rotation: new tokens' rows [c_kv | R(pos) k_rope] into the
// paged latent cache, and R(pos) q_rope of the same tokens, in one launch.
//
// R(pos) turns pair i (of 32) of a 64-wide rope vector by the angle whose cosine and sine
// the caller's table holds at (pos, i): (a, b) -> (a c - b s, a s + b c), in fp32 and
// rounded once to bf16.  Pair i is dims (2i, 2i + 1) or, half-split, (i, i + 32).
//
// Bound by HBM: every input is read and every output written once (36 KB per token with
// 128 heads, of which the query part is 32 KB), with no arithmetic to speak of.  One block
// per token.  A thread keeps a quarter of its token's row of the table (8 pairs: 16 fp32
// values) and applies it to the same pairs of every 32nd head; all of a thread's loads are
// issued before the token's sequence, position and page are looked up, so the chain lengths
// -> page -> store hides behind them.
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerPass = kThreads / 4;  // four threads per head
constexpr int kPasses = MLA_MAX_HEADS / kHeadsPerPass;

// The 16-byte chunks of a 64-wide vector that hold pairs [8j, 8j + 8).
template <bool kInter>
__device__ __forceinline__ int chunk0(int j) { return kInter ? 2 * j : j; }
template <bool kInter>
__device__ __forceinline__ int chunk1(int j) { return kInter ? 2 * j + 1 : j + 4; }

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// The two chunks of pairs [8j, 8j + 8) turned in place.
template <bool kInter>
__device__ __forceinline__ void turn(uint4& x0, uint4& x1, const float (&c)[8], const float (&s)[8]) {
  uint32_t v[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  if (kInter) {  // word i of the eight is pair i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = unpack_bf16x2(v[i]);
      v[i] = pack_bf16x2(p.x * c[i] - p.y * s[i], p.x * s[i] + p.y * c[i]);
    }
  } else {  // first halves in words 0-3, second halves in words 4-7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack_bf16x2(v[i]), b = unpack_bf16x2(v[4 + i]);
      v[i] = pack_bf16x2(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
      v[4 + i] = pack_bf16x2(a.x * s[2 * i] + b.x * c[2 * i], a.y * s[2 * i + 1] + b.y * c[2 * i + 1]);
    }
  }
  x0 = make_uint4(v[0], v[1], v[2], v[3]);
  x1 = make_uint4(v[4], v[5], v[6], v[7]);
}

template <bool kInter>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  const int n = blockIdx.x, tid = threadIdx.x, j = tid & 3, h0 = tid >> 2;

  // Loads of the token's data.
  uint4 lat = make_uint4(0, 0, 0, 0), k0 = lat, k1 = lat, q0[kPasses], q1[kPasses];
  if (tid < kDLatent / 8) lat = reinterpret_cast<const uint4*>(a.c_kv + n * a.ckv_stride)[tid];
  if (tid >= kThreads - 4) {
    const uint4* src = reinterpret_cast<const uint4*>(a.k_rope + n * a.krope_stride);
    k0 = src[chunk0<kInter>(j)];
    k1 = src[chunk1<kInter>(j)];
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int h = h0 + p * kHeadsPerPass;
    if (a.q_rope && h < a.heads) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q_rope + n * a.q_stride_n + h * a.q_stride_h);
      q0[p] = src[chunk0<kInter>(j)];
      q1[p] = src[chunk1<kInter>(j)];
    }
  }

  // The token's sequence: the last one starting at or before it (empty ones start where the
  // next does).  Counted by the whole block, so it takes one round of loads per 128 sequences.
  int b, end;
  if (a.cu_tokens) {
    b = -1;
    for (int i0 = 0; i0 <= a.batch; i0 += kThreads)
      b += __syncthreads_count(i0 + tid <= a.batch && a.cu_tokens[i0 + tid] <= n);
    if (b < 0 || b >= a.batch) return;  // a padding token: nothing is written for it
    end = a.cu_tokens[b + 1];
    if (a.cu_tokens[b] > n || end <= n) return;
  } else {
    const int each = a.tokens / a.batch;
    b = n / each;
    end = (b + 1) * each;
  }
  const int T = a.seqlens[b];
  const int row = T - (end - n);  // its row of the sequence
  const long long pos = (long long)row + (a.pos_offset ? a.pos_offset[b] : 0);
  int code = 0;
  long long slot = 0;
  if (T < 0 || T > a.max_blocks * kPage || row < 0) {
    code = MLA_ERR_DEVICE_BAD_PAGE;
  } else if (pos < 0 || pos >= a.max_pos) {
    code = MLA_ERR_DEVICE_BAD_POSITION;
  } else if (a.block_table) {
    const int id = a.block_table[(size_t)b * a.max_blocks + row / kPage];
    if ((unsigned)id >= (unsigned)a.num_pages) code = MLA_ERR_DEVICE_BAD_PAGE;
    slot = (long long)id * kPage + row % kPage;
  } else {
    slot = (long long)b * a.max_blocks * kPage + row;
  }
  float c[8], s[8];
  if (code == 0) {
    const float4* t = reinterpret_cast<const float4*>(a.cos_sin + pos * kDRope);
    *reinterpret_cast<float4*>(c) = t[2 * j];
    *reinterpret_cast<float4*>(c + 4) = t[2 * j + 1];
    *reinterpret_cast<float4*>(s) = t[8 + 2 * j];
    *reinterpret_cast<float4*>(s + 4) = t[8 + 2 * j + 1];
    uint4* dst = reinterpret_cast<uint4*>(a.kv + slot * kDQK);
    if (tid < kDLatent / 8) dst[tid] = lat;
    if (tid >= kThreads - 4) {
      turn<kInter>(k0, k1, c, s);
      dst[kDLatent / 8 + chunk0<kInter>(j)] = k0;
      dst[kDLatent / 8 + chunk1<kInter>(j)] = k1;
    }
  } else if (tid == 0) {
    set_device_error(a.err, code);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int h = h0 + p * kHeadsPerPass;
    if (a.q_rope && h < a.heads) {
      if (code == 0) turn<kInter>(q0[p], q1[p], c, s);
      else q0[p] = q1[p] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + n * a.qo_stride_n + h * a.qo_stride_h);
      dst[chunk0<kInter>(j)] = q0[p];
      dst[chunk1<kInter>(j)] = q1[p];
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, bool interleaved, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.tokens, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return interleaved ? cudaLaunchKernelEx(&cfg, append_kernel<true>, a) : cudaLaunchKernelEx(&cfg, append_kernel<false>, a);
}

}  // namespace mla
