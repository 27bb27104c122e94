// The merge of a sequence's pieces after the decode over the 8-bit cache:
//   lse = log sum_k exp(lse_k),   out = sum_k exp(lse_k - lse) out_k
// in the order of the pieces.  Sequences in one piece were written by the decode;
// those in none (length 0) get out = 0 and lse = -inf.
//
// Bound by the chain of its loads (pieces' bounds, then lse and values together,
// then the store) and by cold code on small batches, by L2 on large ones.  Its part
// of a call (ten in a graph): 16 heads, 16 sequences in ten pieces each 4.5 us (256
// rows, 5 MB); 60 rows, 37 sequences 3.7 (6.3 with the merge of the bf16 decode); 128
// heads, 128 sequences, most in two pieces 5.9 (57 MB).
#include <cuda_bf16.h>

#include "mla_kv8_internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kInFlight = 8;  // 16-byte loads of a thread

// Of differences of lse, where what is large does not count.
__device__ __forceinline__ float exp_of(float x) { return ex2_approx(x * 1.4426950408889634f); }

// kWarps of a block of four take a row, each thread 4 / kWarps vectors of it.
template <int kWarps>
__global__ void __launch_bounds__(kThreads) mla_kv8_merge_kernel(const CombineParams P) {
  constexpr int kVecs = 4 / kWarps, kAhead = kInFlight / kVecs, kFew = kWarps == 4 ? 4 : 2;
  grid_dependency_wait();  // the decode's partial results are complete
  // The next call's set-up may start (small batches: 8.5 -> 7.9, 15.4 -> 14.8 us a call
  // one after another; on large ones it takes room from this kernel: 125.7 -> 127.1).
  if (kWarps == 4) grid_launch_dependents();
  const int i = blockIdx.x;
  const int rows = P.s_q * P.h_q;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * (4 / kWarps) + warp / kWarps;
  if (row >= rows) return;
  const int s0 = __ldg(P.num_splits + i), ns = __ldg(P.num_splits + i + 1) - s0;
  if (ns == 1) return;
  const float* const lse_of = P.ws_lse + static_cast<int64_t>(s0) * rows + row;
  const float4* const src = static_cast<const float4*>(P.ws_o) + (static_cast<int64_t>(s0) * rows + row) * (kDimV / 4) +
                            warp % kWarps * 32 + lane;
  const int64_t piece = static_cast<int64_t>(rows) * (kDimV / 4);
  float4 x[kAhead][kVecs];
  auto load = [&](int k0, int n) {
#pragma unroll
    for (int a = 0; a < n; ++a)
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        x[a][v] = k0 + a < ns ? src[(k0 + a) * piece + v * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 acc[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int a, float w) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      acc[v].x += w * x[a][v].x;
      acc[v].y += w * x[a][v].y;
      acc[v].z += w * x[a][v].z;
      acc[v].w += w * x[a][v].w;
    }
  };
  float lse = -INFINITY;
  if (ns <= kFew) {  // each thread makes the weights; little code, for it comes cold
    float e[kFew], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int a = 0; a < kFew; ++a) e[a] = a < ns ? lse_of[static_cast<int64_t>(a) * rows] : -INFINITY;
    load(0, kFew);
#pragma unroll
    for (int a = 0; a < kFew; ++a) top = fmaxf(top, e[a]);
    if (top != -INFINITY) {
#pragma unroll
      for (int a = 0; a < kFew; ++a) sum += e[a] = exp_of(e[a] - top);
      lse = top + logf(sum);
      const float inv = 1.f / sum;
#pragma unroll
      for (int a = 0; a < kFew; ++a) add(a, e[a] * inv);
    }
  } else {  // a lane has the weights of pieces lane, lane + 32, ...
    const float mine = lane < ns ? lse_of[static_cast<int64_t>(lane) * rows] : -INFINITY;
    load(0, kAhead);
    float top = mine;
    for (int k = lane + 32; k < ns; k += 32) top = fmaxf(top, lse_of[static_cast<int64_t>(k) * rows]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (top != -INFINITY) {
      float sum = lane < ns ? exp_of(mine - top) : 0.f;
      for (int k = lane + 32; k < ns; k += 32) sum += exp_of(lse_of[static_cast<int64_t>(k) * rows] - top);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      lse = top + logf(sum);
      float weight = exp_of(mine - lse);
      for (int k0 = 0; k0 < ns; k0 += kAhead) {
        if (k0 > 0) {
          load(k0, kAhead);
          if (k0 % 32 == 0) weight = k0 + lane < ns ? exp_of(lse_of[static_cast<int64_t>(k0 + lane) * rows] - lse) : 0.f;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) add(a, __shfl_sync(0xffffffffu, weight, (k0 + a) & 31));
      }
    }
  }
  uint2* const dst = static_cast<uint2*>(P.out) + (static_cast<int64_t>(i) * rows + row) * (kDimV / 4) + warp % kWarps * 32 + lane;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) dst[v * 32] = make_uint2(pack_bf16x2(acc[v].x, acc[v].y), pack_bf16x2(acc[v].z, acc[v].w));
  if (lane == 0 && warp % kWarps == 0) {
    const int j = row / P.h_q;
    P.lse[(static_cast<int64_t>(i) * P.h_q + row - j * P.h_q) * P.s_q + j] = lse;
  }
}

}  // namespace

cudaError_t launch_merge_kv8(const CombineParams& p, cudaStream_t stream) {
  // Where a sequence has many pieces a row's four warps keep them all in flight, with
  // one or two a warp does: 16 sequences over 152 parts 15.4 us a call with four warps,
  // 19.5 with one; 37 over 76 25.3 and 25.8; 128 over 76 130.7 and 125.0.
  // (A grid's second dimension ends at 65535, the rows that a call may have at four times that.)
  const int rows = p.s_q * p.h_q;
  const bool many = p.num_parts >= 2 * static_cast<int64_t>(p.b) && rows <= 65535;
  const int each = many ? 1 : 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.b, (rows + each - 1) / each, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, mla_kv8_merge_kernel<4>, p) : cudaLaunchKernelEx(&cfg, mla_kv8_merge_kernel<1>, p);
}

}  // namespace mla
