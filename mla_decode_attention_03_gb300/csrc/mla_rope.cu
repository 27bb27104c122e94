// Rotary positions of query and key rows.
//
// Pair i of a row at position p turns by 2 pi p f_i.  f_i comes in as 64-bit
// fixed-point turns, so p * f_i is one wrapping integer product whose overflow
// drops whole turns: the remainder is off by p * 2^-65 turns at most at any position,
// and its sine and cosine are taken in fp32 of an angle inside [-pi, pi).
// (A product in fp32 is off by 0.03 rad at position 10^6.)
//
// A block takes kThreads / units consecutive rows of the (token, head) order,
// where a unit is two 16-byte vectors: the same pairs' u and v.  It makes the
// sines of its tokens once, in shared memory, while its loads are in flight.
// Bound by HBM on long inputs: 8191 tokens of 32 heads and a key, 64 of 192 values
// a row into rows of 576, 69 MB: 13.2 us (5.2 TB/s); with blocks of 256 threads 13.6.
// 128 tokens of 128 heads: 3.1 us.  (Of ten calls in a graph; the 69 MB lie in L2.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mla_kv8_internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = kRopeThreads;

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// kPairs pairs of a row (from pair i0): element indexes of u and v
template <typename T, bool kInterleaved, bool kPos64, bool kVec>
__global__ void __launch_bounds__(kThreads) mla_rope_kernel(const RopeParams P, int units, int rows_per_block) {
  constexpr int kPairs = 16 / sizeof(T);  // per unit
  extern __shared__ float2 table[];       // [tokens of the block][pairs]: gain * (cos, sin)
  const int per_token = P.heads + P.k_heads;
  const int64_t rows = P.tokens * per_token;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_block;
  // the block's first token; the division in 32 bits where that is enough
  const int64_t t0 = (r0 >> 32) ? r0 / per_token : static_cast<uint32_t>(r0) / static_cast<uint32_t>(per_token);
  const int skip = static_cast<int>(r0 - t0 * per_token);
  const int block_rows = static_cast<int>(min(static_cast<int64_t>(rows_per_block), rows - r0));
  const int block_tokens = (skip + block_rows - 1) / per_token + 1;

  const int lr = threadIdx.x / units;
  const int i0 = (threadIdx.x - lr * units) * kPairs;
  const bool live = lr < block_rows;
  const int tt = live ? (skip + lr) / per_token : 0;  // of the block's tokens
  const int head = live ? skip + lr - tt * per_token : 0;
  const int64_t t = t0 + tt;
  const bool is_k = head >= P.heads;
  const RopeRows& R = is_k ? P.k : P.x;
  const int hh = is_k ? head - P.heads : head;
  const T* const src = static_cast<const T*>(R.src) + t * R.src_token + hh * R.src_head;
  T* const dst = static_cast<T*>(R.dst) + t * R.dst_token + hh * R.dst_head;
  const int n = min(kPairs, P.pairs - i0);

  alignas(16) T a[kPairs], b[kPairs];  // interleaved: 2 kPairs consecutive values; halves: the u's and the v's
  const int ia = kInterleaved ? 2 * i0 : i0;
  const int ib = kInterleaved ? 2 * i0 + kPairs : P.pairs + i0;
  if (live) {
    if (kVec) {
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(src + ia);
      *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(src + ib);
    } else {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const bool in_a = kInterleaved ? ia + e < 2 * P.pairs : e < n;
        const bool in_b = kInterleaved ? ib + e < 2 * P.pairs : e < n;
        a[e] = in_a ? src[ia + e] : from_f<T>(0.f);
        b[e] = in_b ? src[ib + e] : from_f<T>(0.f);
      }
    }
  }

  const int entries = block_tokens * P.pairs;
  for (int k = threadIdx.x; k < entries; k += kThreads) {
    const int kt = k / P.pairs, i = k - kt * P.pairs;
    const uint64_t pos = kPos64 ? static_cast<uint64_t>(static_cast<const int64_t*>(P.positions)[t0 + kt])
                                : static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(P.positions)[t0 + kt]));
    // turns in [-1/2, 1/2) as a 64-bit fraction; half-turns in fp32
    const float half_turns = static_cast<float>(static_cast<int64_t>(pos * P.turns[i])) * 0x1p-63f;
    float s, c;
    sincospif(half_turns, &s, &c);
    table[k] = make_float2(P.gain * c, P.inverse ? -P.gain * s : P.gain * s);
  }
  __syncthreads();
  if (!live) return;

  const float2* const cs = table + tt * P.pairs + i0;
  if (kInterleaved) {
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      if (!kVec && e >= n) break;
      T& ru = (2 * e < kPairs) ? a[2 * e < kPairs ? 2 * e : 0] : b[2 * e < kPairs ? 0 : 2 * e - kPairs];
      T& rv = (2 * e < kPairs) ? a[2 * e < kPairs ? 2 * e + 1 : 0] : b[2 * e < kPairs ? 0 : 2 * e + 1 - kPairs];
      const float u = to_f(ru), v = to_f(rv);
      ru = from_f<T>(u * cs[e].x - v * cs[e].y);
      rv = from_f<T>(u * cs[e].y + v * cs[e].x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      if (!kVec && e >= n) break;
      const float u = to_f(a[e]), v = to_f(b[e]);
      a[e] = from_f<T>(u * cs[e].x - v * cs[e].y);
      b[e] = from_f<T>(u * cs[e].y + v * cs[e].x);
    }
  }
  if (kVec) {
    *reinterpret_cast<uint4*>(dst + ia) = *reinterpret_cast<const uint4*>(a);
    *reinterpret_cast<uint4*>(dst + ib) = *reinterpret_cast<const uint4*>(b);
  } else {
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      if (kInterleaved ? ia + e < 2 * P.pairs : e < n) dst[ia + e] = a[e];
      if (kInterleaved ? ib + e < 2 * P.pairs : e < n) dst[ib + e] = b[e];
    }
  }
}

template <typename T, bool kInterleaved, bool kPos64>
cudaError_t launch(const RopeParams& p, bool vec, cudaStream_t stream) {
  constexpr int kPairs = 16 / sizeof(T);
  const int units = (p.pairs + kPairs - 1) / kPairs;
  const int64_t rows = p.tokens * (p.heads + p.k_heads);
  const int rows_per_block = kThreads / units;
  const int per_token = p.heads + p.k_heads;
  const int tokens = (rows_per_block + per_token - 2) / per_token + 1;  // most tokens that a block's rows touch
  const int smem = tokens * p.pairs * static_cast<int>(sizeof(float2));
  const unsigned grid = static_cast<unsigned>((rows + rows_per_block - 1) / rows_per_block);
  if (vec)
    mla_rope_kernel<T, kInterleaved, kPos64, true><<<grid, kThreads, smem, stream>>>(p, units, rows_per_block);
  else
    mla_rope_kernel<T, kInterleaved, kPos64, false><<<grid, kThreads, smem, stream>>>(p, units, rows_per_block);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const RopeParams& p, bool interleaved, bool pos64, bool vec, cudaStream_t stream) {
  if (interleaved) return pos64 ? launch<T, true, true>(p, vec, stream) : launch<T, true, false>(p, vec, stream);
  return pos64 ? launch<T, false, true>(p, vec, stream) : launch<T, false, false>(p, vec, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, bool interleaved, bool pos64, bool vec, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  if (dtype == 0) return pick<__nv_bfloat16>(p, interleaved, pos64, vec, stream);
  if (dtype == 1) return pick<__half>(p, interleaved, pos64, vec, stream);
  return pick<float>(p, interleaved, pos64, vec, stream);
}

}  // namespace mla
