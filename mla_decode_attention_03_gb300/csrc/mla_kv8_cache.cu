// Writing new tokens into the 8-bit latent cache, and reading ranges back.
// Both move bytes once: bound by HBM bandwidth on long inputs and by launch
// and load latency on a decode step's few tokens.  Measured, of ten calls in a graph
// (what is written then lies largely in L2): writing 128 tokens 2.0 us, 16001 tokens
// to scattered slots 7.2 us (28 MB: 3.9 TB/s; two tokens a warp were no faster);
// reading 262,000 tokens back 73 us (6.2 TB/s, 0.91 of the copy rate).
#include <cstdint>

#include "mla_kv8_internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kChunks = kDimQK / 8;  // 72 chunks of 8 values: 16 bytes of bf16, 8 bytes of e4m3
constexpr int kWriteWarps = 4;
constexpr int kReadWarps = 4;
constexpr int kReadRows = 8;         // rows per warp: 8 x 72 chunks = 18 rounds of 32 lanes

// |x| of both halves of a bf16 pair as ordered integers; not finite counts as 0.
__device__ __forceinline__ uint32_t finite_abs_max(uint32_t m, uint32_t pair) {
  const uint32_t a = (pair & 0x7fffu) << 16, b = pair & 0x7fff0000u;
  m = a < 0x7f800000u ? max(m, a) : m;
  return b < 0x7f800000u ? max(m, b) : m;
}

__device__ __forceinline__ float finite_or_nan(uint32_t bits) {
  return __uint_as_float((bits & 0x7f800000u) == 0x7f800000u ? 0x7fffffffu : bits);
}

__device__ __forceinline__ uint32_t codes_of(uint32_t p0, uint32_t p1, float inv) {
  const uint32_t lo = e4m3x2(finite_or_nan(p0 << 16) * inv, finite_or_nan(p0 & 0xffff0000u) * inv);
  const uint32_t hi = e4m3x2(finite_or_nan(p1 << 16) * inv, finite_or_nan(p1 & 0xffff0000u) * inv);
  return lo | (hi << 16);
}

// One warp per token: 18 values a lane in registers, one maximum over the
// warp, one rounding.  The scale is the smallest power of two that brings the
// maximum to 448 = 1.75 * 2^8 or less: its exponent is the maximum's minus 8,
// plus one where the mantissa is above 1.75, so it is found exactly from the
// bits, and the division by it is an exact product.
__global__ void __launch_bounds__(32 * kWriteWarps)
mla_write_kv8_kernel(const uint4* __restrict__ kv_c, int64_t kv_c_row, const uint4* __restrict__ k_pe,
                     int64_t k_pe_row, const int64_t* __restrict__ slot_mapping, int64_t num_tokens,
                     uint8_t* __restrict__ codes, float* __restrict__ scales, int64_t num_slots, int64_t entry,
                     int32_t* __restrict__ status) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= num_tokens) return;
  const int64_t s = slot_mapping[t];
  uint4 x[3];
  x[0] = kv_c[t * kv_c_row + lane];
  x[1] = kv_c[t * kv_c_row + 32 + lane];
  x[2] = lane < 8 ? k_pe[t * k_pe_row + lane] : make_uint4(0, 0, 0, 0);
  if (s < 0) return;  // padding token
  if (s >= num_slots) {
    if (lane == 0) atomicExch(status, kStatusBadBlockId);
    return;
  }
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 3; ++c)
    m = finite_abs_max(finite_abs_max(finite_abs_max(finite_abs_max(m, x[c].x), x[c].y), x[c].z), x[c].w);
  m = __reduce_max_sync(0xffffffffu, m);
  const int e = max(1, static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0));  // biased
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  uint2* const dst = reinterpret_cast<uint2*>(codes + s * entry);
#pragma unroll
  for (int c = 0; c < 3; ++c)
    if (c < 2 || lane < 8) dst[32 * c + lane] = make_uint2(codes_of(x[c].x, x[c].y, inv), codes_of(x[c].z, x[c].w, inv));
  if (lane == 0) scales[s] = __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// The last i in [0, b) with cu[i] <= r (cu[0] = 0 <= r), by the whole warp: 32
// probes a round.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int b, int64_t r, int lane) {
  int lo = 0, n = b;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && (lane == 0 || __ldg(cu + i) <= r);
    const unsigned vote = __ballot_sync(0xffffffffu, le);
    const int k = 31 - __clz(vote);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Eight output rows a warp: lane r (of the first 8) finds row r's entry and
// scale, then the warp streams the rows' 576 chunks, 18 coalesced loads and
// stores with the loads of nine rounds in flight.
__global__ void __launch_bounds__(32 * kReadWarps)
mla_read_kv8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t num_blocks,
                    int64_t entry, const int32_t* __restrict__ block_table, int max_blocks,
                    const int32_t* __restrict__ cu, const int32_t* __restrict__ starts, int b,
                    uint4* __restrict__ out, int64_t rows, int32_t* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5)) * kReadRows;
  const int64_t end = min(rows, static_cast<int64_t>(__ldg(cu + b)));
  if (r0 >= end) return;
  int i = find_sequence(cu, b, r0, lane);
  int64_t src = -1;
  float scale = 0.f;
  if (lane < kReadRows && r0 + lane < end) {
    const int64_t r = r0 + lane;
    while (i + 1 < b && __ldg(cu + i + 1) <= r) ++i;
    const int64_t t = r - __ldg(cu + i) + (starts ? __ldg(starts + i) : 0);
    const int64_t p = t / kPage;
    if (t < 0) {
      atomicExch(status, kStatusBadSeqlen);
    } else {
      const int64_t page = p < max_blocks ? __ldg(block_table + static_cast<int64_t>(i) * max_blocks + p) : -1;
      if (page < 0 || page >= num_blocks) {
        atomicExch(status, kStatusBadBlockId);
      } else {
        const int64_t slot = page * kPage + t % kPage;
        src = slot * entry;
        scale = __ldg(scales + slot);
      }
    }
  }
  __syncwarp();
  constexpr int kRound = 9;
  uint4* const dst = out + r0 * kChunks;
#pragma unroll
  for (int c0 = 0; c0 < kReadRows * kChunks / 32; c0 += kRound) {
    uint2 v[kRound];
    float f[kRound];
    bool live[kRound];
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int c = (c0 + u) * 32 + lane;
      const int64_t from = __shfl_sync(0xffffffffu, src, c / kChunks);
      f[u] = __shfl_sync(0xffffffffu, scale, c / kChunks);
      live[u] = from >= 0;
      v[u] = live[u] ? __ldg(reinterpret_cast<const uint2*>(codes + from) + c % kChunks) : make_uint2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      if (!live[u]) continue;
      const float2 a = e4m3x2_to_float2(v[u].x & 0xffffu), b2 = e4m3x2_to_float2(v[u].x >> 16);
      const float2 c = e4m3x2_to_float2(v[u].y & 0xffffu), d = e4m3x2_to_float2(v[u].y >> 16);
      dst[(c0 + u) * 32 + lane] =
          make_uint4(pack_bf16x2(a.x * f[u], a.y * f[u]), pack_bf16x2(b2.x * f[u], b2.y * f[u]),
                     pack_bf16x2(c.x * f[u], c.y * f[u]), pack_bf16x2(d.x * f[u], d.y * f[u]));
    }
  }
}

}  // namespace

cudaError_t launch_write_kv8(const void* kv_c, int64_t kv_c_row_elems, const void* k_pe, int64_t k_pe_row_elems,
                             const int64_t* slot_mapping, int64_t num_tokens, void* codes, float* scales,
                             int64_t num_slots, int stride, int32_t* status, cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((num_tokens + kWriteWarps - 1) / kWriteWarps));
  mla_write_kv8_kernel<<<grid, 32 * kWriteWarps, 0, stream>>>(
      static_cast<const uint4*>(kv_c), kv_c_row_elems / 8, static_cast<const uint4*>(k_pe), k_pe_row_elems / 8,
      slot_mapping, num_tokens, static_cast<uint8_t*>(codes), scales, num_slots, stride, status);
  return cudaGetLastError();
}

cudaError_t launch_read_kv8(const void* codes, const float* scales, int64_t num_blocks, int stride,
                            const int32_t* block_table, int max_blocks, const int32_t* cu_tokens,
                            const int32_t* starts, int b, void* out, int64_t rows, int32_t* status,
                            cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int64_t per = kReadWarps * kReadRows;
  mla_read_kv8_kernel<<<static_cast<unsigned>((rows + per - 1) / per), 32 * kReadWarps, 0, stream>>>(
      static_cast<const uint8_t*>(codes), scales, num_blocks, stride, block_table, max_blocks, cu_tokens, starts, b,
      static_cast<uint4*>(out), rows, status);
  return cudaGetLastError();
}

}  // namespace mla
