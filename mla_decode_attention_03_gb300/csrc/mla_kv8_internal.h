// Internal interface of the 8-bit cache kernels and the rotary kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mla_internal.h"

namespace mla {

// A score is (product x scale kFactorUnit) x c, with 1 / kFactorUnit in c: a product of a row's and
// a token's codes is up to 2^27, a scale up to 2^120, and a query may be as small as the scale is large.
constexpr float kFactorUnit = 0x1p-7f;

struct DecodeKv8Params {
  const void* q;                 // bf16 [b, s_q, h_q, 576]
  const uint8_t* codes;          // e4m3 entries
  const float* scales;           // [num_blocks, h_kv, 64]
  const int32_t* block_table;    // [b, max_blocks]
  const int32_t* cache_seqlens;  // [b]
  const int32_t* metadata;       // [num_parts, kMetaInts]
  const int32_t* num_splits;     // [b + 1] prefix sums
  void* out;                     // bf16 [b, s_q, h_q, 512]
  float* lse;                    // [b, h_q, s_q]
  float* ws_o;                   // fp32 [slots, s_q*h_q, 512]: normalised partial outputs
  float* ws_lse;                 // [slots, s_q*h_q]
  uint8_t* ws_q;                 // CTA pairs: the queries as e4m3, 64 rows at a time
  float* ws_c;                   //   and their factors
  int32_t* status;
  int64_t num_blocks;
  int64_t entry_bytes;
  int b, s_q, h_q, h_kv;
  int heads_per_kv;              // h_q / h_kv
  int rows;                      // s_q * heads_per_kv: query rows per KV head
  int max_blocks;
  int causal;
  float scale_log2;              // softmax_scale * log2(e) / kFactorUnit
};

bool decode_kv8_in_pairs(int rows);
int decode_kv8_ctas(int rows);  // CTAs per part and KV head
size_t decode_kv8_query_bytes(int b, int h_kv, int rows);    // codes, then factors
size_t decode_kv8_factors_at(int b, int h_kv, int rows);     // offset of the factors
cudaError_t launch_decode_kv8_pair(const DecodeKv8Params& p, const CUtensorMap& lat, const CUtensorMap& rope, int num_parts,
                                   cudaStream_t stream);
cudaError_t launch_decode_kv8(const DecodeKv8Params& p, int num_parts, cudaStream_t stream);
cudaError_t launch_merge_kv8(const CombineParams& p, cudaStream_t stream);
cudaError_t launch_write_kv8(const void* kv_c, int64_t kv_c_row_elems, const void* k_pe, int64_t k_pe_row_elems,
                             const int64_t* slot_mapping, int64_t num_tokens, void* codes, float* scales,
                             int64_t num_slots, int stride, int32_t* status, cudaStream_t stream);
cudaError_t launch_read_kv8(const void* codes, const float* scales, int64_t num_blocks, int stride,
                            const int32_t* block_table, int max_blocks, const int32_t* cu_tokens,
                            const int32_t* starts, int b, void* out, int64_t rows, int32_t* status,
                            cudaStream_t stream);

constexpr int kRopeThreads = 128;  // a block

struct RopeRows {
  const void* src;
  void* dst;
  int64_t src_token, src_head, dst_token, dst_head;  // strides in elements
};
struct RopeParams {
  RopeRows x, k;
  int heads, k_heads;
  int64_t tokens;
  int pairs;            // rot_dim / 2
  const void* positions;
  const uint64_t* turns;
  float gain;
  bool inverse;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, bool interleaved, bool pos64, bool vec, cudaStream_t stream);

// ------------------------------------------------------------- e4m3
#ifdef __CUDACC__
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {  // saturating, ties to even, NaN -> 0x7f
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {  // exact: e4m3 values are f16 values
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
#endif

}  // namespace mla
