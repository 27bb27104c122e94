// Host side of the C ABI declared in include/mla_kv8.h: argument checks and
// launches.  No allocation, no synchronisation.
#include <cmath>
#include <cstdint>

#include "../../include/mla_kv8.h"
#include "mla_kv8_internal.h"

namespace mla {
int32_t check_decode_args(const void* q, int b, int s_q, int h_q, int d, const void* kcache, int64_t num_blocks,
                          int block_size, int h_kv, int stride, const int32_t* block_table, int max_blocks_per_seq,
                          const int32_t* cache_seqlens, int dv, const int32_t* metadata, int num_parts,
                          const int32_t* num_splits, float softmax_scale, int causal, const void* out,
                          const float* lse, const void* workspace, size_t workspace_bytes, const int32_t* status);
}

namespace {

using mla::kDimQK;
using mla::kDimV;
using mla::kPage;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What the calls on an 8-bit cache share.
mla_status_t check_cache(const void* codes, const float* scales, int64_t num_blocks, int block_size, int stride,
                         const int32_t* status) {
  if (!codes || !scales || !status || num_blocks < 1) return MLA_ERR_INVALID_ARG;
  if (block_size != kPage) return MLA_ERR_UNSUPPORTED;
  if (stride < kDimQK) return MLA_ERR_INVALID_ARG;
  if (stride % 16 || !aligned(codes, 16) || !aligned(scales, 16)) return MLA_ERR_ALIGNMENT;
  return MLA_OK;
}

// Rows of `dim` elements at ptr + (token * t + head * h) elements.
struct Rows {
  const void* ptr;
  int64_t t, h, heads;
  int64_t span(int64_t dim) const { return (heads > 1 ? (heads - 1) * h : 0) + dim; }  // of one token
};

// Whether the strides are ones to read by, or to write by without writing twice.
bool rows_in_order(const Rows& a, int64_t tokens) { return (tokens <= 1 || a.t >= 0) && (a.heads <= 1 || a.h >= 0); }
bool rows_apart(const Rows& a, int64_t tokens, int64_t dim) {
  if ((tokens > 1 && a.t < dim) || (a.heads > 1 && a.h < dim)) return false;
  return tokens <= 1 || a.heads <= 1 || a.t >= a.span(dim) || a.h >= (tokens - 1) * a.t + dim;
}

// Whether no row of a meets a row of b: their ranges are apart, or the tokens of one
// lie between those of the other, or with the same strides its rows do.  (Other
// layouts that keep apart are not told from ones that do not.)
bool rows_apart(const Rows& a, const Rows& b, int64_t tokens, int64_t dim, int64_t size) {
  const int64_t bytes = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.ptr) - reinterpret_cast<uintptr_t>(a.ptr));
  const int64_t a_end = (tokens > 1 ? (tokens - 1) * a.t : 0) + a.span(dim);
  const int64_t b_end = (tokens > 1 ? (tokens - 1) * b.t : 0) + b.span(dim);
  if (bytes >= a_end * size || -bytes >= b_end * size) return true;
  if (bytes % size) return false;
  int64_t gap = bytes / size;
  if (tokens > 1 && a.t != b.t) return false;
  const int64_t st = tokens > 1 ? a.t : 0;
  if (st > 0) {
    const int64_t g = ((gap % st) + st) % st;
    if (g >= a.span(dim) && g + b.span(dim) <= st) return true;
  }
  if (a.heads > 1 && b.heads > 1 && a.h != b.h) return false;
  const int64_t sh = a.heads > 1 ? a.h : b.heads > 1 ? b.h : 0;
  const int64_t outer = st > sh ? st : sh, inner = st > sh ? sh : st;
  const auto within = [&](const Rows& r) { return (st > sh ? r.span(dim) : (tokens - 1) * st + dim) <= outer; };
  if (inner <= 0 || !within(a) || !within(b)) return false;
  gap = ((gap % outer) + outer) % outer;
  // b's rows that run over an end of a's outer step meet a's next ones at the same
  // remainder only where the inner step divides the outer
  if (outer % inner) return false;
  gap %= inner;
  return gap >= dim && gap <= inner - dim;
}

// Rows of a sequence that a decode takes (see check_decode_args); s_q (h_q / h_kv) is an int below.
bool too_many_rows(int s_q, int h_q) { return static_cast<int64_t>(s_q) * h_q > 4 * 65535; }

mla_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();  // a launch that failed is this call's to report, not the next one's
  return MLA_ERR_CUDA;
}

}  // namespace

extern "C" {

mla_status_t mla_write_cache_kv8(const void* kv_c, int64_t kv_c_row_stride, const void* k_pe, int64_t k_pe_row_stride,
                                 const int64_t* slot_mapping, int64_t num_tokens, void* codes, float* scales,
                                 int64_t num_blocks, int block_size, int stride, int32_t* status,
                                 mla_stream_t stream) {
  const mla_status_t r = check_cache(codes, scales, num_blocks, block_size, stride, status);
  if (r != MLA_OK) return r;
  if (num_tokens < 0 || num_tokens > 0x7fffffff) return MLA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!kv_c || !k_pe || !slot_mapping)) return MLA_ERR_INVALID_ARG;
  if (kv_c_row_stride < kDimV || k_pe_row_stride < kDimQK - kDimV) return MLA_ERR_INVALID_ARG;
  if (kv_c_row_stride % 8 || k_pe_row_stride % 8) return MLA_ERR_ALIGNMENT;
  if (num_tokens > 0 && (!aligned(kv_c, 16) || !aligned(k_pe, 16) || !aligned(slot_mapping, 8)))
    return MLA_ERR_ALIGNMENT;
  return done(mla::launch_write_kv8(kv_c, kv_c_row_stride, k_pe, k_pe_row_stride, slot_mapping, num_tokens, codes,
                                    scales, num_blocks * kPage, stride, status,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_read_cache_kv8(const void* codes, const float* scales, int64_t num_blocks, int block_size, int stride,
                                const int32_t* block_table, int max_blocks_per_seq, const int32_t* cu_tokens,
                                const int32_t* starts, int b, void* out, int64_t rows, int32_t* status,
                                mla_stream_t stream) {
  const mla_status_t r = check_cache(codes, scales, num_blocks, block_size, stride, status);
  if (r != MLA_OK) return r;
  if (rows < 0 || rows > 0x7fffffff || b < 1 || max_blocks_per_seq < 1) return MLA_ERR_INVALID_ARG;
  if (!block_table || !cu_tokens || (rows > 0 && !out)) return MLA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(block_table, 4) || !aligned(cu_tokens, 4) || !aligned(starts, 4))
    return MLA_ERR_ALIGNMENT;
  return done(mla::launch_read_kv8(codes, scales, num_blocks, stride, block_table, max_blocks_per_seq, cu_tokens,
                                   starts, b, out, rows, status, reinterpret_cast<cudaStream_t>(stream)));
}

int mla_num_parts_kv8(int s_q, int h_q, int h_kv, int device) {
  if (s_q < 1 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0) return MLA_ERR_INVALID_ARG;
  if (h_q / h_kv > mla::kRowsPerTile || too_many_rows(s_q, h_q)) return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_INVALID_ARG;
  }
  const int64_t units = static_cast<int64_t>(mla::decode_kv8_ctas(s_q * (h_q / h_kv))) * h_kv;
  const int parts = static_cast<int>(sms / units);  // one CTA per SM
  return parts < 1 ? 1 : parts;
}

size_t mla_workspace_bytes_kv8(int b, int s_q, int h_q, int h_kv, int num_parts) {
  const size_t parts = mla_workspace_bytes(b, s_q, h_q, num_parts);
  if (parts == 0 || h_kv < 1 || h_q % h_kv != 0 || too_many_rows(s_q, h_q)) return 0;
  return parts + mla::decode_kv8_query_bytes(b, h_kv, s_q * (h_q / h_kv));
}

mla_status_t mla_decode_kv8(const void* q, int b, int s_q, int h_q, int d, const void* codes, const float* scales,
                            int64_t num_blocks, int block_size, int h_kv, int stride, const int32_t* block_table,
                            int max_blocks_per_seq, const int32_t* cache_seqlens, int dv, const int32_t* metadata,
                            int num_parts, const int32_t* num_splits, float softmax_scale, int causal, void* out,
                            float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                            mla_stream_t stream) {
  mla_status_t r = mla::check_decode_args(q, b, s_q, h_q, d, codes, num_blocks, block_size, h_kv, stride, block_table,
                                          max_blocks_per_seq, cache_seqlens, dv, metadata, num_parts, num_splits,
                                          softmax_scale, causal, out, lse, workspace, workspace_bytes, status);
  if (r == MLA_OK) r = check_cache(codes, scales, num_blocks, block_size, stride, status);
  if (r == MLA_OK && workspace_bytes < mla_workspace_bytes_kv8(b, s_q, h_q, h_kv, num_parts)) r = MLA_ERR_INVALID_ARG;
  // one grid dimension counts the queries' rows by sixteens, in tiles of 128
  if (r == MLA_OK && static_cast<int64_t>(b) * (static_cast<int64_t>(s_q) * h_q + 127 * static_cast<int64_t>(h_kv)) / 16 > 0x7fffffff)
    r = MLA_ERR_INVALID_ARG;
  if (r != MLA_OK) return r;

  mla::DecodeKv8Params p;
  p.q = q;
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = scales;
  p.block_table = block_table;
  p.cache_seqlens = cache_seqlens;
  p.metadata = metadata;
  p.num_splits = num_splits;
  p.out = out;
  p.lse = lse;
  const size_t slots = static_cast<size_t>(b) + static_cast<size_t>(num_parts);
  const size_t o_bytes = (slots * static_cast<size_t>(s_q) * h_q * kDimV * 4 + 255) & ~static_cast<size_t>(255);
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + o_bytes);
  p.ws_q = static_cast<uint8_t*>(workspace) + mla_workspace_bytes(b, s_q, h_q, num_parts);
  p.ws_c = reinterpret_cast<float*>(p.ws_q + mla::decode_kv8_factors_at(b, h_kv, s_q * (h_q / h_kv)));
  p.status = status;
  p.num_blocks = num_blocks;
  p.entry_bytes = stride;
  p.b = b;
  p.s_q = s_q;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.heads_per_kv = h_q / h_kv;
  p.rows = s_q * p.heads_per_kv;
  p.max_blocks = max_blocks_per_seq;
  p.causal = causal;
  p.scale_log2 = softmax_scale * 1.4426950408889634f * (1.f / mla::kFactorUnit);
  r = done(mla::launch_decode_kv8(p, num_parts, reinterpret_cast<cudaStream_t>(stream)));
  if (r != MLA_OK) return r;
  mla::CombineParams m;
  m.num_splits = num_splits;
  m.ws_o = p.ws_o;
  m.ws_lse = p.ws_lse;
  m.out = out;
  m.lse = lse;
  m.b = b;
  m.s_q = s_q;
  m.h_q = h_q;
  m.num_parts = num_parts;
  return done(mla::launch_merge_kv8(m, reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                      int64_t out_token_stride, int64_t out_head_stride, int heads, const void* k,
                      int64_t k_token_stride, int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
                      int64_t k_out_head_stride, int k_heads, int64_t tokens, int rot_dim, const void* positions,
                      int position_bytes, const uint64_t* turns, float gain, int interleaved, int inverse, int dtype,
                      mla_stream_t stream) {
  if (tokens < 0 || heads < 1 || k_heads < 0 || rot_dim < 2 || rot_dim > 256 || rot_dim % 2) return MLA_ERR_INVALID_ARG;
  if ((position_bytes != 4 && position_bytes != 8) || (interleaved != 0 && interleaved != 1) ||
      (inverse != 0 && inverse != 1) || !std::isfinite(gain))
    return MLA_ERR_INVALID_ARG;
  if (dtype != MLA_BF16 && dtype != MLA_FP16 && dtype != MLA_FP32) return MLA_ERR_UNSUPPORTED;
  if (tokens == 0) return MLA_OK;
  if (!x || !out || !positions || !turns || (k_heads > 0) != (k != nullptr) || (k_heads > 0) != (k_out != nullptr))
    return MLA_ERR_INVALID_ARG;
  if (heads > (1 << 20) || k_heads > (1 << 20) || tokens > (static_cast<int64_t>(1) << 40) / (heads + k_heads))
    return MLA_ERR_INVALID_ARG;
  const unsigned size = dtype == MLA_FP32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(out, size) || !aligned(k, size) || !aligned(k_out, size) || !aligned(turns, 8) ||
      !aligned(positions, position_bytes))
    return MLA_ERR_ALIGNMENT;
  // a row that is written is no other row, but for the one that it comes from
  const Rows in[2] = {{x, x_token_stride, x_head_stride, heads}, {k, k_token_stride, k_head_stride, k_heads}};
  const Rows to[2] = {{out, out_token_stride, out_head_stride, heads}, {k_out, k_out_token_stride, k_out_head_stride, k_heads}};
  const int sets = k_heads > 0 ? 2 : 1;
  for (int i = 0; i < sets; ++i) {
    if (!rows_in_order(in[i], tokens) || !rows_apart(to[i], tokens, rot_dim)) return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < sets; ++j) {
      const bool in_place = i == j && to[i].ptr == in[i].ptr && (tokens <= 1 || to[i].t == in[i].t) &&
                            (in[i].heads <= 1 || to[i].h == in[i].h);
      if (!in_place && !rows_apart(in[j], to[i], tokens, rot_dim, size)) return MLA_ERR_INVALID_ARG;
    }
  }
  if (sets == 2 && !rows_apart(to[0], to[1], tokens, rot_dim, size)) return MLA_ERR_INVALID_ARG;
  mla::RopeParams p;
  p.x = {x, out, x_token_stride, x_head_stride, out_token_stride, out_head_stride};
  p.k = {k, k_out, k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride};
  p.heads = heads;
  p.k_heads = k_heads;
  p.tokens = tokens;
  p.pairs = rot_dim / 2;
  p.positions = positions;
  p.turns = turns;
  p.gain = gain;
  p.inverse = inverse != 0;
  // 16-byte vectors where every row of every tensor allows them
  const int per = 16 / static_cast<int>(size);
  bool vec = p.pairs % per == 0 && aligned(x, 16) && aligned(out, 16) && aligned(k, 16) && aligned(k_out, 16);
  for (int64_t s : {x_token_stride, x_head_stride, out_token_stride, out_head_stride}) vec = vec && s % per == 0;
  if (k_heads > 0)
    for (int64_t s : {k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride}) vec = vec && s % per == 0;
  const int units = (p.pairs + per - 1) / per;
  if (tokens * (heads + k_heads) / (mla::kRopeThreads / units) >= 0x7fffffff) return MLA_ERR_INVALID_ARG;  // blocks
  return done(mla::launch_rope(p, dtype, interleaved != 0, position_bytes == 8, vec,
                               reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
