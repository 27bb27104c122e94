// What the two decode kernels over the 8-bit cache share: the walk over tiles of
// two pages, the form of the weights, and thin wrappers of the instructions
// that only they use.
#pragma once

#include <cuda_bf16.h>

#include "mla_kv8_internal.h"
#include "mla_walk.cuh"
#include "sm103_ptx.cuh"

namespace mla {

constexpr int kTile = 128;  // tokens: two pages

// Weights are stored as kUnit P scale / R.  The running maximum M is the one of the
// weights, of S + log2(scale / R), not of the scores, so that a row's largest weight
// is near kUnit whatever the scales beside it are, those of tokens that it does not
// see among them.  M is moved (and O rescaled, between two products) only when it
// grew by more than kSlack (log2): weights stay below kUnit 2^kSlack < 448, e4m3's
// largest.  R, a power of two, serves the range only: P and its sum l reach R / scale.
constexpr float kMargin = 1.f;             // a maximum that moves goes this far beyond, so that it moves less often
// R is about the largest scale of a segment's first tile, within limits between which both
// ends of the scales' range are in reach: 2^-126 is 2^-100 of the lower, 2^128 2^98 of the upper.
constexpr float kMinR = 0x1p-26f, kMaxR = 0x1p30f;
constexpr float kMinLog = -100.f;          // of log2(scale / R), as far as M goes; 0 has it too: P is up to 2^100
constexpr float kMaxRatio = 0x1p101f;      // of scale / R: a weight's P is 2^-101, and those beside it are held to 2^-25 of it
constexpr float kNothing = 0x1p-60f;       // such scales are next to nothing; an entry of zeros is written with 2^-126

__device__ __forceinline__ float log_ratio(float ratio) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(ratio));
  return fmaxf(y, kMinLog);
}

__device__ __forceinline__ int log2_of_power(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }  // positive, normal
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // normal ones

// R for tokens of which `top` is the largest finite scale, in bits; kMinR where that is nothing.
//
// These are the tokens that every row sees, for what a row does not see must not change
// its bits; and a segment's first, which every row that sees one of them sees.  While they
// hold nothing, R stays kMinR (rows that see more see scales up to 2^75 well), and moves once,
// at the first tile that has more for every row.  O is in units of R; P, l and M stay: M, of
// what was nothing, is 34 to 100 below its scores, low enough for what comes.
__device__ __forceinline__ float reference_scale(uint32_t top) {
  return fminf(fmaxf(__uint_as_float(top & 0x7f800000u), kMinR), kMaxR);
}
__device__ __forceinline__ bool is_nothing(uint32_t top) { return !(__uint_as_float(top) > kNothing); }

// A move of M by d changes l by 2^d, which is made as the square of this: l may reach 2^100
// by tokens of no scale, and what is then left of it still counts although 2^d is below 2^-126.
__device__ __forceinline__ float root_of_move(float d) { return ex2_approx(0.5f * d); }

// m + log2(l) where both may be large and of opposite signs.
__device__ __forceinline__ float log_sum(float m, float l) {
  if (!(l < INFINITY)) return l;
  const int bits = __float_as_int(l);
  return (m + static_cast<float>((bits >> 23) - 127)) + log2f(__int_as_float((bits & 0x7fffff) | 0x3f800000));
}

struct TileWalk : PageWalk {
  __device__ __forceinline__ bool last() const { return p + 2 >= p_end; }
  __device__ __forceinline__ void advance() {
    p += 2;
    if (p >= p_end) next_segment();
  }
};

// kind::f8f6f4, e4m3 operands, fp32 accumulators.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N, bool a_mn, bool b_mn) {  // M = 128
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float warp_max(float x) {  // NaN is ignored
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// N consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[16]) { tmem_ld16(a, r); }
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[16]) { tmem_st16(a, r); }
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[32]) { tmem_ld32(a, r); }
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[32]) { tmem_st32(a, r); }
// The register pass-through keeps the compiler from reading them before the wait.
__device__ __forceinline__ void tmem_landed() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void hold(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// Bytes 0x7f and 0xff (NaN) of four codes become zero.
__device__ __forceinline__ uint32_t without_nan(uint32_t v) {
  const uint32_t nan = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // a byte's top bit where its 7 low bits are all set
  return v & ~((nan >> 7) * 0xffu);
}

// A 4 x 4 block of bytes over four lanes, one register each, transposed.
__device__ __forceinline__ uint32_t turn_4x4(uint32_t w, int lane) {
  const uint32_t y = __shfl_xor_sync(0xffffffffu, w, 1);
  w = __byte_perm(w, y, lane & 1 ? 0x3715 : 0x6240);
  const uint32_t z = __shfl_xor_sync(0xffffffffu, w, 2);
  return __byte_perm(w, z, lane & 2 ? 0x3276 : 0x5410);
}

// A query row times 2^-e as hi + lo, two e4m3 numbers a value, at rows r and
// kR + r of the operand at `qs`: four chunks of 128 dims (128-byte rows, 128B
// swizzle), then the 64 rope dims (64B swizzle).  e is the smallest with
// max |q| <= 448 * 2^e, as for the cache's scales; 255 stands for a row that is
// not finite, which becomes NaN codes.  A row is handled in pieces of 8 dims.
constexpr int kQueryPieces = kDimQK / 8;

__device__ __forceinline__ uint32_t query_max(uint32_t m, const uint4& x) {  // |x| of bf16 pairs, as integers of 16 bits
  return __vmaxu2(__vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu)), x.w & 0x7fff7fffu);
}

__device__ __forceinline__ int query_exponent(uint32_t m) {  // e + 127 of a row with that maximum
  m = max(m & 0xffffu, m >> 16);
  if (m >= 0x7f80u) return 255;
  return max(1, static_cast<int>(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0));
}

__device__ __forceinline__ float query_step(int e) { return __uint_as_float(static_cast<uint32_t>(e < 255 ? e : 127) << 23); }

// By way of f16, which holds what either number can of a bf16 value: it is exact
// down to 2^-17, and e4m3 ends at 2^-9.
template <int kR>
__device__ __forceinline__ void store_query_piece(uint8_t* qs, int r, int piece, const uint4& x, int e) {
  const uint32_t inv = e < 255 ? static_cast<uint32_t>(254 - e) * 0x00800080u : 0x7fff7fffu;  // bf16 pair
  const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t w, h;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(ws[p]), "r"(inv));  // exact
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
    hi[p] = e4m3x2_of_f16x2(h);
    uint32_t rest;
    asm("{\n\t.reg .b32 f;\n\tcvt.rn.f16x2.e4m3x2 f, %2;\n\tsub.rn.f16x2 %0, %1, f;\n\t}"
        : "=r"(rest)
        : "r"(h), "h"(static_cast<uint16_t>(hi[p])));
    lo[p] = e4m3x2_of_f16x2(rest);
  }
  const bool rope = piece >= kDimV / 8;
  const int unit = (piece & (rope ? 7 : 15)) >> 1;  // 16 bytes; a piece is half of one
  uint8_t* const d = qs + (piece >> 4) * (2 * kR * 128) + (piece & 1) * 8 +
                     (rope ? r * 64 + ((unit ^ ((r >> 1) & 3)) << 4) : r * 128 + ((unit ^ (r & 7)) << 4));
  *reinterpret_cast<uint2*>(d) = make_uint2(__byte_perm(hi[0], hi[1], 0x5410), __byte_perm(hi[2], hi[3], 0x5410));
  *reinterpret_cast<uint2*>(d + (rope ? kR * 64 : kR * 128)) =
      make_uint2(__byte_perm(lo[0], lo[1], 0x5410), __byte_perm(lo[2], lo[3], 0x5410));
}

// The loops below run against instruction fetch: what is rare (a wait that is not
// over at once among it) is told to the compiler, which then lays it out of line.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

template <bool kCluster = false>
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (rare(!(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))))
    return mbar_wait<kCluster>(bar, parity, abort_flag);
  return true;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_on(bar, parity, abort_flag));
}

}  // namespace mla
