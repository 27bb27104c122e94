// Split-KV MLA decode over the 8-bit latent cache (e4m3 codes, one scale per
// token and head), for sm_103a.  Same schedule and workspace as the
// bf16 kernels.
//
//   S[t, r] = c_r scale_t <q'_r, code_t>       c_r = softmax_scale log2(e) 2^e_r
//   P[t, r] = 2^(S[t, r] - M_r)                M_r the running maximum of S[t, r] + log2(scale_t / R)
//   O[:, r] = sum_t (P[t, r] scale_t / R) code_t[0:512],   l_r = sum_t P[t, r]
//   out_r   = R O[:, r] / l_r                  R about the first tile's largest scale
//
// The codes go to the tensor cores as they lie in the cache: nothing is
// converted.  The other operand is made of two e4m3 numbers, x = hi + lo, in
// two products of twice the bf16 rate: q' (a row of q times a power of two that
// brings its maximum to 448 or less) is held exactly down to 2^-10 (its 8
// significant bits are 4 + 4), and a weight to 2^-8 of itself at most, 2^-10.9
// in the mean: as exact as a bf16 weight.
//
// The products are transposed, tokens or dims as the 128 rows of a tile and
// query rows as its columns, so few query rows cost few columns:
//   S^T [128 tokens x 2 kR]       = K_tile [128 x 576] (q_hi | q_lo)^T
//   O^T [4 x 128 dims x kR]      += V_tile^T [128 dims x 128 tokens] (P_hi | P_lo)^T
// V_tile is the same shared memory as K_tile, read MN-major.  A CTA takes up to
// kR = 16 or 32 query rows of one (sequence part, KV head); O^T, hi and lo
// apart (256 columns), and two S^T buffers fit its tensor memory.  33 to 64 rows
// take two such CTAs, which share the pages by way of L2; more go to CTA pairs
// (mla_decode_kv8_pair.cu).
//
// Warps (512 threads, one CTA per SM):
//   0-7   softmax: warpgroup g takes rows [g kR/2, (g+1) kR/2), a thread one token
//   8-11  quantise a segment's queries into shared memory
//   12    TMA: tiles of two pages, in chunks of 128 dims through a ring of slots
//   13    issues S^T; 14 and 15 issue O^T, half of the dims each (one thread issues
//         an MMA per 125 cycles here: a tile's 16 took 2,100, 1,200 like this)
// Hand-offs are mbarriers with bounded waits, as in the bf16 kernels.
//
// Bound at the sizes of a decode step by the chain of a tile's hand-overs (load, S,
// softmax, O), of which a CTA has two or three, and the merge after it: 16 sequences
// of 1024-4096 tokens, 16 heads, 14.8 us a call where the bytes alone take 3.6; one
// sequence of 256 tokens 7.9 us (of ten calls in a graph, inputs in L2; as the only
// call of a graph, L2 cold, 23.7 and 15.5).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "mla_kv8_dev.cuh"

namespace mla {
namespace {

constexpr int kChunk = kTile * 128;        // 128 latent dims of a tile
constexpr int kRopeBytes = kTile * 64;
constexpr int kRopeSlots = 2;
constexpr int kScaleSlots = 4;             // see the scale ring below
constexpr int kCSlots = 8;                 // see the queries' hand-over below
constexpr int kSoftmaxWarps = 8;
constexpr int kQWarps = 4;
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;

// A weight is hi + lo, both e4m3: off by 2^-8 of itself at most, or half of e4m3's
// smallest step, 2^-10, that is 2^-16 of a weight of 1.
constexpr float kUnit = 64.f;
constexpr float kSlack = 2.8f;
constexpr uint32_t kTmemS = 256;           // O^T: columns 0-255

template <int kR>
struct Cfg {
  static constexpr int H = kR / 2;                       // rows per softmax warpgroup
  static constexpr int QBufs = kR == 16 ? 2 : 1;
  static constexpr int Slots = kR == 16 ? 10 : 9;
  static constexpr int QChunk = 2 * kR * 128;
  static constexpr int QBytes = 2 * kR * kDimQK;
  static constexpr int PBytes = 2 * kR * kTile;
  static constexpr int OCols = 2 * kR;                   // columns of an O^T tile: hi, lo
  static constexpr int OffK = 0;
  static constexpr int OffRope = OffK + Slots * kChunk;
  static constexpr int OffQ = OffRope + kRopeSlots * kRopeBytes;
  static constexpr int OffP = OffQ + QBufs * QBytes;
  static constexpr int OffScale = OffP + PBytes;
  static constexpr int OffMx = OffScale + kScaleSlots * kTile * 4;    // float[2][2][4][32] partial maxima
  static constexpr int OffLs = OffMx + 2 * 2 * 4 * 32 * 4;            // float[2][4][32] partial row sums
  static constexpr int OffBc = OffLs + 2 * 4 * 32 * 4;                // float[8][2][32] per-warp broadcasts
  static constexpr int OffC = OffBc + 8 * 2 * 32 * 4;                 // float[kCSlots][kR] c_r of the last segments
  static constexpr int OffRow = OffC + kCSlots * kR * 4;              // int[kR] row in the sequence, int[kR] position
  static constexpr int OffBar = OffRow + 2 * kR * 4;
  // barriers
  static constexpr int KFull = 0, KEmpty = KFull + Slots, RopeFull = KEmpty + Slots, RopeEmpty = RopeFull + kRopeSlots,
                       ScFull = RopeEmpty + kRopeSlots, QFull = ScFull + kScaleSlots, QEmpty = QFull + 2,
                       CFull = QEmpty + 2, SFull = CFull + kCSlots, SEmpty = SFull + 2, PFull = SEmpty + 2, PvDone = PFull + 1,
                       Mx = PvDone + 1, Ls = Mx + 4, Drain = Ls + 2, NumBars = Drain + 1;
  static constexpr int OffMisc = OffBar + NumBars * 8;
  static constexpr int Bytes = OffMisc + 16 + 1024;      // abort flag, tensor memory address; slack to align the base
  static_assert(OffQ % 1024 == 0 && QChunk % 1024 == 0 && OffP % 1024 == 0 && OffRope % 1024 == 0 && QBytes % 1024 == 0,
                "swizzle atoms");
  static_assert(OffBar % 8 == 0 && OffScale % 16 == 0 && Bytes <= 232448, "shared memory per CTA");
  static_assert(4 * OCols <= static_cast<int>(kTmemS) && kTmemS + 2 * 2 * kR <= kTmemCols, "tensor memory");
};

template <int kR>
__global__ void __launch_bounds__(kThreads, 1)
mla_decode_kv8_kernel(const __grid_constant__ CUtensorMap lat_map, const __grid_constant__ CUtensorMap rope_map,
                      const DecodeKv8Params P, const int row_tiles) {
  using C = Cfg<kR>;
  constexpr int H = C::H;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_addr);
  auto bar = [&](int idx) -> uint32_t { return base + C::OffBar + 8u * idx; };
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + C::OffMisc);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OffMisc + 8);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int part = blockIdx.x / row_tiles;
  const int row0 = (blockIdx.x - part * row_tiles) * kR;
  const int g_kv = blockIdx.y;
  const int32_t* const meta = P.metadata + part * kMetaInts;
  int* const row_of = reinterpret_cast<int*>(gbase + C::OffRow);       // row in the sequence's [s_q, h_q], -1 past the last
  int* const pos_of = row_of + kR;                                     // its query position

  if (tid < kR) {
    const int row = row0 + tid;
    const int j = row / P.heads_per_kv;
    row_of[tid] = row < P.rows ? j * P.h_q + g_kv * P.heads_per_kv + row - j * P.heads_per_kv : -1;
    pos_of[tid] = row < P.rows ? j : P.s_q - 1;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::Slots; ++s) {
      mbar_init(bar(C::KFull + s), 1);
      mbar_init(bar(C::KEmpty + s), 1);
    }
    for (int s = 0; s < kRopeSlots; ++s) {
      mbar_init(bar(C::RopeFull + s), 1);
      mbar_init(bar(C::RopeEmpty + s), 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(bar(C::ScFull + s), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::QFull + s), kQWarps);
      mbar_init(bar(C::QEmpty + s), 1);
      mbar_init(bar(C::SFull + s), 1);
      mbar_init(bar(C::SEmpty + s), kSoftmaxWarps);
      mbar_init(bar(C::Ls + s), 4);
    }
    for (int s = 0; s < kCSlots; ++s) mbar_init(bar(C::CFull + s), kQWarps);
    for (int s = 0; s < 4; ++s) mbar_init(bar(C::Mx + s), 4);
    mbar_init(bar(C::PFull), kSoftmaxWarps);
    mbar_init(bar(C::PvDone), 2);
    mbar_init(bar(C::Drain), 3);
    fence_mbar_init();
  }
  if (warp == 14) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the scheduler's output (and q) are complete from here on
  grid_launch_dependents();

  bool ok = true;
  if (warp < kSoftmaxWarps) {
    // ================================================= softmax and epilogue
    regs_inc<168>();
    const int g = warp >> 2, quad = warp & 3;
    const int tl = quad * 32 + lane;                       // this thread's token of a tile
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    float* const mx = reinterpret_cast<float*>(gbase + C::OffMx);
    float* const ls = reinterpret_cast<float*>(gbase + C::OffLs) + g * 128;
    float* const bc = reinterpret_cast<float*>(gbase + C::OffBc) + warp * 64;  // [0]: -M or 1/l, [1]: roots of l's factors, then O's factors
    const float* const scales = reinterpret_cast<const float*>(gbase + C::OffScale);
    const int rows_total = P.s_q * P.h_q;

    TileWalk w;
    w.start(meta, P.cache_seqlens, P.max_blocks);
    int n = 0, seg = -1;
    float l[H];
    float m_run = -INFINITY;   // of row g H + lane (lanes below H)
    float bound = 1.f;         // R
    bool nothing = false;      // of which R was made
    int L = 0, seg_end = 0, all_see = 0;
    const float* c_row = nullptr;

    while (w.valid) {
      const bool first = w.first();
      if (rare(first)) {
        ++seg;
        L = __ldg(P.cache_seqlens + w.i);
        seg_end = min(L, w.p_end * kPage);
        all_see = min(seg_end, P.causal ? L - P.s_q + 1 : L);  // tokens before it are seen by every row
        m_run = -INFINITY;
#pragma unroll
        for (int r = 0; r < H; ++r) l[r] = 0.f;
        ok = warp_wait(bar(C::CFull + seg % kCSlots), (seg / kCSlots) & 1, abort_flag);
        if (rare(!ok)) break;
        c_row = reinterpret_cast<const float*>(gbase + C::OffC) + seg % kCSlots * kR + g * H;
      }
      const int t0 = w.p * kPage;
      const int tok = t0 + tl;
      const bool ragged = t0 + kTile > all_see;

      // ---- this tile's scales
      ok = warp_wait(bar(C::ScFull + (n & 3)), (n >> 2) & 1, abort_flag);
      if (rare(!ok)) break;
      const float* const sc = scales + (n & 3) * kTile;
      float scale = tok < seg_end ? sc[tl] : 0.f;
      if (!(scale < INFINITY)) scale = __uint_as_float(0x7fffffffu);  // a row that sees it becomes NaN
      int shift = 0;                                       // by which log2(R) moves
      if (rare(first || (nothing && t0 < all_see))) {
        uint32_t top = 0;
#pragma unroll 1
        for (int e = lane; e < kTile; e += 32) {
          const uint32_t a = __float_as_uint(sc[e]);
          if ((t0 + e < all_see || (first && e == 0)) && a < 0x7f800000u) top = max(top, a);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        nothing = is_nothing(top);
        const float r = reference_scale(top);
        if (!first) shift = log2_of_power(r) - log2_of_power(bound);
        bound = r;
      }
      // (a NaN scale counts as 0 here: to a row that does not see it, it is nothing)
      const float ratio = scale < INFINITY ? fminf(scale * (1.f / bound), kMaxRatio) : 0.f;
      const float log_of = log_ratio(ratio), factor = scale * kFactorUnit;

      // ---- scores
      ok = warp_wait(bar(C::SFull + (n & 1)), (n >> 1) & 1, abort_flag);
      if (rare(!ok)) break;
      tc_fence_after_sync();
      float v[H];
      {
        uint32_t hi[H], lo[H];
        const uint32_t at = tmem + lanes + kTmemS + (n & 1) * (2 * kR) + g * H;
        tmem_ld(at, hi);
        tmem_ld(at + kR, lo);
        tmem_landed();
        hold(hi);
        hold(lo);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::SEmpty + (n & 1)));
#pragma unroll
        for (int r = 0; r < H; ++r) v[r] = (__uint_as_float(hi[r]) + __uint_as_float(lo[r])) * factor * c_row[r];
      }
      if (rare(ragged)) {
#pragma unroll
        for (int r = 0; r < H; ++r) {
          const int lim = P.causal ? min(seg_end, L - P.s_q + 1 + pos_of[g * H + r]) : seg_end;
          if (tok >= lim) v[r] = -INFINITY;
        }
      }

      // ---- maxima over the tile: this warp's 32 tokens, then the four warps'
      float mine = -INFINITY;
#pragma unroll
      for (int r = 0; r < H; ++r) {
        const float x = warp_max(v[r] + log_of);
        if (lane == r) mine = x;
      }
      float* const mxb = mx + ((n & 1) * 2 + g) * 128;
      if (lane < H) mxb[quad * 32 + lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::Mx + 2 * g + (n & 1)));
      ok = warp_wait(bar(C::Mx + 2 * g + (n & 1)), (n >> 1) & 1, abort_flag);
      if (rare(!ok)) break;
      float root = 1.f;  // of the factor by which l moves
      if (lane < H) {
        const float m = fmaxf(fmaxf(mxb[lane], mxb[32 + lane]), fmaxf(mxb[64 + lane], mxb[96 + lane]));
        const float to = m > m_run + kSlack ? m : m_run;
        if (to != m_run) {
          root = root_of_move(m_run - to);  // 0 from -inf
          m_run = to;
        }
        bc[lane] = m_run == -INFINITY ? 0.f : -m_run;
        bc[32 + lane] = root;
      }
      const bool moved = __any_sync(0xffffffffu, root != 1.f || shift != 0);
      __syncwarp();

      // ---- weights: hi and lo bytes of four rows a register
      const float unit = ratio * kUnit;
      uint32_t ph[H / 4], pl[H / 4];
      if (moved) {
#pragma unroll
        for (int r = 0; r < H; ++r) l[r] = l[r] * bc[32 + r] * bc[32 + r];
      }
#pragma unroll
      for (int r = 0; r < H; r += 2) {
        const float p0 = ex2_approx(v[r] + bc[r]), p1 = ex2_approx(v[r + 1] + bc[r + 1]);
        l[r] += p0;
        l[r + 1] += p1;
        const float x0 = p0 * unit, x1 = p1 * unit;
        const uint32_t h = e4m3x2(x0, x1);
        const float2 b = e4m3x2_to_float2(h);
        const uint32_t t = e4m3x2(x0 - b.x, x1 - b.y);
        ph[r / 4] = r & 2 ? ph[r / 4] | h << 16 : h;
        pl[r / 4] = r & 2 ? pl[r / 4] | t << 16 : t;
      }
      // four lanes' 4 x 4 bytes turned over: lane k of them gets row k's bytes of the four tokens
#pragma unroll
      for (int r = 0; r < H / 4; ++r) {
        ph[r] = turn_4x4(ph[r], lane);
        pl[r] = turn_4x4(pl[r], lane);
      }

      // ---- what a hidden entry holds must not reach O by way of 0 x NaN: V past the
      // end becomes 0, and so do the NaN codes of a token that only some rows see (a
      // row that sees one is NaN by its score already)
      if (rare(ragged)) {
#pragma unroll 1
        for (int c = 2 * g; c < 2 * g + 2; ++c) {
          // S^T has read the slot, and nothing refills it before this tile's O^T
          const int q = 4 * n + c;
          ok = ok && warp_wait(bar(C::KFull + q % C::Slots), (q / C::Slots) & 1, abort_flag);
          uint4* const rowp = reinterpret_cast<uint4*>(gbase + C::OffK + q % C::Slots * kChunk + tl * 128);
          if (tok >= seg_end) {
#pragma unroll
            for (int x = 0; x < 8; ++x) rowp[x ^ (tl & 7)] = make_uint4(0, 0, 0, 0);
          } else if (tok >= all_see) {
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {
              const uint4 a = rowp[x ^ (tl & 7)];
              rowp[x ^ (tl & 7)] = make_uint4(without_nan(a.x), without_nan(a.y), without_nan(a.z), without_nan(a.w));
            }
          }
        }
      }

      if (rare(!ok)) break;

      // ---- once the previous product is done: move O, hand P over
      if (n > 0) {
        ok = warp_wait(bar(C::PvDone), (n - 1) & 1, abort_flag);
        if (rare(!ok)) break;
      }
      if (rare(!first && moved)) {
        tc_fence_after_sync();
        __syncwarp();
        if (lane < H) bc[32 + lane] = root * root * power_of_two(-shift);
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[H];
          const uint32_t at = tmem + lanes + (c >> 1) * C::OCols + (c & 1) * kR + g * H;
          tmem_ld(at, o);
          tmem_landed();
          hold(o);
#pragma unroll
          for (int r = 0; r < H; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * bc[32 + r]);
          tmem_st(at, o);
        }
        tmem_wait_st();
        tc_fence_before_sync();
      }
      {
        uint8_t* const pb = gbase + C::OffP + (g * H + (lane & 3)) * 128 + (tl & 12);
#pragma unroll
        for (int r = 0; r < H; r += 4) {  // row r + (lane & 3)
          const int at = r * 128 + (((tl >> 4) ^ ((r & 4) + (lane & 3))) << 4);
          *reinterpret_cast<uint32_t*>(pb + at) = ph[r / 4];
          *reinterpret_cast<uint32_t*>(pb + kR * 128 + at) = pl[r / 4];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::PFull));

      // ---- end of a segment: row sums over the four warps, O out
      if (rare(w.last())) {
        const int s0 = __ldg(P.num_splits + w.i);
        const bool whole = __ldg(P.num_splits + w.i + 1) - s0 == 1;
        const int64_t out_row = whole ? static_cast<int64_t>(w.i) * rows_total : (static_cast<int64_t>(s0) + w.k) * rows_total;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < H; ++r) {
          float x = l[r];
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
          if (lane == r) sum = x;
        }
        if (lane < H) ls[quad * 32 + lane] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::Ls + g));
        ok = warp_wait(bar(C::Ls + g), seg & 1, abort_flag);
        if (rare(!ok)) break;
        if (lane < H) {
          const float t = (ls[lane] + ls[32 + lane]) + (ls[64 + lane] + ls[96 + lane]);
          bc[lane] = t == 0.f ? 0.f : 1.f / (kUnit * t);  // and R apart: the two may be far below 2^-126 together
          const int row = row_of[g * H + lane];
          if (quad == 0 && row >= 0) {
            const float lse = t == 0.f ? -INFINITY : log_sum(m_run, t) * 0.69314718055994531f;
            if (whole) {
              const int j = pos_of[g * H + lane];
              P.lse[(static_cast<int64_t>(w.i) * P.h_q + (row - j * P.h_q)) * P.s_q + j] = lse;
            } else {
              P.ws_lse[out_row + row] = t == t ? lse : INFINITY;  // which the merge turns into NaN beside any other piece
            }
          }
        }
        __syncwarp();
        ok = warp_wait(bar(C::PvDone), n & 1, abort_flag);
        if (rare(!ok)) break;
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[H];
          const uint32_t at = tmem + lanes + c * C::OCols + g * H;
          tmem_ld(at, o);
          uint32_t lo[H];
          tmem_ld(at + kR, lo);
          tmem_landed();
          hold(o);
          hold(lo);
#pragma unroll
          for (int r = 0; r < H; ++r) o[r] = __float_as_uint((__uint_as_float(o[r]) + __uint_as_float(lo[r])) * bc[r] * bound);
          const int dim = c * 128 + tl;
          if (whole) {
            // two rows at a time: even lanes store a pair of dims of the first, odd lanes of the second
            __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(P.out) + out_row * kDimV + (dim & ~1);
#pragma unroll
            for (int r = 0; r < H; r += 2) {
              const float a = __uint_as_float(o[r]), b = __uint_as_float(o[r + 1]);
              const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
              const int row = row_of[g * H + r + (lane & 1)];
              if (row >= 0)
                *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(row) * kDimV) =
                    lane & 1 ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
            }
          } else {
            float* const dst = P.ws_o + out_row * kDimV + dim;
#pragma unroll
            for (int r = 0; r < H; ++r) {
              const int row = row_of[g * H + r];
              if (row >= 0) dst[static_cast<int64_t>(row) * kDimV] = __uint_as_float(o[r]);
            }
          }
        }
        tc_fence_before_sync();
      }
      ++n;
      w.advance();
    }
  } else if (warp < kSoftmaxWarps + kQWarps) {
    // ================================================= queries
    regs_dec<104>();
    const int qw = warp - kSoftmaxWarps;
    TileWalk w;
    w.start(meta, P.cache_seqlens, P.max_blocks);
    int seg = 0;
    while (w.valid) {
      const int qb = seg % C::QBufs;
      const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(P.q) + static_cast<int64_t>(w.i) * P.s_q * P.h_q * kDimQK;
      uint8_t* const qs = gbase + C::OffQ + qb * C::QBytes;
#pragma unroll 1
      for (int r0 = qw * 4; r0 < kR; r0 += kQWarps * 4) {
        const int r = r0 + (lane >> 3);
        const int row = row_of[r];
        const __nv_bfloat16* const at = src + static_cast<int64_t>(row < 0 ? 0 : row) * kDimQK;
        uint4 x[kQueryPieces / 8];  // eight lanes a row
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kQueryPieces / 8; ++k) x[k] = row >= 0 ? ld_global_nc_v4(at + (8 * k + (lane & 7)) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kQueryPieces / 8; ++k) m = query_max(m, x[k]);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int e = query_exponent(m);
        if (r0 < kQWarps * 4) ok = warp_wait(bar(C::QEmpty + qb), ((seg / C::QBufs) & 1) ^ 1, abort_flag);
        if (rare(!ok)) break;
#pragma unroll
        for (int k = 0; k < kQueryPieces / 8; ++k) store_query_piece<kR>(qs, r, 8 * k + (lane & 7), x[k], e);
        const float step = query_step(e);
        if ((lane & 7) == 0) reinterpret_cast<float*>(gbase + C::OffC)[seg % kCSlots * kR + r] = P.scale_log2 * step;
      }
      if (rare(!ok)) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::QFull + qb));
        // c_r is kept for eight segments: Q of segment s + 8 waits for the last
        // S^T of s + 6 at least, so for the softmax of a tile of s + 4 or later
        mbar_arrive(bar(C::CFull + seg % kCSlots));
      }
      ++seg;
      w.next_segment();
    }
  } else {
    regs_dec<64>();
    if (warp == 12) {
      // ================================================= TMA
      if (lane == 0) {
        tma_prefetch_desc(&lat_map);
        tma_prefetch_desc(&rope_map);
        const uint64_t evict_first = l2_policy_evict_first();
        auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t b, int x, int token) {
          // one row tile: a page is read once; two: the other finds it in L2
          if (row_tiles == 1)
            tma_load_3d_hint(dst, map, b, x, g_kv, token, evict_first);
          else
            tma_load_3d(dst, map, b, x, g_kv, token);
        };
        const int past = static_cast<int>(P.num_blocks * kPage);  // a coordinate outside: such a box is filled with zeros
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0, q = 0;
        while (w.valid && ok) {
          const int pages = min(2, w.p_end - w.p);
          int token[2] = {past, past};
          int64_t phys[2] = {0, 0};
          for (int e = 0; e < pages; ++e) {
            int id = __ldg(P.block_table + static_cast<int64_t>(w.i) * P.max_blocks + w.p + e);
            if (id < 0 || id >= P.num_blocks) {
              raise_status(P.status, kStatusBadBlockId);
              id = 0;
            }
            phys[e] = id;
            token[e] = id * kPage;
          }
          const int rs = n % kRopeSlots;
          ok = wait_on(bar(C::RopeEmpty + rs), ((n / kRopeSlots) & 1) ^ 1, abort_flag);
          if (rare(!ok)) break;
          // The scales of tile n sit in one of four slots.  S^T(n - 2) is done (its
          // rope slot is free), so the softmax has read the scales of tile n - 4.
          const uint32_t sb = bar(C::ScFull + (n & 3));
          mbar_arrive_expect_tx(sb, pages * kPage * 4);
          for (int e = 0; e < pages; ++e)
            bulk_load(base + C::OffScale + ((n & 3) * kTile + e * kPage) * 4, P.scales + (phys[e] * P.h_kv + g_kv) * kPage,
                      kPage * 4, sb);
          mbar_arrive_expect_tx(bar(C::RopeFull + rs), kRopeBytes);
          for (int e = 0; e < 2; ++e)
            load(base + C::OffRope + rs * kRopeBytes + e * (kRopeBytes / 2), &rope_map, bar(C::RopeFull + rs), kDimV, token[e]);
          ++n;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int s = q % C::Slots;
            ok = wait_on(bar(C::KEmpty + s), ((q / C::Slots) & 1) ^ 1, abort_flag);
            if (rare(!ok)) break;
            mbar_arrive_expect_tx(bar(C::KFull + s), kChunk);
            for (int e = 0; e < 2; ++e)
              load(base + C::OffK + s * kChunk + e * (kChunk / 2), &lat_map, bar(C::KFull + s), c * 128, token[e]);
            ++q;
          }
          w.advance();
        }
        // the last copies land before this CTA can exit, whoever gave up
        for (int m = max(0, q - C::Slots); m < q; ++m) drain_wait(bar(C::KFull + m % C::Slots), (m / C::Slots) & 1);
        for (int m = max(0, n - kRopeSlots); m < n; ++m) {
          drain_wait(bar(C::RopeFull + m % kRopeSlots), (m / kRopeSlots) & 1);
          drain_wait(bar(C::ScFull + (m & 3)), (m >> 2) & 1);
        }
      }
    } else if (warp == 13) {
      // ================================================= S^T
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3(2 * kR, false, false);
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0, q = 0, seg = -1;
        while (w.valid && ok) {
          if (w.first()) {
            ++seg;
            ok = wait_on(bar(C::QFull + seg % C::QBufs), (seg / C::QBufs) & 1, abort_flag);
            if (rare(!ok)) break;
          }
          const uint32_t qs = base + C::OffQ + (seg % C::QBufs) * C::QBytes;
          ok = wait_on(bar(C::SEmpty + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag);
          if (rare(!ok)) break;
          const int rs = n % kRopeSlots;
          ok = wait_on(bar(C::RopeFull + rs), (n / kRopeSlots) & 1, abort_flag);
          if (rare(!ok)) break;
          tc_fence_after_sync();
          const uint32_t d = tmem + kTmemS + (n & 1) * (2 * kR);
          {
            const uint64_t a = smem_desc(base + C::OffRope + rs * kRopeBytes, 0, 512, kSwizzle64B);
            const uint64_t b = smem_desc(qs + 4 * C::QChunk, 0, 512, kSwizzle64B);
            umma_e4m3(d, a, b, idesc, 0);
            umma_e4m3(d, a + 2, b + 2, idesc, 1);
          }
          umma_commit(bar(C::RopeEmpty + rs));
#pragma unroll 1
          for (int c = 0; c < 4; ++c, ++q) {
            const int s = q % C::Slots;
            ok = wait_on(bar(C::KFull + s), (q / C::Slots) & 1, abort_flag);
            if (rare(!ok)) break;
            const uint64_t a = smem_desc(base + C::OffK + s * kChunk, 0, 1024, kSwizzle128B);
            const uint64_t b = smem_desc(qs + c * C::QChunk, 0, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_e4m3(d, a + 2 * k, b + 2 * k, idesc, 1);
          }
          if (rare(!ok)) break;
          umma_commit(bar(C::SFull + (n & 1)));
          if (w.last()) umma_commit(bar(C::QEmpty + seg % C::QBufs));
          ++n;
          w.advance();
        }
        umma_commit(bar(C::Drain));
        drain_wait(bar(C::Drain), 0);
      }
    } else {
      // ================================================= O^T: dims below (14) and from 256 (15)
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3(C::OCols, true, false);
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0;
        while (w.valid && ok) {
          const bool first = w.first();
          ok = wait_on(bar(C::PFull), n & 1, abort_flag);
          if (rare(!ok)) break;
          tc_fence_after_sync();
          const uint64_t b = smem_desc(base + C::OffP, 0, 1024, kSwizzle128B);
#pragma unroll 1
          for (int c = 2 * (warp - 14); c < 2 * (warp - 13); ++c) {
            const int q = 4 * n + c, s = q % C::Slots;
            ok = wait_on(bar(C::KFull + s), (q / C::Slots) & 1, abort_flag);  // S^T waited already: this thread's acquire
            if (rare(!ok)) break;
            // MN-major: rows of 128 dims, 8 tokens every 1024 bytes
            const uint64_t a = smem_desc(base + C::OffK + s * kChunk, kChunk, 1024, kSwizzle128B);
            const uint32_t d = tmem + c * C::OCols;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 tokens
              umma_e4m3(d, a + k * (4096 >> 4), b + 2 * k, idesc, !first || k > 0);
            umma_commit(bar(C::KEmpty + s));
          }
          if (rare(!ok)) break;
          umma_commit(bar(C::PvDone));
          ++n;
          w.advance();
        }
        umma_commit(bar(C::Drain));
        drain_wait(bar(C::Drain), 0);
      }
    }
    __syncwarp();
  }
  if (!ok) raise_status(P.status, kStatusTimeout);
  __syncthreads();  // every wait above is bounded
  if (warp == 14) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kR>
cudaError_t launch(const DecodeKv8Params& p, const CUtensorMap& lat, const CUtensorMap& rope, int num_parts,
                   cudaStream_t stream) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(mla_decode_kv8_kernel<kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<kR>::Bytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const int row_tiles = (p.rows + kR - 1) / kR;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_parts * row_tiles, p.h_kv, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<kR>::Bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_decode_kv8_kernel<kR>, lat, rope, p, row_tiles);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Boxes of `dims` bytes of 64 entries of one head.
bool encode(CUtensorMap* map, const DecodeKv8Params& p, uint32_t dims, CUtensorMapSwizzle swizzle) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t entry = static_cast<cuuint64_t>(p.entry_bytes);
  const cuuint64_t size[3] = {kDimQK, static_cast<cuuint64_t>(p.h_kv), static_cast<cuuint64_t>(p.num_blocks) * kPage};
  const cuuint64_t stride[2] = {entry, entry * p.h_kv};
  const cuuint32_t box[3] = {dims, 1, kPage};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.codes), size, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool decode_kv8_in_pairs(int rows) { return rows > 64; }

int decode_kv8_ctas(int rows) { return rows <= 32 ? 1 : 2 * ((rows + 127) / 128); }

cudaError_t launch_decode_kv8(const DecodeKv8Params& p, int num_parts, cudaStream_t stream) {
  CUtensorMap lat, rope;
  if (!encode(&lat, p, 128, CU_TENSOR_MAP_SWIZZLE_128B) || !encode(&rope, p, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  // Columns cost tensor time and shared memory: the narrowest tile that holds the
  // rows, and up to 64 rows two CTAs of 32 rather than a half-empty pair: 60 rows (37
  // sequences of up to 3001 tokens) 32.0 us against 34.7, 64 rows 23.2 against 26.9 (16
  // sequences of 1024-4096), 113.9 against 115.2 (128 of 4096), 64.4 against 79.3 (512
  // of 100-300).
  if (p.rows <= 16) return launch<16>(p, lat, rope, num_parts, stream);
  if (!decode_kv8_in_pairs(p.rows)) return launch<32>(p, lat, rope, num_parts, stream);
  return launch_decode_kv8_pair(p, lat, rope, num_parts, stream);
}

}  // namespace mla
