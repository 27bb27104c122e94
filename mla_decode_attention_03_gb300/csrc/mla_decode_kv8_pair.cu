// The decode over the 8-bit cache for more than 64 query rows per KV head: two
// CTAs of a cluster share a tile of up to 128 rows, 64 rows each.  Same
// mathematics as mla_decode_kv8.cu (e4m3 codes as they lie, queries and weights
// as hi + lo, a weight's lo in e5m2); here with rows as rows:
//   S [128 rows x 128 tokens]  = q_hi K^T, q_lo K^T     two accumulators, added by the softmax
//   O [128 rows x 2 x 256 dims] += P_hi V + P_lo V
// by MMAs that span both SMs (cta_group::2, M = 128): each CTA holds its 64 rows
// of A and of the result, and each supplies half of B's columns, which the
// tensor cores of both read.
//
// A tile is two pages.  For S, CTA r supplies the tokens of page r, all 576
// dims; for O, the dims [256 r, 256 r + 256) of both pages.  Half of that it has
// already; the other page's half of the dims (16 KB) is loaded, once S is done,
// over the two of its own four chunks that O does not need here:
//                    chunk 0   chunk 1   chunk 2   chunk 3     (128 dims each)
//   CTA 0 for S      page 0    page 0    page 0    page 0      dims 0, 128, 256, 384
//   CTA 0 for O      page 0    page 0    page 1    page 1      dims 0, 128,   0, 128
//   CTA 1 for S      page 1    page 1    page 1    page 1      dims 0, 128, 256, 384
//   CTA 1 for O      page 0    page 0    page 1    page 1      dims 256, 384, 256, 384
// so that in both CTAs one address holds what one MMA needs, a tile takes 36 KB
// and three are in flight, and an SM takes in 53 KB per 128 tokens (an SM's
// loads reach about 41 GB/s on this GPU, 6.2 TB/s over all; two CTAs that both
// read every page would be bound there).
//
// In tensor memory a row is two lanes, l and l + 64: for S the tokens of page 0
// and of page 1, for O the dims below and from 256.  With four warpgroups each
// taking a quarter of the columns, eight threads share a row.
//
// A segment's queries, 73 KB as hi + lo, come from global memory in the form that
// the MMAs read: mla_kv8_queries_kernel makes them once per call (a few warps of
// each CTA, making them per segment, took 18,000 cycles a segment; as a kernel of
// its own they take 5 us of the 126, and converting them in here, by warps that are
// spare, at a segment's beginning or end or in place, 2 to 20 us more).
//
// Bound: the tensor cores' operand traffic (S reads 4 KB of shared memory per 32
// cycles of MMA, all that there is) and a tile's residence of about 10,000 cycles
// over the three that fit.  128 sequences of 4096 tokens, 128 heads: 126 us a call
// (ten in a graph; 134 as the only one, L2 cold), 1.16 PFLOP/s, the pipe busy 56% of
// this kernel's cycles.
//
// Warps (768 threads, one CTA per SM, 2 CTAs per cluster):
//   0-15   softmax and epilogue
//   16     TMA of the other page's half, once S is done; the scales' part in the weights
//   17     TMA of the own page, with its scales
//   18-20  in CTA 0: issue S_hi, S_lo, O (one thread issues an MMA per 64 cycles,
//          whatever its size, and S's take 32: two threads share them).
//          In CTA 1: tell CTA 0 what has landed.
//   21     copies of the segments' queries
#include <cudaTypedefs.h>

#include "mla_kv8_dev.cuh"

namespace mla {
namespace {

constexpr int kRows = 64;                        // per CTA
constexpr int kTiles = 3;                        // tiles in flight
constexpr int kCell = kPage * 128;               // 64 tokens x 128 dims
constexpr int kTileBytes = 4 * kCell + kPage * 64;
constexpr int kScaleSlots = 4;
constexpr int kCSlots = 4;
constexpr int kThreads = 768;  // six warpgroups, for the register split; two warps are spare
constexpr int kSoftmaxWarps = 16;
constexpr int kSlices = 8;                       // threads of a row: 16 tokens of a tile, or 64 dims, each
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;                 // two buffers of (hi 64, lo 64) columns; O: columns 0-255

// A weight is hi (e4m3) + lo (e5m2): off by 2^-4 2^-3 of itself at most, 1.2e-3 in
// the mean.  e5m2's wider range is what lets a maximum lag by 2^4.8: where hi is
// below its normal range, lo still holds it to 2^-13, 2^-17 of a weight of 1.
// (Both e4m3, with this slack: output errors of 3.1e-3 against 1.75e-3 where scales
// spread; with a slack of 2.8 and kUnit 64, 1.8e-3, and 2-4% more time.)
constexpr float kUnit = 16.f;
constexpr float kSlack = 4.8f;

constexpr int kQChunk = 2 * kRows * 128;         // hi rows, then lo rows
constexpr int kQBytes = 2 * kRows * kDimQK;
constexpr int kPBytes = 2 * kRows * kTile;       // hi rows, then lo rows

constexpr int kOffK = 0;
constexpr int kOffQ = kOffK + kTiles * kTileBytes;
constexpr int kOffP = kOffQ + kQBytes;
constexpr int kOffScale = kOffP + 2 * kPBytes;
constexpr int kOffMx = kOffScale + kScaleSlots * kTile * 4;  // float[2][kSlices][64] partial maxima, and row sums
constexpr int kOffUnit = kOffMx + 2 * kSlices * kRows * 4;             // float[kScaleSlots][3][128] scales; their part in the weights; its log2
constexpr int kOffBound = kOffUnit + 3 * kScaleSlots * kTile * 4;  // float[kScaleSlots][4] R, whether a scale is 0 or not finite, log2 of R's move
constexpr int kOffC = kOffBound + kScaleSlots * 16;          // float[kCSlots][64] c_r of the last segments
constexpr int kOffRow = kOffC + kCSlots * kRows * 4;         // int[64] row in the sequence
constexpr int kOffBar = kOffRow + kRows * 4;
// Barriers, in each CTA.  The kPeer ones are CTA 0's view of CTA 1, whose warps
// arrive there themselves.  What they hand over is in their own SM (shared memory
// that its tensor core reads, tensor memory), so these arrivals release at CTA
// scope; one that releases at cluster scope stalls its warp for over 1000 cycles.
enum : int {
  kLanded = 0,                     // own page: rope and chunks 0, 1, then chunks 2, 3, by tile slot
  kPeerLanded = kLanded + 2 * kTiles,
  kCrossed = kPeerLanded + 2 * kTiles,  // the other page's half, by tile slot
  kPeerCrossed = kCrossed + kTiles,
  kScaleFull = kPeerCrossed + kTiles,
  kUnitFull = kScaleFull + kScaleSlots,
  kQFull = kUnitFull + kScaleSlots,
  kPeerQFull = kQFull + 1,
  kQEmpty = kPeerQFull + 1,
  kCFull = kQEmpty + 1,
  kSFull = kCFull + kCSlots,
  kSEmpty = kSFull + 2,
  kPeerSEmpty = kSEmpty + 2,
  kPFull = kPeerSEmpty + 2,
  kPeerPFull = kPFull + 2,
  kOHalf = kPeerPFull + 2,         // by tile slot: the part of O from page 0 is done (and chunks 0, 1 free)
  kODone = kOHalf + kTiles,        // all of it
  kMx = kODone + kTiles,
  kLs = kMx + 2,
  kDrain = kLs + 1,
  kNumBars = kDrain + 1
};
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kBytes = kOffMisc + 16 + 1024;     // abort flag, tensor memory address; slack to align the base
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kTileBytes % 1024 == 0, "swizzle atoms");
static_assert(kOffScale % 16 == 0 && kOffUnit % 16 == 0 && kOffBar % 8 == 0 && kBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kAIsE5m2 = 1u << 7;           // in an instruction descriptor

__device__ __forceinline__ void umma2_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on this barrier of both CTAs when the MMAs issued so far by this thread are done.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}

// Arrives on a barrier of either CTA of the cluster (an address from mapa, or of
// this CTA), releasing at CTA scope.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16-byte pieces w[4 k .. 4 k + 3] of four lanes turned over: afterwards lane k
// of the four holds piece k of each, in their order.
__device__ __forceinline__ void turn_4x4x16(uint32_t* w, int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step <<= 1) {
    const bool odd = lane & step;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p & step) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t& a = w[4 * p + e];
        uint32_t& b = w[4 * (p + step) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a : b, step);
        if (odd)
          a = got;
        else
          b = got;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
mla_decode_kv8_pair_kernel(const __grid_constant__ CUtensorMap lat_map, const __grid_constant__ CUtensorMap rope_map,
                           const DecodeKv8Params P, const int row_tiles) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;  // the same in both CTAs
  uint8_t* const gbase = smem_raw + (base - raw_addr);
  auto bar = [&](int idx) -> uint32_t { return base + kOffBar + 8u * idx; };
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + kOffMisc);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kOffMisc + 8);

  const int tid = threadIdx.x;
  // The same in all lanes, and by the shuffle the compiler knows it: branches on it are then uniform, and so are the
  // operands of what is issued in them (128 heads, batch 128: 126.1 us a call; with tid >> 5 alone 132.4).
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int unit = blockIdx.x >> 1;
  const int part = unit / row_tiles;
  const int row0 = (unit - part * row_tiles) * (2 * kRows) + rank * kRows;
  const int g_kv = blockIdx.y;
  const int32_t* const meta = P.metadata + part * kMetaInts;
  int* const row_of = reinterpret_cast<int*>(gbase + kOffRow);  // row in the sequence's [s_q, h_q], -1 past the last
  auto leader = [&](int idx) -> uint32_t { return cluster_map(bar(idx), 0); };
  // a barrier of CTA 0: `at_home` from CTA 0's warps, `peer` from CTA 1's
  auto tell = [&](int at_home, int peer) { arrive_at(rank == 0 ? bar(at_home) : leader(peer)); };

  if (tid < kRows) {
    const int row = row0 + tid;
    const int j = row / P.heads_per_kv;
    row_of[tid] = row < P.rows ? j * P.h_q + g_kv * P.heads_per_kv + row - j * P.heads_per_kv : -1;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < 2 * kTiles; ++s) {
      mbar_init(bar(kLanded + s), 1);
      mbar_init(bar(kPeerLanded + s), 1);
    }
    for (int s = 0; s < kTiles; ++s) {
      mbar_init(bar(kCrossed + s), 1);
      mbar_init(bar(kPeerCrossed + s), 1);
      mbar_init(bar(kOHalf + s), 1);
      mbar_init(bar(kODone + s), 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(bar(kScaleFull + s), 1);
      mbar_init(bar(kUnitFull + s), 1);
    }
    for (int s = 0; s < kCSlots; ++s) mbar_init(bar(kCFull + s), 1);
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kPeerQFull), 1);
    mbar_init(bar(kQEmpty), 2);                            // S_hi's and S_lo's commits
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSFull + s), 2);
      mbar_init(bar(kSEmpty + s), kSoftmaxWarps + 1);  // the softmax warps and the cross loader
      mbar_init(bar(kPeerSEmpty + s), kSoftmaxWarps + 1);
      mbar_init(bar(kPFull + s), kSoftmaxWarps);
      mbar_init(bar(kPeerPFull + s), kSoftmaxWarps);
      mbar_init(bar(kMx + s), kSoftmaxWarps);
    }
    mbar_init(bar(kLs), kSoftmaxWarps);
    mbar_init(bar(kDrain), 3);
    fence_mbar_init();
  }
  if (warp == 20) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before_sync();
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory are there
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the queries, and what came before them: the schedule, the cache
  grid_launch_dependents();

  bool ok = true;
  if (warp < kSoftmaxWarps) {
    // ================================================= softmax and epilogue
    regs_inc<88>();
    const int g = warp >> 2, quad = warp & 3;
    const int page = quad >> 1;                            // of the tile, for S; half of the dims, for O
    const int row = (quad & 1) * 32 + lane;                // of this CTA
    const int slice = page * 4 + g;                        // one of the eight threads of a row
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    float* const mx = reinterpret_cast<float*>(gbase + kOffMx);
    const float* const scales = reinterpret_cast<const float*>(gbase + kOffScale);
    const float* const factors_of = reinterpret_cast<const float*>(gbase + kOffUnit);
    const float* const bounds = reinterpret_cast<const float*>(gbase + kOffBound);
    const int rows_total = P.s_q * P.h_q;
    const int pos = row0 + row < P.rows ? (row0 + row) / P.heads_per_kv : P.s_q - 1;

    TileWalk w;
    w.start(meta, P.cache_seqlens, P.max_blocks);
    int n = 0, seg = -1;
    float m_run = -INFINITY, neg = 0.f, l_run = 0.f, c = 0.f;  // neg: -m_run, or 0
    int seg_end = 0, all_see = 0, lim = 0;

    for (; w.valid; ++n, w.advance()) {
      const bool first = w.first();
      if (rare(first)) {
        ++seg;
        const int L = __ldg(P.cache_seqlens + w.i);
        seg_end = min(L, w.p_end * kPage);
        all_see = min(seg_end, P.causal ? L - P.s_q + 1 : L);  // tokens before it are seen by every row
        lim = min(seg_end, P.causal ? L - P.s_q + 1 + pos : L);
        m_run = -INFINITY;
        neg = 0.f;
        l_run = 0.f;
        ok = warp_wait(bar(kCFull + seg % kCSlots), (seg / kCSlots) & 1, abort_flag);
        if (rare(!ok)) break;
        c = fmaxf(reinterpret_cast<const float*>(gbase + kOffC)[seg % kCSlots * kRows + row], 0x1p-149f);  // -inf c stays -inf
      }
      const int t0 = w.p * kPage;
      const int tok0 = t0 + page * kPage + g * 16;         // this thread's 16 tokens
      const bool ragged = t0 + kTile > all_see;
      const int slot = n % kTiles;

      ok = warp_wait(bar(kUnitFull + (n & 3)), (n >> 2) & 1, abort_flag) &&
           warp_wait(bar(kSFull + (n & 1)), (n >> 1) & 1, abort_flag);
      if (rare(!ok)) break;
      tc_fence_after_sync();

      const uint32_t s_at = tmem + lanes + kTmemS + (n & 1) * 128 + g * 16;
      const float* const raw = scales + (n & 3) * kTile + page * kPage + g * 16;
      const float* const factors = factors_of + (n & 3) * (3 * kTile) + page * kPage + g * 16;
      const float* const bnd = bounds + 4 * (n & 3);
      if (rare(ragged || bnd[1] != 0.f)) {
        // Before they are read below, scores of hidden tokens become -inf, those of tokens
        // whose scale is not finite NaN, and those of scale 0 zero: the factor of the last
        // two is 1, for a hidden one may be among them, and -inf x 0 is NaN.
#pragma unroll 1
        for (int k = 0; k < 16; k += 8) {
          uint32_t x[8], y[8];
          tmem_ld(s_at + k, x);
          tmem_ld(s_at + 64 + k, y);
          tmem_landed();
          hold(x);
          hold(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!(raw[k + e] < INFINITY)) x[e] = 0x7fffffffu;
            if (!(raw[k + e] > 0.f)) {  // 0, or NaN
              x[e] = __float_as_uint((__uint_as_float(x[e]) + __uint_as_float(y[e])) * 0.f);
              y[e] = 0;
            }
            if (tok0 + k + e >= lim) {
              x[e] = 0xff800000u;
              y[e] = 0;
            }
          }
          tmem_st(s_at + k, x);
          tmem_st(s_at + 64 + k, y);
        }
        tmem_wait_st();
      }

      // ---- scores times scale, and the weights' maximum
      const uint64_t c2 = f2(c, c);
      uint64_t v[8];
      float m = -INFINITY;
      {
        uint32_t hi[16], lo[16];
        tmem_ld(s_at, hi);
        tmem_ld(s_at + 64, lo);
        tmem_landed();
        hold(hi);
        hold(lo);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) tell(kSEmpty + (n & 1), kPeerSEmpty + (n & 1));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const ulonglong2 s2 = reinterpret_cast<const ulonglong2*>(factors)[k];
          const ulonglong2 g2 = reinterpret_cast<const ulonglong2*>(factors + 2 * kTile)[k];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 4 * k + 2 * e;
            v[2 * k + e] = f2_mul(f2_add(f2(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1])),
                                         f2(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1]))),
                                  e ? s2.y : s2.x);
            float a, b;
            f2_split(f2_fma(v[2 * k + e], c2, e ? g2.y : g2.x), a, b);
            m = fmax3(m, a, b);
          }
        }
      }

      // ---- the row's maximum over its eight threads
      float* const mxb = mx + (n & 1) * (kSlices * kRows);
      mxb[slice * kRows + row] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kMx + (n & 1)));
      ok = warp_wait(bar(kMx + (n & 1)), (n >> 1) & 1, abort_flag);
      // P's buffer: the product that read it two tiles ago is done
      if (n >= 2) ok = ok && warp_wait(bar(kODone + (n - 2) % kTiles), ((n - 2) / kTiles) & 1, abort_flag);
      if (rare(!ok)) break;
      m = mxb[row];
#pragma unroll
      for (int k = 1; k < kSlices; ++k) m = fmaxf(m, mxb[k * kRows + row]);
      float root = 1.f, alpha = 1.f;  // l moves by root^2, O by alpha
      const float to = m > m_run + kSlack ? (first ? m : m + kMargin) : m_run;
      if (to != m_run) {
        root = root_of_move(m_run - to);  // 0 from -inf
        alpha = root * root;
        m_run = to;
        neg = -to;
      }
      if (rare(bnd[2] != 0.f)) alpha *= power_of_two(-static_cast<int>(bnd[2]));
      const bool moved = __any_sync(0xffffffffu, alpha != 1.f);

      // ---- weights as hi and lo bytes, a 16-byte unit of P's row, and their sum
      float sum;
      {
        const uint64_t n2 = f2(neg, neg), back = f2(-256.f, -256.f);
        uint64_t l2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const ulonglong2 u2 = reinterpret_cast<const ulonglong2*>(factors + kTile)[k];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a, b;
            f2_split(f2_fma(v[2 * k + e], c2, n2), a, b);
            const uint64_t p2 = f2(ex2_approx(a), ex2_approx(b));
            l2[e] = f2_add(l2[e], p2);
            const uint64_t x2 = f2_mul(p2, e ? u2.y : u2.x);
            float x0, x1;
            f2_split(x2, x0, x1);
            const uint32_t hb = e4m3x2(x0, x1);
            // the codes back as f16, 2^-8 times their value: cheaper than a conversion, as they are not negative
            const uint32_t hf = __byte_perm(hb, 0, 0x1404) >> 1;
            float f0, f1, r0, r1;
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                : "=f"(f0), "=f"(f1)
                : "r"(hf));
            f2_split(f2_fma(f2(f0, f1), back, x2), r0, r1);
            const uint32_t lb = e5m2x2(r0, r1);
            ph[k] = e ? __byte_perm(ph[k], hb, 0x5410) : hb;
            pl[k] = e ? __byte_perm(pl[k], lb, 0x5410) : lb;
          }
        }
        uint8_t* const pr = gbase + kOffP + (n & 1) * kPBytes + row * 128 + ((slice ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(pr) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        *reinterpret_cast<uint4*>(pr + kRows * 128) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
        float a, b;
        f2_split(f2_add(l2[0], l2[1]), a, b);
        sum = a + b;
      }
      l_run = l_run * root * root + sum;

      if (rare(ragged)) {
        // where a hidden entry may hold anything, NaN codes of V become 0 (a zero
        // weight would not silence them).  A row that sees such an entry is NaN by
        // its score already.
        const uint32_t phase = (n / kTiles) & 1;
        ok = warp_wait(bar(kLanded + 2 * slot), phase, abort_flag) && warp_wait(bar(kLanded + 2 * slot + 1), phase, abort_flag) &&
             warp_wait(bar(kCrossed + slot), phase, abort_flag);
        if (rare(!ok)) break;
        uint4* const half = reinterpret_cast<uint4*>(gbase + kOffK + slot * kTileBytes + tid * 64);
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const uint4 a = half[x ^ (lane & 3)];
          const uint4 b = make_uint4(without_nan(a.x), without_nan(a.y), without_nan(a.z), without_nan(a.w));
          if (a.x != b.x || a.y != b.y || a.z != b.z || a.w != b.w) half[x ^ (lane & 3)] = b;
        }
      }
      if (rare(!first && moved)) {
        // ---- O moves with the maximum, between two products
        ok = warp_wait(bar(kODone + (n - 1) % kTiles), ((n - 1) / kTiles) & 1, abort_flag);
        if (rare(!ok)) break;
        tc_fence_after_sync();
        const uint64_t f2f = f2(alpha, alpha);
        const uint32_t at = tmem + lanes + g * 64;
#pragma unroll 1
        for (int k = 0; k < 64; k += 32) {
          uint32_t o[32];
          tmem_ld(at + k, o);
          tmem_landed();
          hold(o);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x, y;
            f2_split(f2_mul(f2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), f2f), x, y);
            o[e] = __float_as_uint(x);
            o[e + 1] = __float_as_uint(y);
          }
          tmem_st(at + k, o);
        }
        tmem_wait_st();
        tc_fence_before_sync();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tell(kPFull + (n & 1), kPeerPFull + (n & 1));

      // ---- end of a segment: row sums over the eight threads, O out
      if (rare(w.last())) {
        const int s0 = __ldg(P.num_splits + w.i);
        const bool whole = __ldg(P.num_splits + w.i + 1) - s0 == 1;
        const int64_t out_row = whole ? static_cast<int64_t>(w.i) * rows_total : (static_cast<int64_t>(s0) + w.k) * rows_total;
        // the sums go where this tile's maxima were: all have read those once all have come to kLs
        if (lane == 0) mbar_arrive(bar(kLs));
        ok = warp_wait(bar(kLs), 0, abort_flag);
        mxb[slice * kRows + row] = l_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kLs));
        ok = ok && warp_wait(bar(kLs), 1, abort_flag);
        if (rare(!ok)) break;
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) t += mxb[k * kRows + row];
        const float inv = t == 0.f ? 0.f : 1.f / (kUnit * t), bound = bnd[0];  // the two may be far below 2^-126 together
        const int my_row = row_of[row];
        if (slice == 0 && my_row >= 0) {
          const float lse = t == 0.f ? -INFINITY : log_sum(m_run, t) * 0.69314718055994531f;
          if (whole)
            P.lse[(static_cast<int64_t>(w.i) * P.h_q + (my_row - pos * P.h_q)) * P.s_q + pos] = lse;
          else
            P.ws_lse[out_row + my_row] = t == t ? lse : INFINITY;  // which the merge turns into NaN beside any other piece
        }
        if (n >= 1) {
          ok = warp_wait(bar(kODone + (n - 1) % kTiles), ((n - 1) / kTiles) & 1, abort_flag);
          if (rare(!ok)) break;
        }
        ok = warp_wait(bar(kOHalf + slot), (n / kTiles) & 1, abort_flag) &&
             warp_wait(bar(kODone + slot), (n / kTiles) & 1, abort_flag);
        if (rare(!ok)) break;
        tc_fence_after_sync();
        const int dim0 = page * 256 + g * 64;
        int dst_row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dst_row[j] = row_of[(row & ~3) + j];
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint32_t o[32];
          tmem_ld(tmem + lanes + g * 64 + k * 32, o);
          tmem_landed();
          hold(o);
          const int dim = dim0 + k * 32;
          if (whole) {
            uint32_t b[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              b[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv * bound, __uint_as_float(o[2 * e + 1]) * inv * bound);
            turn_4x4x16(b, lane);
            __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(P.out) + out_row * kDimV + dim + (lane & 3) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (dst_row[j] >= 0)
                *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(dst_row[j]) * kDimV) =
                    make_uint4(b[4 * j], b[4 * j + 1], b[4 * j + 2], b[4 * j + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv * bound);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t* const q = o + 16 * h;
              turn_4x4x16(q, lane);
              float* const dst = P.ws_o + out_row * kDimV + dim + h * 16 + (lane & 3) * 4;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (dst_row[j] >= 0)
                  *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(dst_row[j]) * kDimV) =
                      make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
            }
          }
        }
        tc_fence_before_sync();
      }
    }
  } else {
    regs_dec<64>();  // here: all warps of a warpgroup have to execute the same one, and warps 16 and 17 share one
    if (warp == 16) {
      // ================================================= the other page's half of V; the weights' factors
      const uint64_t evict_first = l2_policy_evict_first();
      const int past = static_cast<int>(P.num_blocks * kPage);
      float* const units = reinterpret_cast<float*>(gbase + kOffUnit);
      float* const bounds = reinterpret_cast<float*>(gbase + kOffBound);
      TileWalk w, next;  // `next`: the tile whose factors are made next
      w.start(meta, P.cache_seqlens, P.max_blocks);
      next = w;
      int n = 0, m = 0;
      float bound = 1.f;
      bool nothing = false;
      // The scales, times kFactorUnit (1 past the end, and for one that is 0 or not finite), kUnit scale / R (0 there), and
      // log2(scale / R).  A row that sees a token whose scale is not finite gets a NaN score; to the others it is nothing.
      // Four slots: factors m + 4 are made once S(m + 3) is done, which waits until the softmax has left tile m.
      auto factors = [&]() {
        ok = warp_wait(bar(kScaleFull + (m & 3)), (m >> 2) & 1, abort_flag);
        if (!ok) return;
        const int L = __ldg(P.cache_seqlens + next.i), t0 = next.p * kPage, t = t0 + 4 * lane;
        const int end = min(L, next.p_end * kPage), all_see = P.causal ? min(end, L - P.s_q + 1) : end;
        const bool first = next.first();
        const float4 s4 = reinterpret_cast<const float4*>(gbase + kOffScale)[(m & 3) * 32 + lane];
        float s[4] = {s4.x, s4.y, s4.z, s4.w}, scale[4];
        bool odd = false;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool fine = t + e < end && s[e] > 0.f && s[e] < INFINITY;
          odd = odd || (t + e < end && !fine);
          scale[e] = fine ? fmaxf(s[e] * kFactorUnit, 0x1p-149f) : 1.f;
          if (!fine) s[e] = 0.f;
          if (t + e < all_see || (first && t + e == t0)) top = max(top, __float_as_uint(s[e]));
        }
        odd = __any_sync(0xffffffffu, odd);
        float shift = 0.f;
        if (rare(first || (nothing && t0 < all_see))) {
          top = __reduce_max_sync(0xffffffffu, top);
          nothing = is_nothing(top);
          const float r = reference_scale(top);
          if (!first) shift = static_cast<float>(log2_of_power(r) - log2_of_power(bound));
          bound = r;
        }
        const float u = 1.f / bound;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fminf(s[e] * u, kMaxRatio);
        float4* const to = reinterpret_cast<float4*>(units) + (m & 3) * 96 + lane;
        to[0] = make_float4(scale[0], scale[1], scale[2], scale[3]);
        to[32] = make_float4(s[0] * kUnit, s[1] * kUnit, s[2] * kUnit, s[3] * kUnit);
        to[64] = make_float4(log_ratio(s[0]), log_ratio(s[1]), log_ratio(s[2]), log_ratio(s[3]));
        if (lane == 0) {
          bounds[4 * (m & 3)] = bound;
          bounds[4 * (m & 3) + 1] = odd ? 1.f : 0.f;
          bounds[4 * (m & 3) + 2] = shift;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kUnitFull + (m & 3)));
        ++m;
        next.advance();
      };
      if (w.valid) factors();
      while (w.valid && ok) {
        ok = warp_wait(bar(kSFull + (n & 1)), (n >> 1) & 1, abort_flag);
        if (rare(!ok)) break;
        if (lane == 0) {
          // S(n + 2) waits for this arrival, so this phase cannot be missed
          tell(kSEmpty + (n & 1), kPeerSEmpty + (n & 1));
          const int p = w.p + 1 - rank;
          int token = past;
          if (p < w.p_end) {
            const int id = __ldg(P.block_table + static_cast<int64_t>(w.i) * P.max_blocks + p);
            token = id < 0 || id >= P.num_blocks ? 0 : id * kPage;  // reported by the CTA whose own page it is
          }
          const int slot = n % kTiles;
          mbar_arrive_expect_tx(bar(kCrossed + slot), 2 * kCell);
          for (int i = 0; i < 2; ++i) {
            const uint32_t dst = base + kOffK + slot * kTileBytes + (2 * (1 - rank) + i) * kCell;
            if (row_tiles == 1)
              tma_load_3d_hint(dst, &lat_map, bar(kCrossed + slot), (2 * rank + i) * 128, g_kv, token, evict_first);
            else
              tma_load_3d(dst, &lat_map, bar(kCrossed + slot), (2 * rank + i) * 128, g_kv, token);
          }
        }
        __syncwarp();
        ++n;
        w.advance();
        if (next.valid) factors();
      }
      if (lane == 0)  // the last copies land before this CTA can exit, whoever gave up
        for (int k = max(0, n - kTiles); k < n; ++k) drain_wait(bar(kCrossed + k % kTiles), (k / kTiles) & 1);
    } else if (lane == 0) {
      if (warp == 17) {
        // ================================================= the own page
        tma_prefetch_desc(&lat_map);
        tma_prefetch_desc(&rope_map);
        const int past = static_cast<int>(P.num_blocks * kPage);  // a coordinate outside: such a box is filled with zeros
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0, halves = 0;
        while (w.valid) {
          const int pages = min(2, w.p_end - w.p);
          int64_t phys[2] = {0, 0};
          for (int e = 0; e < pages; ++e) {
            int id = __ldg(P.block_table + static_cast<int64_t>(w.i) * P.max_blocks + w.p + e);
            if (id < 0 || id >= P.num_blocks) {
              raise_status(P.status, kStatusBadBlockId);
              id = 0;
            }
            phys[e] = id;
          }
          const int token = rank < pages ? static_cast<int>(phys[rank]) * kPage : past;
          const int slot = n % kTiles;
          const uint32_t dst = base + kOffK + slot * kTileBytes, b0 = bar(kLanded + 2 * slot), b1 = b0 + 8;
          if (n >= kTiles) ok = wait_on(bar(kOHalf + slot), (n / kTiles - 1) & 1, abort_flag);
          if (rare(!ok)) break;
          mbar_arrive_expect_tx(b0, kTileBytes - 2 * kCell);
          tma_load_3d(dst + 4 * kCell, &rope_map, b0, kDimV, g_kv, token);
          tma_load_3d(dst, &lat_map, b0, 0, g_kv, token);
          tma_load_3d(dst + kCell, &lat_map, b0, 128, g_kv, token);
          ++halves;
          // half of O(n - 3) is done, so the softmax has read the scales of tile n - 4
          mbar_arrive_expect_tx(bar(kScaleFull + (n & 3)), pages * kPage * 4);
          for (int e = 0; e < pages; ++e)
            bulk_load(base + kOffScale + ((n & 3) * kTile + e * kPage) * 4, P.scales + (phys[e] * P.h_kv + g_kv) * kPage,
                      kPage * 4, bar(kScaleFull + (n & 3)));
          if (n >= kTiles) ok = wait_on(bar(kODone + slot), (n / kTiles - 1) & 1, abort_flag);
          if (rare(!ok)) break;
          mbar_arrive_expect_tx(b1, 2 * kCell);
          tma_load_3d(dst + 2 * kCell, &lat_map, b1, 256, g_kv, token);
          tma_load_3d(dst + 3 * kCell, &lat_map, b1, 384, g_kv, token);
          ++n;
          w.advance();
        }
        for (int m = max(0, halves - kTiles); m < halves; ++m) {
          drain_wait(bar(kLanded + 2 * (m % kTiles)), (m / kTiles) & 1);
          if (m < n) drain_wait(bar(kLanded + 2 * (m % kTiles) + 1), (m / kTiles) & 1);
          drain_wait(bar(kScaleFull + (m & 3)), (m >> 2) & 1);
        }
      } else if (warp == 21) {
        // ================================================= queries
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int seg = 0;
        while (w.valid) {
          ok = wait_on(bar(kQEmpty), (seg & 1) ^ 1, abort_flag);
          if (rare(!ok)) break;
          const int64_t tile = ((static_cast<int64_t>(w.i) * P.h_kv + g_kv) * row_tiles + (unit - part * row_tiles)) * 2 + rank;
          // c_r is kept for four segments: Q of segment s + 4 waits for the last S of
          // s + 3, so for the softmax of a tile of s + 1 or later
          mbar_arrive_expect_tx(bar(kCFull + seg % kCSlots), kRows * 4);
          bulk_load(base + kOffC + seg % kCSlots * (kRows * 4), P.ws_c + tile * kRows, kRows * 4, bar(kCFull + seg % kCSlots));
          mbar_arrive_expect_tx(bar(kQFull), kQBytes);
          bulk_load(base + kOffQ, P.ws_q + tile * kQBytes, kQBytes, bar(kQFull));
          ++seg;
          w.next_segment();
        }
        if (seg > 0) drain_wait(bar(kQFull), (seg - 1) & 1);
        for (int m = max(0, seg - kCSlots); m < seg; ++m) drain_wait(bar(kCFull + m % kCSlots), (m / kCSlots) & 1);
      } else if (rank == 0 && warp < 20) {
        // ================================================= S_hi (18), S_lo (19)
        constexpr uint32_t idesc = idesc_e4m3(kTile, false, false);
        const int lo = warp - 18;
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0, seg = -1;
        while (w.valid) {
          if (w.first()) {
            ++seg;
            if (seg > 0) umma2_commit(bar(kQEmpty));  // the last segment's queries are read
            ok = wait_on(bar(kQFull), seg & 1, abort_flag) && wait_on<true>(bar(kPeerQFull), seg & 1, abort_flag);
            if (rare(!ok)) break;
          }
          const int slot = n % kTiles;
          const uint32_t phase = (n / kTiles) & 1;
          ok = wait_on(bar(kSEmpty + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag) &&
               wait_on<true>(bar(kPeerSEmpty + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag) &&
               wait_on(bar(kLanded + 2 * slot), phase, abort_flag) && wait_on<true>(bar(kPeerLanded + 2 * slot), phase, abort_flag);
          if (rare(!ok)) break;
          tc_fence_after_sync();
          const uint32_t d = tmem + kTmemS + (n & 1) * 128 + lo * 64;
          const uint32_t k0 = base + kOffK + slot * kTileBytes, q0 = base + kOffQ;
          {
            const uint64_t a = smem_desc(q0 + 4 * kQChunk + lo * (kRows * 64), 0, 512, kSwizzle64B);
            const uint64_t b = smem_desc(k0 + 4 * kCell, 0, 512, kSwizzle64B);
            umma2_e4m3(d, a, b, idesc, 0);
            umma2_e4m3(d, a + 2, b + 2, idesc, 1);
          }
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            if (i == 2) {
              ok = wait_on(bar(kLanded + 2 * slot + 1), phase, abort_flag) &&
                   wait_on<true>(bar(kPeerLanded + 2 * slot + 1), phase, abort_flag);
              if (rare(!ok)) break;
              tc_fence_after_sync();
            }
            const uint64_t a = smem_desc(q0 + i * kQChunk + lo * (kRows * 128), 0, 1024, kSwizzle128B);
            const uint64_t b = smem_desc(k0 + i * kCell, 0, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma2_e4m3(d, a + 2 * k, b + 2 * k, idesc, 1);
          }
          if (rare(!ok)) break;
          umma2_commit(bar(kSFull + (n & 1)));
          ++n;
          w.advance();
        }
      } else if (rank == 0 && warp == 20) {
        // ================================================= O
        constexpr uint32_t idesc = idesc_e4m3(256, false, true);
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0;
        while (w.valid) {
          const bool first = w.first();
          const int slot = n % kTiles;
          ok = wait_on(bar(kCrossed + slot), (n / kTiles) & 1, abort_flag) &&
               wait_on<true>(bar(kPeerCrossed + slot), (n / kTiles) & 1, abort_flag) &&
               wait_on(bar(kPFull + (n & 1)), (n >> 1) & 1, abort_flag) &&
               wait_on<true>(bar(kPeerPFull + (n & 1)), (n >> 1) & 1, abort_flag);
          if (rare(!ok)) break;
          tc_fence_after_sync();
          const uint64_t a = smem_desc(base + kOffP + (n & 1) * kPBytes, 0, 1024, kSwizzle128B);
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {  // 32 tokens: two steps a page
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // MN-major: rows of 128 dims, 8 tokens every 1024 bytes
              const uint64_t b = smem_desc(base + kOffK + slot * kTileBytes + (2 * (k >> 1) + i) * kCell + (k & 1) * 4096, kCell, 1024,
                                           kSwizzle128B);
              umma2_e4m3(tmem + i * 128, a + 2 * k, b, idesc, !first || k > 0);
              umma2_e4m3(tmem + i * 128, a + ((kRows * 128) >> 4) + 2 * k, b, idesc | kAIsE5m2, 1);
            }
            if (k == 1) umma2_commit(bar(kOHalf + slot));
          }
          umma2_commit(bar(kODone + slot));
          ++n;
          w.advance();
        }
      } else if (rank == 1 && warp < 21) {
        // ================================================= CTA 1: its page (18), the other's half (19), the queries (20)
        TileWalk w;
        w.start(meta, P.cache_seqlens, P.max_blocks);
        int n = 0, seg = 0;
        auto pass_on = [&](int from, int to, int phase) {
          ok = ok && wait_on(bar(from), phase & 1, abort_flag);
          if (ok) arrive_at(leader(to));
        };
        while (w.valid && ok) {
          const int slot = n % kTiles;
          if (warp == 18) {
            pass_on(kLanded + 2 * slot, kPeerLanded + 2 * slot, n / kTiles);
            pass_on(kLanded + 2 * slot + 1, kPeerLanded + 2 * slot + 1, n / kTiles);
          } else if (warp == 19) {
            pass_on(kCrossed + slot, kPeerCrossed + slot, n / kTiles);
          } else if (w.first()) {
            pass_on(kQFull, kPeerQFull, seg++);
          }
          ++n;
          w.advance();
        }
      }
      if (rank == 0 && warp >= 18 && warp <= 20) {  // every MMA is done before tensor memory goes
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar(kDrain)) : "memory");
        drain_wait(bar(kDrain), 0);
      }
    }
    __syncwarp();
  }
  if (!ok) raise_status(P.status, kStatusTimeout);
  __syncthreads();  // every wait above is bounded
  tc_fence_before_sync();
  cluster_sync();   // and no arrival of the other CTA is still to come
  if (warp == 20) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// The queries in the form that the MMAs read, and c_r, 64 rows (one CTA's) a tile;
// rows past the last are zero.  Eight lanes take a row.
constexpr int kQueryWarps = 4;
constexpr int kQueryRows = 4 * kQueryWarps;  // a block

__global__ void __launch_bounds__(32 * kQueryWarps, 8) mla_kv8_queries_kernel(const DecodeKv8Params P, const int row_tiles) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int64_t tile = blockIdx.x / (kRows / kQueryRows);
  const int r = blockIdx.x % (kRows / kQueryRows) * kQueryRows + (threadIdx.x >> 3);
  const int row = static_cast<int>(tile % (2 * row_tiles)) * kRows + r;
  const int64_t seq_head = tile / (2 * row_tiles);
  const int64_t i = seq_head / P.h_kv;
  const int g_kv = static_cast<int>(seq_head - i * P.h_kv);
  const int j = row / P.heads_per_kv;
  const int64_t at = (i * P.s_q + j) * P.h_q + g_kv * P.heads_per_kv + row - j * P.heads_per_kv;
  const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(P.q) + at * kDimQK + l * 8;
  constexpr int kEach = kQueryPieces / 8;
  uint4 x[kEach];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) x[k] = row < P.rows ? ld_global_nc_v4(src + k * 64) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < kEach; ++k) m = query_max(m, x[k]);
#pragma unroll
  for (int step = 1; step < 8; step <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, step));
  const int e = query_exponent(m);
#pragma unroll
  for (int k = 0; k < kEach; ++k) store_query_piece<kRows>(P.ws_q + tile * kQBytes, r, k * 8 + l, x[k], e);
  if (l == 0) P.ws_c[tile * kRows + r] = P.scale_log2 * query_step(e);
}

cudaError_t configure() {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || configured_device == dev) return e;
  e = cudaFuncSetAttribute(mla_decode_kv8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e == cudaSuccess) configured_device = dev;
  return e;
}

}  // namespace

static size_t query_tiles(int b, int h_kv, int rows) {
  return decode_kv8_in_pairs(rows) ? static_cast<size_t>(b) * h_kv * (2 * ((rows + 2 * kRows - 1) / (2 * kRows))) : 0;
}

size_t decode_kv8_factors_at(int b, int h_kv, int rows) { return query_tiles(b, h_kv, rows) * kQBytes; }

size_t decode_kv8_query_bytes(int b, int h_kv, int rows) { return query_tiles(b, h_kv, rows) * (kQBytes + kRows * 4); }

cudaError_t launch_decode_kv8_pair(const DecodeKv8Params& p, const CUtensorMap& lat, const CUtensorMap& rope, int num_parts,
                                   cudaStream_t stream) {
  const cudaError_t e = configure();
  if (e != cudaSuccess) return e;
  const int row_tiles = (p.rows + 2 * kRows - 1) / (2 * kRows);
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * row_tiles) * p.b * p.h_kv * (kRows / kQueryRows), 1, 1);
    cfg.blockDim = dim3(32 * kQueryWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t r = cudaLaunchKernelEx(&cfg, mla_kv8_queries_kernel, p, row_tiles);
    if (r != cudaSuccess) return r;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_parts * row_tiles, p.h_kv, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mla_decode_kv8_pair_kernel, lat, rope, p, row_tiles);
}

}  // namespace mla
