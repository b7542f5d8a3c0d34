// Attention of a drafted block (or tree) over a paged 8-bit cache.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i . k_j)
//
// over the sequence's cached tokens (all of them) and its new tokens: j <= i
// of a block, or i's ancestors of a tree. Cached keys and values are e4m3 codes
// with a scale per page and head; the new ones are bfloat16.
//
// Two launches. cached_kernel leaves float32 partial sums over the cached tokens
// in the workspace, finish_kernel adds the new tokens and joins the partials.
//
// Bound. A cached token costs 2 D bytes per KV head and 4 D flops per query row
// (rows = new tokens x query heads per KV head): the stream of codes (HBM)
// bounds the call as long as products and exponentials of a 128-token tile
// stay under the 1420 clocks in which an SM's share of the bandwidth brings it.
//
// Split. The work items are (sequence, KV head, tile of 128 query rows), each a
// list of 128-token tiles of the cache. The items form one line, each as long as
// its tiles and kLead units for its start, that the CTAs share out evenly, whatever
// the lengths of the sequences; a CTA's part starts and ends inside items. (Lengths
// are on the device: a split planned on the host would have to assume the longest.)
//
// Products. tcgen05, rows on the 128 TMEM lanes. Scores: kind::f8f6f4 on the codes
// as they are; the queries are split into two e4m3 parts, q 2^s = hi + lo
// (bfloat16's 8 bits are two signed 4-bit halves; 2^s brings the row's largest
// into [128, 256), and half of e4m3's smallest step 2^-9, which is dropped, is at most
// 2^-17 of it). Weighted values: kind::f16, weights rounded to half (2^-11; kHead says
// how they are scaled) as the A operand in TMEM over the scores they came from, values
// decoded to half in shared memory by warps of their own (exact: e4m3 is a subset). With weights in e4m3 parts
// the decode would go, but splitting a weight costs the softmax warps more than
// the decode costs (7 clocks an element against 1).
//
// Softmax. A lane holds a row, and the warps of a lane quarter share the tile's
// tokens and its ref, each with a sum of its own. Value scales go into the exponent:
// t = score log2(e) + log2(v_scale), p = 2^(t - ref), and the normaliser sums
// p / v_scale in float32. ref moves only when a tile's largest t exceeds it by kTop (then o and
// l are rescaled and the tile's weights taken again), so the common tile is one
// pass over the scores. With 17 to 64 (32) rows the lanes hold 2 (4) copies of
// them, and each copy takes its half (quarter) of a tile's tokens: a warp's work
// per tile falls with the rows, and the copies' sums are joined like those of
// CTAs.
//
// Few rows. Up to 16 rows (a decode step's single tokens: the query heads of a KV
// head) the sides are swapped: the tile's tokens are on the lanes, the rows are 16
// columns. Keys are then the A operand as they lie, the queries' parts B in shared
// memory; values (D x tokens) are A, the weights B, written to shared memory as
// half. The products take an eighth of the tensor pipe's time and of the scores
// nothing is computed twice, so the stream of codes is what is left (32 single
// tokens of lengths 1 to 8191: 64 us against 82 with row copies).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sm100.cuh"
#include "uno.h"
#include "uno_device.cuh"
#include "uno_host.h"

namespace {

constexpr int kTile = 128;     // cached tokens per unit of work
constexpr int kRows = 128;     // rows (TMEM lanes) of a tile
constexpr int kProducers = 2;  // TMA warps, alternating tiles
// Warps of cached_kernel: 4 parts() for the softmax (TMEM lane quarter = warp % 4, part
// of a row's tokens = warp / 4), decoders() for the value decode (the first four of them
// for the queries too), the producers, and two MMA issuers (scores; weighted values): a
// thread that has issued products waits at its next barrier until they are done, so one
// issuer would leave the tensor pipe idle between the two.
// (`copies` 3 stands for tokens on the lanes in two parts, of the rows.)
__host__ __device__ constexpr int parts(int copies) { return copies == 1 ? 4 : copies == 3 ? 2 : 1; }
__host__ __device__ constexpr int decoders(int copies) { return copies == 1 ? 4 : 8; }
constexpr int threads(int copies) {
  return 32 * (4 * parts(copies) + decoders(copies) + kProducers + 2);
}
constexpr int kMaxCtas = 148;  // one CTA per SM
constexpr int kMaxT = 4096;    // new tokens per sequence
constexpr long long kWaitClocks = 2000000000ll;  // bound of every wait: about a second
constexpr int kStages = 4;     // tiles of codes in shared memory
constexpr int kCachedSeqs = 512;  // sequences whose sizes a CTA keeps in shared memory
// Up to so many rows the tokens take the TMEM lanes: the products are 16 columns wide
// instead of 128, and the softmax has no lanes to fill. Its work grows with the rows,
// though, a warp's 32 tokens at a time (64 sequences of 2040 to 4000 tokens, 8 KV heads;
// us with tokens and with row copies on the lanes: 4 rows 105 and 132, 8 rows 111 and
// 133, 16 rows 129 and 138; 48 rows 190 and 178, 68 rows 305 and 192).
constexpr int kFewRows = 16;
constexpr float kLog2e = 1.4426950408889634f;
// Units that an item's start counts for, in tiles (32 single tokens of lengths 1 to
// 8191: 64 us with 2 to 5; a tree of 241 nodes over 5001: 47 us with 2, 44 with 5).
constexpr int kLead = 5;
// A row's weights are scaled so that the largest when its ref is set is 2^kHead, and may grow
// to 2^kTop (half ends just below 2^16) before the ref moves. The head is for long
// caches that one token dominates: half keeps its 11 bits down to 2^-14, so down to 2^-23 of
// the largest weight, and is off by 2^-34 of it below. (With the largest at 1, each of 131072
// tokens that share 1% was 1.3 of half's smallest steps, and a quarter of their sum was lost.)
// The rest of half's range is for the maxima of later tiles: 64 sequences of 17 rows take
// 182 us with heads of 7 to 9, 188 with 10, 213 with 11 and a top of 15.
constexpr float kHead = 9.f, kTop = 15.9f;
// Floor of a row's ref: a tile without a finite score leaves it there.
constexpr float kLowest = -3.0e38f;

enum : unsigned { kFaultProducer = 8u, kFaultMma = 16u, kFaultSoftmax = 32u };
__device__ unsigned int g_attn_fault;
constexpr int kLost = -1;  // how many, of an item whose CTA had given up before it

struct AttnArgs {
  const uint16_t* q;      // [B][T][Hq][D]
  const uint16_t* k_new;  // [B][T][Hkv][D]
  const uint16_t* v_new;
  uint16_t* out;          // [B][T][Hq][D]
  const float* k_scale;   // [num_pages][Hkv]
  const float* v_scale;
  const int32_t* table;   // [B][width]
  const int32_t* lens;    // [B]
  const int32_t* parent;  // [B][T] or null
  const int32_t* num_new; // [B] or null
  int B, T, Hq, Hkv, G, page, width, num_pages;
  int copies;             // of the rows on the lanes: 4, 2 or 1
  float scale;            // softmax scale
  int query_segments;     // parts of a CTA whose queries are announced (all, but in tests)
  // workspace: partial sums of parts that begin an item, [B][Hkv][copies][T G], and
  // of those that begin inside one (a CTA's first), [CTA][128 lanes]; per item
  // [B][Hkv][row tiles] the CTAs of the latter, (first, how many), or kLost
  int2* item_ctas;
  float2* item_ml;        // (ref, normaliser)
  float* item_o;          // [..][D]
  float2* cta_ml;
  float* cta_o;
};

// A sequence's share of the line of units.
struct Seq {
  int len;    // cached tokens (0 when invalid)
  int nn;     // new tokens
  int tiles;  // per item
  int rts;    // row tiles
  bool bad;   // length outside the page table: the rows come out as NaN
  long long units;
};

__device__ __forceinline__ Seq seq_from(const AttnArgs& a, int len, int num_new) {
  Seq s;
  s.len = len;
  s.bad = s.len < 0 || s.len > a.width * a.page;
  if (s.bad) s.len = 0;
  s.nn = min(max(num_new, 0), a.T);
  s.tiles = (s.len + kTile - 1) / kTile;
  s.rts = (s.nn * a.G + kRows - 1) / kRows;
  s.units = s.tiles ? static_cast<long long>(a.Hkv) * s.rts * (s.tiles + kLead) : 0;
  return s;
}

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  return seq_from(a, a.lens[b], a.num_new ? a.num_new[b] : a.T);
}

__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes (low, high byte of 16 bits) as a half pair.
__device__ __forceinline__ uint32_t halves(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ bool nonfinite2(uint32_t w) {  // either bfloat16 of a pair
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}


__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 floats(uint32_t halves2) {
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(halves2));
  return f;
}

// The queries' two e4m3 parts, q 2^sh = hi + lo with the row's largest magnitude (top, its
// bfloat16 bits) in [128, 256), and what takes their scores back to log2 of a weight.
__device__ __forceinline__ int query_shift(uint32_t top) {
  return min(7 + 127 - static_cast<int>(top >> 7), 120);
}
__device__ __forceinline__ float query_factor(float scale, uint32_t top, int sh) {
  // an infinite or NaN query saturates in e4m3: its scores are NaN instead
  return top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                        : scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
}
__device__ __forceinline__ void split_e4m3(uint32_t pair, float f, uint32_t& hi, uint32_t& lo) {
  const float x = bf_lo(pair) * f, y = bf_hi(pair) * f;
  hi = e4m3x2(x, y);
  const float2 back = floats(halves(hi));
  lo = e4m3x2(x - back.x, y - back.y);
}

__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(sm100::smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One thread waits for the phase with the given parity, giving up after about a
// second (false then). It polls with test_wait: try_wait may suspend the thread, and
// waking it took 500 to 600 clocks of a tile's 1900.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity) {
  if (phase_done(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (phase_done(bar, parity)) return true;
    if ((it & 255u) == 0 && clock64() - t0 > kWaitClocks) return false;
  }
}

// The whole warp waits. The lanes poll together: none runs ahead of one that still
// has copies to issue, and each has seen the phase for itself.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  __syncwarp();
  if (__all_sync(0xFFFFFFFFu, phase_done(bar, parity))) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xFFFFFFFFu, phase_done(bar, parity))) return true;
    if ((it & 255u) == 0 && __any_sync(0xFFFFFFFFu, clock64() - t0 > kWaitClocks)) return false;
  }
}

// The softmax warps of a TMEM lane quarter meet (they take the same path throughout,
// on the give-up path too, so none is ever missing).
template <int PARTS>
__device__ __forceinline__ void meet(int quarter) {
  if constexpr (PARTS > 1)
    asm volatile("bar.sync %0, %1;" ::"r"(quarter + 1), "n"(32 * PARTS) : "memory");
}

// TMEM loads and stores of N consecutive columns (one lane per thread).
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    sm100::tmem_ld_32x32b_x32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

// R (a multiple of 4) consecutive columns.
template <int R>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
  if constexpr (R >= 16) {
    tmem_ld<16>(taddr, r);
    if constexpr (R > 16) tmem_ld_cols<R - 16>(taddr + 16, r + 16);
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
    if constexpr (R > 4) tmem_ld_cols<R - 4>(taddr + 4, r + 4);
  }
}
template <int R>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
  if constexpr (R > 4) tmem_st_cols<R - 4>(taddr + 4, r + 4);
}

// D[tmem] (+)= A[smem desc] B[smem desc] on e4m3 codes, one thread.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem desc], one thread. kF8: kind::f8f6f4, else kind::f16.
template <bool kF8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       bool accumulate) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    sm100::tmem_st_32x32b_x32(taddr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]));
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
  }
}

// Shared-memory descriptors. Codes of a tile of keys: K-major rows of D bytes (one
// row per token), swizzled by TMA over the row's bytes (128 or 64), 8-row groups
// 8 D bytes apart. Decoded values: MN-major, D on the MN side in atoms of 64
// halves (128-byte rows, one per token, 128-byte swizzle): groups of 8 tokens
// 1024 bytes apart (stride offset), the second 64 columns behind the tile's
// tokens (leading offset).
template <int D>
__device__ __forceinline__ uint64_t key_desc(uint32_t saddr) {
  uint64_t d = (saddr >> 4) & 0x3FFFu;
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>((8 * D) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(D == 128 ? 2u : 4u) << 61;
  return d;
}
template <bool kTwice = false>  // kTwice: the first 64 columns again for the second
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
  uint64_t d = (saddr >> 4) & 0x3FFFu;
  d |= static_cast<uint64_t>(kTwice ? 0 : (kTile * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Shared memory: [stage]{keys, values}, two tiles of decoded values, scales
// [stage][16-token group], the rows' score factors [segment parity][lane], what the
// parts of a row tell each other, barriers.
template <int D, int FEW = 0>
struct Plan {
  static constexpr int kStage = 2 * kTile * D;
  static constexpr int kHalfTile = kTile * D * 2;
  static constexpr int kDecoded = kStages * kStage;
  // (few rows) [segment parity][part][kFewRows][D] codes; [tile parity] weights
  static constexpr int kQueries = kDecoded + 2 * kHalfTile;
  static constexpr int kQueryPart = kFewRows * D;
  static constexpr int kWeights = kQueries + (FEW ? 4 * kQueryPart : 0);
  static constexpr int kWeightTile = kFewRows * kTile * 2;
  static constexpr int kScales = kWeights + (FEW ? 2 * kWeightTile : 0);
  static constexpr int kFactors = kScales + kStages * (kTile / 16) * 16;
  static constexpr int kTops = kFactors + 2 * kRows * 4;  // [part][lane], or [quarter][row]
  static constexpr int kRefs = kTops + 4 * kRows * 4;  // (few rows) [quarter][row]
  static constexpr int kFlags = kRefs + (FEW ? 4 * kFewRows * 4 : 0);  // [tile parity][quarter][part]
  static constexpr int kBars = kFlags + 2 * 4 * 4 * 4;
  static constexpr int kBytes = kBars + (2 * kStages + 8) * 8 + 8 + 1024;  // + alignment
  static_assert(kBytes + 2 * 4 * kCachedSeqs + 128 <= 232448, "dynamic shared memory per CTA (227 KB)");
};

// Row of a tile that a TMEM lane holds: with 4 copies of at most 32 rows, with 2 of
// at most 64.
template <int COPIES>
__device__ __forceinline__ int row_of_lane(int lane) {
  return lane & (kRows / COPIES - 1);
}

// FEW > 0: at most FEW rows, tokens on the lanes (COPIES then says the warps' roles, and
// the sums are one copy).
template <int D, int COPIES, int FEW>
__global__ void __launch_bounds__(threads(COPIES), 1)
    cached_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttnArgs a) {
  using P = Plan<D, FEW>;
  constexpr int CW = kTile / COPIES;  // a row copy's tokens per tile
  constexpr int PARTS = parts(COPIES);
  constexpr int HC = CW / PARTS;      // a softmax thread's
  constexpr int DECODERS = decoders(COPIES);
  constexpr int kFirstDecode = 4 * PARTS, kFirstProducer = kFirstDecode + DECODERS;
  constexpr int kMmaWarp = kFirstProducer + kProducers;  // scores (and TMEM); + 1: values
  // TMEM columns: two score tiles, o, then either the queries' parts of two segments,
  // with a tile's weights over its scores, or those of one segment and weights of
  // their own. The latter (row copies) lets a tile's scores follow as soon as the one two
  // before has been read, without its weighted values, for a softmax that is shorter
  // than the products; the next segment's queries then come late, but the epilogue of
  // the segment before takes longer still.
  constexpr bool kOwnWeights = COPIES > 1 || FEW > 0;
  constexpr bool kLateQueries = COPIES > 1 && !FEW;
  constexpr uint32_t kColO = 2 * kTile, kColQ = kColO + D, kColP = kColQ + D / 2;
  static_assert(kColQ + D <= 512 && kColP + kTile / 2 <= 512, "TMEM columns");
  constexpr uint32_t kIdescS = (1u << 4) | ((kTile >> 3) << 17) | ((kRows >> 4) << 24);
  constexpr uint32_t kIdescO =
      (1u << 4) | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((kRows >> 4) << 24);
  // few rows: keys (tokens x D) times queries, and values (D x tokens, the values'
  // descriptor on the A side) times weights
  constexpr uint32_t kColFewO = 2 * kFewRows;
  constexpr uint32_t kIdescFewS = (1u << 4) | ((kFewRows >> 3) << 17) | ((kRows >> 4) << 24);
  constexpr uint32_t kIdescFewO =
      (1u << 4) | (1u << 15) | ((kFewRows >> 3) << 17) | ((kRows >> 4) << 24);
  constexpr uint32_t kTmemCols = FEW ? 64 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float4* s_scale = reinterpret_cast<float4*>(smem + P::kScales);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBars);  // codes and scales are there
  uint64_t* empty = full + kStages;   // nobody needs them any more
  uint64_t* s_full = empty + kStages; // [2] scores of a tile
  uint64_t* pv_full = s_full + 2;     // [2] weights and decoded values of a tile
  uint64_t* o_done = pv_full + 2;     // [2] a tile's weighted values are in o
  uint64_t* q_full = o_done + 2;      // [2] a segment's queries
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(q_full + 2);
  float* s_factor = reinterpret_cast<float*>(smem + P::kFactors);
  float* s_top = reinterpret_cast<float*>(smem + P::kTops);
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + P::kFlags);
  __shared__ uint64_t s_end;          // every MMA has completed
  __shared__ long long s_total, s_u0, s_u1, s_base;
  __shared__ int s_b, s_ctas;
  __shared__ int s_size[2][kCachedSeqs];  // cached and new tokens
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&empty[s], 4 * PARTS + DECODERS + 1);  // softmax and decode warps, a commit
    }
    for (int k = 0; k < 2; ++k) {
      sm100::mbar_init(&s_full[k], 1);
      sm100::mbar_init(&pv_full[k], 4 * PARTS + DECODERS);  // softmax and decode warps
      sm100::mbar_init(&o_done[k], 1);
      sm100::mbar_init(&q_full[k], 4);
    }
    sm100::mbar_init(&s_end, 2);  // one commit per issuer
    s_abort = 0;
    sm100::fence_mbar_init();
  }
  if (warp == kMmaWarp) sm100::tmem_alloc(tmem_holder, kTmemCols);
  if (warp == kFirstProducer && lane < 2) sm100::tma_prefetch_desc(lane ? &map_v : &map_k);
  uno::grid_dependency_wait();
  // finish_kernel may start: what it reads before its own wait is older than this launch
  uno::launch_dependents();

  const bool small = a.B <= kCachedSeqs;
  if (small) {
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
      s_size[0][i] = a.lens[i];
      s_size[1][i] = a.num_new ? a.num_new[i] : a.T;
    }
    __syncthreads();
  }
  auto seq = [&](int i) {
    return small ? seq_from(a, s_size[0][i], s_size[1][i]) : seq_of(a, i);
  };
  // This CTA's part [u0, u1) of the line, and the sequence it starts in.
  if (warp == 0) {
    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long long n = b0 + lane < a.B ? seq(b0 + lane).units : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
      total += n;
    }
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    const int i = blockIdx.x;
    const long long u0 = i < ctas ? total * i / ctas : total;
    const long long u1 = i < ctas ? total * (i + 1) / ctas : total;
    long long base = 0;
    int at = 0;
    for (int b0 = 0; u0 < u1; b0 += 32) {  // ends: u0 < total
      const long long n = b0 + lane < a.B ? seq(b0 + lane).units : 0;
      long long pre = n;  // inclusive prefix over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, pre, o);
        if (lane >= o) pre += up;
      }
      const unsigned in = __ballot_sync(0xFFFFFFFFu, u0 < base + pre);
      if (in) {
        const int l = __ffs(in) - 1;
        base += __shfl_sync(0xFFFFFFFFu, pre - n, l);
        at = b0 + l;
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, pre, 31);
    }
    if (lane == 0) {
      s_total = total;
      s_ctas = ctas;
      s_u0 = u0;
      s_u1 = u1;
      s_base = base;
      s_b = at;
    }
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const long long u0 = s_u0, u1 = s_u1;

  // A segment: the part of one item that this CTA does.
  struct Segment {
    Seq s;
    int b, h, rt, t0, t1;  // tiles [t0, t1) of the item (none, when it has only lead units)
    long long end;         // the line's unit behind the segment, and behind the item
    long long item_end;
  };
  long long base = s_base;
  int b = s_b;
  auto segment_at = [&](long long u) {
    Segment g;
    g.s = seq(b);
    while (u >= base + g.s.units) {
      base += g.s.units;
      g.s = seq(++b);
    }
    g.b = b;
    const int len = g.s.tiles + kLead;
    const long long rel = u - base;
    const int item = rel < 0x7FFFFFFF ? static_cast<int>(rel) / len : static_cast<int>(rel / len);
    const long long start = base + static_cast<long long>(item) * len;
    g.item_end = start + len;
    g.end = min(u1, g.item_end);
    g.t0 = max(static_cast<int>(u - start) - kLead, 0);
    g.t1 = max(static_cast<int>(g.end - start) - kLead, 0);
    g.h = item / g.s.rts;
    g.rt = item - g.h * g.s.rts;
    return g;
  };
  // The next segment with tiles at or behind u (u behind it on return); false at the end.
  auto next_segment = [&](long long& u, Segment& g) {
    while (u < u1) {
      g = segment_at(u);
      u = g.end;
      if (g.t1 > g.t0) return true;
    }
    return false;
  };
  auto give_up = [&](unsigned bit) {
    if (lane == 0) atomicOr(&g_attn_fault, bit);
    s_abort = 1;
  };

  if (warp >= kMmaWarp) {
    // ---- MMA issuers ----
    if (lane == 0) {
      bool ok = true;
      auto need = [&](uint64_t* bar, uint32_t parity) {
        if (phase_done(bar, parity)) return true;
        if (s_abort || !wait_one(bar, parity)) {
          give_up(kFaultMma);
          ok = false;
        }
        return ok;
      };
      auto scores = [&](int it, int seg) {
        const int s = it % kStages;
        if (!need(&full[s], (it / kStages) & 1)) return;
        // the tile's columns held the scores of tile it - 2 (and its weights)
        if (it >= 2 &&
            !need(kOwnWeights ? &pv_full[it & 1] : &o_done[it & 1], ((it >> 1) - 1) & 1))
          return;
        sm100::tc_fence_after();
        const uint64_t kd = key_desc<D>(sm100::smem_addr(smem + s * P::kStage));
        if constexpr (FEW > 0) {
          const uint64_t qd = key_desc<D>(
              sm100::smem_addr(smem + P::kQueries + (seg & 1) * 2 * P::kQueryPart));
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_f8(tmem + (it & 1) * kFewRows, kd + 2 * k, qd + part * (P::kQueryPart >> 4) + 2 * k,
                     kIdescFewS, part + k > 0);
        } else {
          const uint32_t d = tmem + (it & 1) * kTile;
          const uint32_t q = tmem + kColQ + (kOwnWeights ? 0 : (seg & 1) * (D / 2));
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)  // 32 codes: 32 bytes, 8 columns of queries
              mma_ts<true>(d, q + part * (D / 4) + 8 * k, kd + 2 * k, kIdescS, part + k > 0);
        }
        sm100::mma_commit(&s_full[it & 1]);
        sm100::mma_commit(&empty[s]);
      };
      auto values = [&](int it, bool first) {
        const int k2 = it & 1;
        if (!need(&pv_full[k2], (it >> 1) & 1)) return;
        sm100::tc_fence_after();
        const uint64_t vd =
            value_desc<FEW && D == 64>(
                sm100::smem_addr(smem + P::kDecoded + k2 * P::kHalfTile));
        if constexpr (FEW > 0) {
          const uint64_t wd =
              key_desc<128>(sm100::smem_addr(smem + P::kWeights + k2 * P::kWeightTile));
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)  // 16 tokens: 32 bytes of weights
            sm100::mma<false>(tmem + kColFewO, vd + k * 128,
                              wd + (k >> 2) * (P::kWeightTile / 2 >> 4) + 2 * (k & 3), kIdescFewO,
                              !first || k > 0);
        } else {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)  // 16 tokens: 8 columns of weights, 2048 bytes
            mma_ts<false>(tmem + kColO, tmem + (kOwnWeights ? kColP : k2 * kTile) + 8 * k,
                          vd + k * 128, kIdescO, !first || k > 0);
        }
        sm100::mma_commit(&o_done[k2]);
      };
      int it = 0, seg = 0;
      Segment g;
      const int rts = (a.T * a.G + kRows - 1) / kRows;
      long long u = u0;
      for (; ok && next_segment(u, g); ++seg) {
        if (warp == kMmaWarp && !need(&q_full[seg & 1], (seg >> 1) & 1)) break;
        if (g.t0 == 0 && warp > kMmaWarp) {
          // CTA j begins at unit floor(total j / ctas): inside the item while that is
          // below its end
          int n = 0;
          if (g.end < g.item_end)
            n = static_cast<int>((g.item_end * s_ctas + s_total - 1) / s_total) -
                static_cast<int>(blockIdx.x) - 1;
          a.item_ctas[(static_cast<size_t>(g.b) * a.Hkv + g.h) * rts + g.rt] =
              make_int2(static_cast<int>(blockIdx.x) + 1, n);
        }
        for (int j = 0; j < g.t1 - g.t0 && ok; ++j, ++it) {
          if (warp == kMmaWarp) scores(it, seg);
          else values(it, j == 0);
        }
      }
      // Given up: finish_kernel reads the entries of the items that are left all the same.
      while (!ok && warp > kMmaWarp && next_segment(u, g))
        if (g.t0 == 0)
          a.item_ctas[(static_cast<size_t>(g.b) * a.Hkv + g.h) * rts + g.rt] =
              make_int2(0, kLost);
      sm100::mma_commit(&s_end);
      if (!wait_one(&s_end, 0)) give_up(kFaultMma);
    }
  } else if (warp >= kFirstProducer) {
    // ---- producers: tiles of the cache, alternating ----
    const int pr = warp - kFirstProducer;
    const int unit = min(a.page, kTile);  // tokens per TMA copy
    const int per = kTile / unit;         // copies per tile (and of keys and values each)
    int it = 0;                           // tiles of this CTA so far, over all segments
    int mine = -1;                        // this warp's last tile
    bool ok = true;
    Segment g;
    for (long long u = u0; ok && next_segment(u, g);) {
      const int n = g.t1 - g.t0;
      // 32 / per of this warp's tiles at a time: page ids and scales of all their
      // copies in one round of loads, a copy per lane
      const int batch = 32 / per;
      const int skip = (pr - it % kProducers + kProducers) % kProducers;  // first own tile
      for (int j0 = skip; j0 < n && ok; j0 += batch * kProducers) {
        const int j = j0 + lane / per * kProducers;
        const int pos = (g.t0 + j) * kTile + lane % per * unit;
        const bool wanted = j < n && pos < g.s.len;
        int id = -1;
        if (wanted) id = a.table[static_cast<size_t>(g.b) * a.width + pos / a.page];
        const bool have = wanted && id >= 0 && id < a.num_pages;
        const size_t at = static_cast<size_t>(have ? id : 0) * a.Hkv + g.h;
        // a page id outside the pool makes the sequence's rows NaN
        const float ks = have ? a.k_scale[at] : wanted ? __uint_as_float(0x7FC00000u) : 0.f;
        const float vs = have ? a.v_scale[at] : 1.f;
        const float vc = fminf(fmaxf(vs, 8.67361738e-19f), 1.15292150e18f);  // 2^-60 .. 2^60
        const float4 sc = make_float4(ks, vs != vs ? vs : log2f(vc), 1.f / vc, 0.f);
        const int row = static_cast<int>(at) * a.page + pos % a.page;
        for (int k = 0; k < batch && j0 + k * kProducers < n; ++k) {
          const int i = it + j0 + k * kProducers;
          const int s = i % kStages;
          if (i >= kStages && !wait(&empty[s], ((i / kStages) - 1) & 1)) give_up(kFaultProducer);
          if (__any_sync(0xFFFFFFFFu, s_abort)) {
            ok = false;
            break;
          }
          const bool turn = lane / per == k;
          if (turn) {
            const int first = lane % per * (unit / 16);
            for (int e = 0; e < unit / 16; ++e) s_scale[s * (kTile / 16) + first + e] = sc;
          }
          const int copies = __popc(__ballot_sync(0xFFFFFFFFu, turn && have));
          __syncwarp();
          if (lane == 0)
            sm100::mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * copies * unit * D));
          __syncwarp();
          if (turn && have) {
            uint8_t* dst = smem + s * P::kStage + lane % per * unit * D;
            sm100::tma_load_2d(dst, &map_k, &full[s], 0, row);
            sm100::tma_load_2d(dst + kTile * D, &map_v, &full[s], 0, row);
          }
          mine = i;
        }
      }
      it += n;
    }
    // No copy may still be landing when the CTA exits: wait for this warp's
    // among the last kStages tiles (their readers have done so too, unless they
    // have given up).
    for (int i = max((ok ? it : mine + 1) - kStages, 0); i <= mine; ++i)
      if (i % kProducers == pr) wait(&full[i % kStages], (i / kStages) & 1);
  } else if (warp >= kFirstDecode) {
    // ---- queries of a segment to e4m3 parts, codes of a tile's values to halves ----
    const int tid = threadIdx.x - 32 * kFirstDecode;
    const uint32_t lanes = static_cast<uint32_t>(tid & 96) << 16;
    // (the first four warps) The queries of segment `seg`, in columns that an earlier
    // segment's have left.
    auto stage_queries = [&](const Segment& g, int seg) {
      if (tid >= 128) return;
      if constexpr (FEW > 0) {
        // eight threads to a row, D / 8 elements each, to the codes' layout of keys
        constexpr int kW = D / 64;  // 16-byte pieces
        const int r = tid >> 3, part = tid & 7;
        const bool valid = r < g.s.nn * a.G;
        const int t = valid ? r / a.G : 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((static_cast<size_t>(g.b) * a.T + t) * a.Hq + g.h * a.G + (r - t * a.G)) * D +
            part * (D / 8));
        uint4 w[kW];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kW; ++k) {
          w[k] = valid ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
          top = __vmaxu2(__vmaxu2(top, w[k].x & 0x7FFF7FFFu),
                         __vmaxu2(w[k].y & 0x7FFF7FFFu,
                                  __vmaxu2(w[k].z & 0x7FFF7FFFu, w[k].w & 0x7FFF7FFFu)));
        }
        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int sh = query_shift(top);
        const float f = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
        if (part == 0) s_factor[(seg & 1) * kRows + r] = query_factor(a.scale, top, sh);
        uint8_t* dst = smem + P::kQueries + (seg & 1) * 2 * P::kQueryPart + r * D;
#pragma unroll
        for (int k = 0; k < kW; ++k) {  // 8 codes of each part
          const uint32_t x4[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
          uint32_t h2[4], l2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) split_e4m3(x4[j], f, h2[j], l2[j]);
          const int at = part * (D / 8) + 8 * k;  // byte of the row, 16-byte chunks swizzled
          const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
          uint8_t* p = dst + ((((at >> 4) ^ sw) << 4) | (at & 15));
          *reinterpret_cast<uint2*>(p) = make_uint2(h2[0] | (h2[1] << 16), h2[2] | (h2[3] << 16));
          *reinterpret_cast<uint2*>(p + P::kQueryPart) =
              make_uint2(l2[0] | (l2[1] << 16), l2[2] | (l2[3] << 16));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && seg < a.query_segments) sm100::mbar_arrive(&q_full[seg & 1]);
        return;
      }
      // q 2^sh = hi + lo, its largest magnitude in [128, 256)
      const int r = g.rt * kRows + row_of_lane<COPIES>(tid);
      const bool valid = r < g.s.nn * a.G;
      const int t = valid ? r / a.G : 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<size_t>(g.b) * a.T + t) * a.Hq + g.h * a.G + (r - t * a.G)) * D);
      // 16-byte pieces at a time: the whole row where the registers hold it (with one
      // copy they are 80), else a part, read again for the conversion
      constexpr int kAll = D / 8, kPart = COPIES == 1 ? 8 : kAll;
      uint4 w[kPart];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kPart; ++k)
          w[k] = valid ? __ldg(src + k0 + k) : make_uint4(0u, 0u, 0u, 0u);
      };
      uint32_t top = 0;
#pragma unroll 1
      for (int k0 = 0; k0 < kAll; k0 += kPart) {
        load(k0);
#pragma unroll
        for (int k = 0; k < kPart; ++k)
          top = __vmaxu2(__vmaxu2(top, w[k].x & 0x7FFF7FFFu),
                         __vmaxu2(w[k].y & 0x7FFF7FFFu,
                                  __vmaxu2(w[k].z & 0x7FFF7FFFu, w[k].w & 0x7FFF7FFFu)));
      }
      top = max(top & 0xFFFFu, top >> 16);
      const int sh = query_shift(top);
      const float f = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
      s_factor[(seg & 1) * kRows + tid] = query_factor(a.scale, top, sh);
      const uint32_t dst = tmem + lanes + kColQ + (kOwnWeights ? 0 : (seg & 1) * (D / 2));
#pragma unroll 1
      for (int k0 = 0; k0 < kAll; k0 += kPart) {
        if (kPart < kAll) load(k0);
#pragma unroll
        for (int k = 0; k < kPart; k += 4) {  // 32 elements: 8 columns of each part
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x4[4] = {w[k + e].x, w[k + e].y, w[k + e].z, w[k + e].w};
            uint32_t h2[4], l2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split_e4m3(x4[j], f, h2[j], l2[j]);
            hi[2 * e] = h2[0] | (h2[1] << 16);
            hi[2 * e + 1] = h2[2] | (h2[3] << 16);
            lo[2 * e] = l2[0] | (l2[1] << 16);
            lo[2 * e + 1] = l2[2] | (l2[3] << 16);
          }
          tmem_st<8>(dst + 2 * (k0 + k), hi);
          tmem_st<8>(dst + D / 4 + 2 * (k0 + k), lo);
        }
      }
      sm100::tmem_st_wait();
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0 && seg < a.query_segments) sm100::mbar_arrive(&q_full[seg & 1]);
    };
    int it = 0, seg = 0;
    bool ok = true;
    Segment g, next;
    long long u = u0;
    bool more = next_segment(u, next);
    if (more) stage_queries(next, 0);
    for (; ok && more; ++seg) {
      g = next;
      more = next_segment(u, next);
      const int before = it - 1;  // last tile of the segment before
      for (int ti = g.t0; ti < g.t1; ++ti, ++it) {
        const int s = it % kStages, k2 = it & 1;
        if (!wait(&full[s], (it / kStages) & 1) ||
            (it >= 2 && !wait(&o_done[k2], ((it >> 1) - 1) & 1))) {
          give_up(kFaultSoftmax);
          ok = false;
          break;
        }
        const uint8_t* src = smem + s * P::kStage + kTile * D;
        uint8_t* dst = smem + P::kDecoded + k2 * P::kHalfTile;
        const int left = g.s.len - ti * kTile;
        constexpr int kPieces = D / 16;  // 16-byte pieces of a token
        const int ch = tid % kPieces;
#pragma unroll
        for (int st = 0; st < kTile * kPieces / (32 * DECODERS); ++st) {
          const int t = tid / kPieces + st * (32 * DECODERS / kPieces);
          const int sw = D == 128 ? (t & 7) : ((t >> 1) & 3);
          uint4 w = *reinterpret_cast<const uint4*>(src + t * D + ((ch ^ sw) << 4));
          // slots behind the sequence may hold anything, NaN too
          if (t >= left) w = make_uint4(0u, 0u, 0u, 0u);
          const uint4 x = make_uint4(halves(w.x & 0xFFFFu), halves(w.x >> 16),
                                     halves(w.y & 0xFFFFu), halves(w.y >> 16));
          const uint4 y = make_uint4(halves(w.z & 0xFFFFu), halves(w.z >> 16),
                                     halves(w.w & 0xFFFFu), halves(w.w >> 16));
          // columns 16 ch.. : chunks 2 (ch % 4), + 1 of the token's row in its half
          uint8_t* row = dst + (ch >> 2) * (kTile * 128) + t * 128;
          const int c0 = (ch & 3) * 2, r = t & 7;
          const int flip = (ch >> 2) & 1;  // lanes of the two halves write different banks
          *reinterpret_cast<uint4*>(row + (((c0 + flip) ^ r) << 4)) = flip ? y : x;
          *reinterpret_cast<uint4*>(row + (((c0 + 1 - flip) ^ r) << 4)) = flip ? x : y;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          sm100::mbar_arrive(&pv_full[k2]);
          sm100::mbar_arrive(&empty[s]);
        }
        if (more && tid < 128 && ti == (kLateQueries ? g.t1 - 1 : min(g.t0 + 1, g.t1 - 1))) {
          // The next segment's queries, once those of the segment before, whose factors
          // and barrier they take, have been used by all: its last weighted values are
          // done. (From a segment's second tile on that has been waited for above; asked
          // again now, this tile's own could have ended a phase later.) Late queries
          // also take the columns of this segment's, which its last scores release; that
          // alone says nothing of the softmax warps, which after a segment of one tile may
          // still be at the sums of the one before it.
          if ((ti == g.t0 && before >= 0 && !wait(&o_done[before & 1], (before >> 1) & 1)) ||
              (kLateQueries && !wait(&s_full[k2], (it >> 1) & 1))) {
            give_up(kFaultSoftmax);
            ok = false;
            break;
          }
          // the products that read the columns come before the stores that replace them
          sm100::tc_fence_after();
          stage_queries(next, seg + 1);
        }
      }
    }
  } else if constexpr (FEW > 0) {
    // ---- softmax of few rows: a token per thread, its weights for R of the rows ----
    constexpr int R = FEW / PARTS;
    static_assert(FEW % PARTS == 0 && R % 4 == 0, "rows of a part");
    const int quarter = warp & 3, part = warp >> 2;
    const int tok = quarter * 32 + lane;  // token of a tile, and TMEM lane
    const uint32_t cols = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * R;
    int it = 0, seg = 0;
    bool ok = true;  // false: go on without waiting, the results are abandoned
    auto need = [&](uint64_t* bar, uint32_t parity) {
      if (!phase_done(bar, parity) && ok && !wait_one(bar, parity)) {
        atomicOr(&g_attn_fault, kFaultSoftmax);
        s_abort = 1;
        ok = false;
      }
      __syncwarp();
    };
    // the part's warps, one per quarter, share the rows: they meet
    auto part_meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(part + 1) : "memory"); };
    float* const tops = s_top + part * R;  // [quarter][kFewRows]
    // this warp's own copy of the rows' refs
    float4* const refs =
        reinterpret_cast<float4*>(smem + P::kRefs) + (quarter * kFewRows + part * R) / 4;
    // weights of a tile: [half of the tokens][row][64 tokens], 16-byte chunks swizzled
    uint8_t* const wrow = smem + P::kWeights + (tok >> 6) * (P::kWeightTile / 2) + (tok & 7) * 2 +
                          part * R * 128;
    const int chunk = (tok & 63) >> 3;
    Segment g;
    for (long long u = u0; next_segment(u, g); ++seg) {
      need(&q_full[seg & 1], (seg >> 1) & 1);
      const float4* qf = reinterpret_cast<const float4*>(s_factor + (seg & 1) * kRows + part * R);
      float l[R];
#pragma unroll
      for (int n = 0; n < R; ++n) l[n] = 0.f;
      for (int ti = g.t0; ti < g.t1; ++ti, ++it) {
        const int s = it % kStages, k2 = it & 1;
        need(&full[s], (it / kStages) & 1);  // the scales
        const float4 x = s_scale[s * (kTile / 16) + tok / 16];
        const bool in = ti * kTile + tok < g.s.len;
        need(&s_full[k2], (it >> 1) & 1);
        sm100::tc_fence_after();
        uint32_t v[R];
        tmem_ld_cols<R>(cols + k2 * kFewRows, v);
        sm100::tmem_ld_wait();
        float t[R], top = -INFINITY;
#pragma unroll
        for (int n = 0; n < R; n += 4) {
          const float4 f = qf[n / 4], ref = refs[n / 4];
          t[n] = in ? fmaf(__uint_as_float(v[n]), f.x * x.x, x.y) : -INFINITY;
          t[n + 1] = in ? fmaf(__uint_as_float(v[n + 1]), f.y * x.x, x.y) : -INFINITY;
          t[n + 2] = in ? fmaf(__uint_as_float(v[n + 2]), f.z * x.x, x.y) : -INFINITY;
          t[n + 3] = in ? fmaf(__uint_as_float(v[n + 3]), f.w * x.x, x.y) : -INFINITY;
          top = fmaxf(top, fmaxf(fmaxf(t[n] - ref.x, t[n + 1] - ref.y),
                                 fmaxf(t[n + 2] - ref.z, t[n + 3] - ref.w)));
        }
        bool move = ti == g.t0;  // the first tile sets the refs
        if (!move) {
          // they move when any token asks for it (the flags alternate with the tiles, so
          // a meeting later they may be rewritten)
          const bool ask = __any_sync(0xFFFFFFFFu, top > kTop);
          if (lane == 0) s_flag[(k2 * 4 + part) * 4 + quarter] = ask;
          part_meet();
#pragma unroll
          for (int k = 0; k < 4; ++k) move |= s_flag[(k2 * 4 + part) * 4 + k] != 0;
        }
        if (move) {
#pragma unroll
          for (int n = 0; n < R; ++n) {
            float mx = fmaxf(t[n], kLowest);
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            if (lane == 0) tops[quarter * kFewRows + n] = mx;
          }
          // (read before the next write: a tile's flags or a segment's end lie between)
          part_meet();
          // o holds the tiles before this one once the last of them has been added
          if (ti > g.t0) need(&o_done[k2 ^ 1], ((it - 1) >> 1) & 1);
          sm100::tc_fence_after();
#pragma unroll
          for (int n = 0; n < R; n += 4) {
            float mx[4], al[4];
            const float4 old4 = refs[n / 4];
            const float old[4] = {old4.x, old4.y, old4.z, old4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              mx[e] = tops[n + e];
#pragma unroll
              for (int k = 1; k < 4; ++k) mx[e] = fmaxf(mx[e], tops[k * kFewRows + n + e]);
              mx[e] = ti == g.t0 || mx[e] > old[e] + kTop ? mx[e] - kHead : old[e];
              al[e] = uno::ex2(old[e] - mx[e]);
            }
            if (ti > g.t0) {
              tmem_ld_cols<4>(cols + kColFewO + n, v);
              sm100::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                l[n + e] *= al[e];
                v[e] = __float_as_uint(__uint_as_float(v[e]) * al[e]);
              }
              tmem_st_cols<4>(cols + kColFewO + n, v);
            }
            __syncwarp();
            if (lane == 0) refs[n / 4] = make_float4(mx[0], mx[1], mx[2], mx[3]);
          }
          sm100::tmem_st_wait();
          __syncwarp();
        }
        if (it >= 2) need(&o_done[k2], ((it >> 1) - 1) & 1);  // the weights of tile it - 2
#pragma unroll
        for (int n = 0; n < R; n += 4) {
          const float4 ref = refs[n / 4];
          const float w[4] = {uno::ex2(t[n] - ref.x), uno::ex2(t[n + 1] - ref.y),
                              uno::ex2(t[n + 2] - ref.z), uno::ex2(t[n + 3] - ref.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[n + e] = fmaf(w[e], x.z, l[n + e]);
            *reinterpret_cast<__half*>(wrow + k2 * P::kWeightTile + (n + e) * 128 +
                                       ((chunk ^ ((part * R + n + e) & 7)) << 4)) =
                __float2half_rn(w[e]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          sm100::mbar_arrive(&pv_full[k2]);
          sm100::mbar_arrive(&empty[s]);
        }
      }
      // ---- the segment's sums: NaN once a wait has run out (where a segment is not complete
      // the one for its last tile does) ----
      const int last = it - 1, rows = min(max(g.s.nn * a.G - part * R, 0), R);  // of this part
      need(&o_done[last & 1], (last >> 1) & 1);
      sm100::tc_fence_after();
      uint32_t v[R];
      tmem_ld_cols<R>(cols + kColFewO, v);
      sm100::tmem_ld_wait();
      const size_t row0 = (g.t0 == 0 ? (static_cast<size_t>(g.b) * a.Hkv + g.h) *
                                           (static_cast<size_t>(a.T) * a.G)
                                     : static_cast<size_t>(blockIdx.x) * kRows) +
                          part * R;
      float* dst = (g.t0 == 0 ? a.item_o : a.cta_o) + row0 * D + tok;
#pragma unroll
      for (int n = 0; n < R; ++n) {
#pragma unroll
        for (int o = 16; o; o >>= 1) l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], o);
        if (lane == 0) tops[quarter * kFewRows + n] = l[n];
        if (n < rows && tok < D) dst[n * D] = __uint_as_float(v[n]);
      }
      part_meet();
      if (tok < rows) {  // (the first quarter's lanes)
        float sum = tops[tok];
#pragma unroll
        for (int k = 1; k < 4; ++k) sum += tops[k * kFewRows + tok];
        (g.t0 == 0 ? a.item_ml : a.cta_ml)[row0 + tok] =
            make_float2(reinterpret_cast<float*>(refs)[tok], s_abort ? quiet_nan() : sum);
      }
      part_meet();  // read before the next segment writes
      sm100::tc_fence_before();  // o may be written again
    }
  } else {
    // ---- softmax: a part of a row's tokens per thread ----
    const int quarter = warp & 3, part = warp >> 2;
    const int tl = quarter * 32 + lane;  // TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_row = row_of_lane<COPIES>(tl);
    const int copy = COPIES == 4 ? quarter : COPIES == 2 ? quarter >> 1 : 0;
    const int c0 = copy * CW + part * HC;  // this thread's tokens of a tile
    constexpr int CH = 16;  // of which it loads so many at once
    int it = 0, seg = 0;
    bool ok = true;  // false: go on without waiting, the results are abandoned
    // (each lane for itself, and mostly for a phase that is over: a vote as in wait()
    // costs as much as the test)
    auto need = [&](uint64_t* bar, uint32_t parity) {
      if (!phase_done(bar, parity) && ok && !wait_one(bar, parity)) {
        atomicOr(&g_attn_fault, kFaultSoftmax);
        s_abort = 1;
        ok = false;
      }
      __syncwarp();
    };
    Segment g;
    if constexpr (kOwnWeights) {
      // the other copies' tokens have weight 0, in every tile
#pragma unroll
      for (int k = 0; k < kTile / 32; ++k) {
        const uint32_t z[16] = {};
        tmem_st<16>(tmem + lanes + kColP + 16 * k, z);
      }
      sm100::tmem_st_wait();
    }
    for (long long u = u0; next_segment(u, g); ++seg) {
      const int r = g.rt * kRows + my_row;  // row of the sequence and KV head
      const bool valid = r < g.s.nn * a.G;
      const bool live = __any_sync(0xFFFFFFFFu, valid);
      need(&q_full[seg & 1], (seg >> 1) & 1);
      const float qf = s_factor[(seg & 1) * kRows + tl];
      float ref = kLowest, l = 0.f;
      for (int ti = g.t0; ti < g.t1; ++ti, ++it) {
        const int s = it % kStages, k2 = it & 1;
        need(&full[s], (it / kStages) & 1);  // the scales
        need(&s_full[k2], (it >> 1) & 1);
        sm100::tc_fence_after();
        const uint32_t st = tmem + lanes + k2 * kTile;
        if (live) {
          const int left = g.s.len - ti * kTile - c0;  // of this thread's tokens, those that exist
          const float4* sc = s_scale + s * (kTile / 16) + c0 / 16;
          uint32_t pk[HC / 2];  // weights, two to a column
          float add, top;
          // weights against the current ref; top: the largest t - ref
          auto pass = [&](auto whole) {  // whole: all of the thread's tokens exist
            add = 0.f;
            top = -INFINITY;
            uint32_t v[2][CH];  // a chunk ahead
            tmem_ld<CH>(st + c0, v[0]);
#pragma unroll
            for (int k = 0; k < HC / CH; ++k) {
              sm100::tmem_ld_wait();
              if (k + 1 < HC / CH) tmem_ld<CH>(st + c0 + (k + 1) * CH, v[(k + 1) & 1]);
              const float4 x = sc[k];
              const float f = qf * x.x, off = x.y - ref;
              const uint64_t ff = uno::pack2(f, f), offs = uno::pack2(off, off);
              uint64_t sums = uno::pack2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < CH; e += 2) {
                const int i = k * CH + e;
                const float2 tt = uno::unpack2(uno::fma2(
                    uno::pack2(__uint_as_float(v[k & 1][e]), __uint_as_float(v[k & 1][e + 1])), ff,
                    offs));
                float t0 = tt.x, t1 = tt.y;
                if constexpr (!decltype(whole)::value) {
                  if (i >= left) t0 = -INFINITY;
                  if (i + 1 >= left) t1 = -INFINITY;
                }
                asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(t0), "f"(t1));
                t0 = uno::ex2(t0);
                t1 = uno::ex2(t1);
                sums = uno::add2(sums, uno::pack2(t0, t1));
                pk[i / 2] = pack_f16(t0, t1);
              }
              const float2 sum = uno::unpack2(sums);
              add = fmaf(sum.x + sum.y, x.z, add);
            }
          };
          // A ref moves when any part of a row of the quarter asks for it (the
          // flags alternate with the tiles, so a meeting later they may be rewritten).
          bool move = ti == g.t0;  // the first tile sets it
          for (;;) {
            if (move) {
              // to the tile's largest t, in rows where that is far above it
              float mx = kLowest;
#pragma unroll 1
              for (int k = 0; k < HC / CH; ++k) {
                uint32_t v[CH];
                tmem_ld<CH>(st + c0 + k * CH, v);
                sm100::tmem_ld_wait();
                const float4 x = sc[k];
                const float f = qf * x.x;
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                  const float t = fmaf(__uint_as_float(v[e]), f, x.y);
                  if (k * CH + e < left) mx = fmaxf(mx, t);
                }
              }
              if constexpr (PARTS > 1) {
                s_top[part * kRows + tl] = mx;
                meet<PARTS>(quarter);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) mx = fmaxf(mx, s_top[k * kRows + tl]);
                meet<PARTS>(quarter);  // read before a next move writes
              }
              if (ti == g.t0) {
                ref = mx - kHead;
              } else {
                const float to = mx > ref + kTop ? mx - kHead : ref;
                const float al = uno::ex2(ref - to);
                ref = to;
                l *= al;
                // o holds the tiles before this one once the last of them has been added;
                // each part rescales its share of the columns
                need(&o_done[k2 ^ 1], ((it - 1) >> 1) & 1);
                sm100::tc_fence_after();
#pragma unroll 1
                for (int c = part * (D / PARTS); c < (part + 1) * (D / PARTS); c += 16) {
                  uint32_t v[16];
                  tmem_ld<16>(tmem + lanes + kColO + c, v);
                  sm100::tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
                  tmem_st<16>(tmem + lanes + kColO + c, v);
                }
              }
            }
            if (left >= HC) pass(std::true_type{});
            else pass(std::false_type{});
            const bool ask = !move && __any_sync(0xFFFFFFFFu, top > kTop);
            if (PARTS > 1 && lane == 0) s_flag[(k2 * 4 + quarter) * 4 + part] = ask;
            meet<PARTS>(quarter);  // all parts have read the scores that the weights overwrite
            if (move) break;
            if constexpr (PARTS > 1) {
#pragma unroll
              for (int k = 0; k < PARTS; ++k) move |= s_flag[(k2 * 4 + quarter) * 4 + k] != 0;
            } else {
              move = ask;
            }
            if (!move) break;
          }
          l += add;
          if constexpr (kOwnWeights) {
            // tile it - 1's weights have been used
            if (it > 0) need(&o_done[k2 ^ 1], ((it - 1) >> 1) & 1);
            sm100::tc_fence_after();
            tmem_st<HC / 2>(tmem + lanes + kColP + c0 / 2, pk);
          } else {
            tmem_st<HC / 2>(st + c0 / 2, pk);
          }
          sm100::tmem_st_wait();
        }
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          sm100::mbar_arrive(&pv_full[k2]);
          sm100::mbar_arrive(&empty[s]);
        }
      }
      // ---- the segment's sums: NaN once a wait has run out (where a segment is not complete
      // the one for its last tile does) ----
      const int last = it - 1;
      need(&o_done[last & 1], (last >> 1) & 1);
      sm100::tc_fence_after();
      if (live) {
        const size_t row =
            g.t0 == 0 ? ((static_cast<size_t>(g.b) * a.Hkv + g.h) * COPIES + copy) *
                                (static_cast<size_t>(a.T) * a.G) + r
                      : static_cast<size_t>(blockIdx.x) * kRows + tl;
        float* dst = (g.t0 == 0 ? a.item_o : a.cta_o) + row * D;
        if constexpr (PARTS > 1) {
          s_top[part * kRows + tl] = l;
          meet<PARTS>(quarter);
        }
        if (part == 0 && valid) {
#pragma unroll
          for (int k = 1; k < PARTS; ++k) l += s_top[k * kRows + tl];
          (g.t0 == 0 ? a.item_ml : a.cta_ml)[row] = make_float2(ref, s_abort ? quiet_nan() : l);
        }
        meet<PARTS>(quarter);
#pragma unroll 1
        for (int c = part * (D / PARTS); c < (part + 1) * (D / PARTS); c += 16) {
          uint32_t v[16];
          tmem_ld<16>(tmem + lanes + kColO + c, v);
          sm100::tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      }
      sm100::tc_fence_before();  // o may be written again
    }
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, kTmemCols);
  }
}

// New tokens, and the join with the cached tokens' partial sums. 16 query rows
// of a sequence and KV head per group of KW warps: the groups of 16 new tokens and
// the partial sums are dealt to the warps, whose sums meet in shared memory.
//
// mma.sync m16n8k16 (bfloat16, weights rounded to bfloat16, 2^-9). A
// contraction's index needs no particular order, so it is permuted until a
// lane's share is contiguous: lane (g, c) (g = lane / 4, c = lane % 4) reads keys'
// elements [c D/4, (c + 1) D/4) of token g, and of values the D/8 elements from
// g D/8 of the four tokens whose weights it holds from the score fragment.
template <int D, int KW>
__global__ void __launch_bounds__(128, 2) finish_kernel(const AttnArgs a) {
  constexpr int KS = D / 16;  // k-steps of a score
  constexpr int DN = D / 8;   // output column tiles
  constexpr int kGroups = 4 / KW;
  __shared__ float4 s_sum[KW > 1 ? KW - 1 : 1][KW > 1 ? DN + 1 : 1][32];
  __shared__ int16_t s_parent[kGroups][kMaxT];  // of the item's sequence
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kw = warp % KW;
  const int g = lane >> 2, c = lane & 3;
  const int rgs = (a.T * a.G + 15) / 16;  // groups of 16 rows
  const long long item = static_cast<long long>(blockIdx.x) * kGroups + warp / KW;
  const long long items = static_cast<long long>(a.B) * a.Hkv * rgs;
  uno::launch_dependents();
  // Every thread waits for cached_kernel before it leaves: the next launch takes
  // this one's end for cached_kernel's. (Whole warps leave; with KW > 1 whole CTAs.)
  if (item >= items) {
    uno::grid_dependency_wait();
    return;
  }
  const int rg = static_cast<int>(item % rgs);
  const int h = static_cast<int>(item / rgs % a.Hkv);
  const int b = static_cast<int>(item / rgs / a.Hkv);
  const Seq sq = seq_of(a, b);
  const int R = sq.nn * a.G;  // rows of the sequence and head
  const int r0 = rg * 16;
  if (r0 >= R) {
    uno::grid_dependency_wait();
    return;
  }
  const int rows[2] = {r0 + g, r0 + g + 8};
  // query row r: token r / G, head h G + r % G (rows past the end repeat the last
  // one, unstored)
  auto token = [&](int i) { return min(rows[i], R - 1) / a.G; };
  auto q_at = [&](int i) {
    const int r = min(rows[i], R - 1), t = r / a.G;
    return ((static_cast<size_t>(b) * a.T + t) * a.Hq + h * a.G + (r - t * a.G)) * D;
  };
  auto load_q = [&](int i, uint32_t* w) {
    const uint4* p = reinterpret_cast<const uint4*>(a.q + q_at(i) + c * (D / 4));
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 v = __ldg(p + k);
      w[4 * k] = v.x;
      w[4 * k + 1] = v.y;
      w[4 * k + 2] = v.z;
      w[4 * k + 3] = v.w;
    }
  };
  uint32_t qa[KS][4];
  float o[DN][4];
#pragma unroll
  for (int i = 0; i < DN; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  // New reference for t[0..1][..]: weights in place, o and l rescaled.
  auto rescale = [&](float (*t)[4]) {
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mx[0] = fmaxf(mx[0], fmaxf(t[j][0], t[j][1]));
      mx[1] = fmaxf(mx[1], fmaxf(t[j][2], t[j][3]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
    }
    if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] || mx[1] > m[1])) {
      float al[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        al[i] = m[i] == -INFINITY ? 0.f : uno::ex2(m[i] - mx[i]);
        l[i] *= al[i];
        m[i] = mx[i];
      }
#pragma unroll
      for (int j = 0; j < DN; ++j) {
        o[j][0] *= al[0];
        o[j][1] *= al[0];
        o[j][2] *= al[1];
        o[j][3] *= al[1];
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[j][e] = uno::ex2(t[j][e] - ref[e >> 1]);
  };

  // ---- new tokens: groups of 16, from the last one any row sees down ----
  {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[D / 8];
      load_q(i, w);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qa[k][i] = w[2 * k];
        qa[k][i + 2] = w[2 * k + 1];
      }
    }
    const float f = a.scale * kLog2e;
    const bool tree = a.parent != nullptr;
    int16_t* par = s_parent[KW > 1 ? 0 : warp];
    if (tree) {
      // up to the last of these rows' tokens; parents come before their children, any
      // other value ends the chain
      const int32_t* src = a.parent + static_cast<size_t>(b) * a.T;
      const int n = min(r0 + 15, R - 1) / a.G + 1;
      for (int t = KW > 1 ? threadIdx.x : lane; t < n; t += 32 * KW) {
        const int up = __ldg(src + t);
        par[t] = static_cast<int16_t>(up < t ? max(up, -1) : -1);
      }
      if (KW > 1) __syncthreads();
      else __syncwarp();
    }
    const int tok[2] = {token(0), token(1)};
    int cur[2] = {tok[0], tok[1]};  // the next ancestor to mark (trees)
    const int last = min(r0 + 15, R - 1) / a.G;
    for (int gi = last / 16; gi >= 0; --gi) {
      // rows see columns (bits) of this group
      uint32_t see[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (tree) {
          see[i] = 0u;
          while (cur[i] >= gi * 16) {
            see[i] |= 1u << (cur[i] - gi * 16);
            cur[i] = par[cur[i]];
          }
        } else {
          const int n = tok[i] - gi * 16 + 1;
          see[i] = n >= 16 ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
        }
      }
      if (gi % KW != kw) continue;
      // the group's keys and values in one round of loads
      uint4 kv[2][D / 32], vv[4][D / 64];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int col = min(gi * 16 + n * 8 + g, last);
        const uint4* p = reinterpret_cast<const uint4*>(
            a.k_new + ((static_cast<size_t>(b) * a.T + col) * a.Hkv + h) * D + c * (D / 4));
#pragma unroll
        for (int k = 0; k < D / 32; ++k) kv[n][k] = __ldg(p + k);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tk = min(gi * 16 + 2 * c + (e & 1) + (e >> 1) * 8, last);
        const uint4* p = reinterpret_cast<const uint4*>(
            a.v_new + ((static_cast<size_t>(b) * a.T + tk) * a.Hkv + h) * D + g * (D / 8));
#pragma unroll
        for (int k = 0; k < D / 64; ++k) vv[e][k] = __ldg(p + k);
      }
      float t[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          mma_bf16(t[n], qa[2 * k], kv[n][k].x, kv[n][k].y);
          mma_bf16(t[n], qa[2 * k + 1], kv[n][k].z, kv[n][k].w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          t[n][e] = (see[e >> 1] >> (n * 8 + 2 * c + (e & 1))) & 1u ? t[n][e] * f : -INFINITY;
      }
      rescale(t);
      l[0] += (t[0][0] + t[0][1]) + (t[1][0] + t[1][1]);
      l[1] += (t[0][2] + t[0][3]) + (t[1][2] + t[1][3]);
      uint32_t pa[4] = {pack_bf16(t[0][0], t[0][1]), pack_bf16(t[0][2], t[0][3]),
                        pack_bf16(t[1][0], t[1][1]), pack_bf16(t[1][2], t[1][3])};
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {  // eight of a lane's columns at a time
        uint32_t w[4][4];
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 v = vv[e][k];
          w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
          odd |= nonfinite2(v.x) || nonfinite2(v.y) || nonfinite2(v.z) || nonfinite2(v.w);
        }
        if (__any_sync(0xFFFFFFFFu, odd)) {
          // An infinity or NaN among the values: rows that do not see its token
          // must not meet it (0 times infinity), so these columns go row by row.
          for (int tk = 0; tk < 16; ++tk) {
            float pr[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = tk & 1 ? t[0][2 * i + 1] : t[0][2 * i];
              const float y = tk & 1 ? t[1][2 * i + 1] : t[1][2 * i];
              pr[i] = __shfl_sync(0xFFFFFFFFu, tk < 8 ? x : y, (lane & 28) | ((tk & 7) >> 1));
            }
            if (gi * 16 + tk > last) continue;
            const uint16_t* p =
                a.v_new + ((static_cast<size_t>(b) * a.T + gi * 16 + tk) * a.Hkv + h) * D;
#pragma unroll
            for (int j = 8 * k; j < 8 * k + 8; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((see[e >> 1] >> tk) & 1u)
                  o[j][e] = fmaf(pr[e >> 1],
                                 uno::bf16_bits_to_float(p[(2 * c + (e & 1)) * DN + j]),
                                 o[j][e]);
          }
          continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = 8 * k + 2 * q;
          mma_bf16(o[j], pa, __byte_perm(w[0][q], w[1][q], 0x5410),
                   __byte_perm(w[2][q], w[3][q], 0x5410));
          mma_bf16(o[j + 1], pa, __byte_perm(w[0][q], w[1][q], 0x7632),
                   __byte_perm(w[2][q], w[3][q], 0x7632));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
  }

  // ---- partial sums over the cached tokens ----
  uno::grid_dependency_wait();
  bool lost = false;  // the cached tokens' sums: the rows come out as NaN
  if (sq.tiles > 0) {
    const int rt = r0 / kRows;
    // kLost, or anything else that is no range of CTAs: no other part is read
    int2 more = a.item_ctas[(static_cast<size_t>(b) * a.Hkv + h) *
                                ((a.T * a.G + kRows - 1) / kRows) + rt];
    lost = more.x < 1 || more.x > kMaxCtas || more.y < 0 || more.y > kMaxCtas - more.x;
    if (lost) more = make_int2(0, 0);
    const int lanes_per_copy = kRows / a.copies;
    // adds the partial sums at rows at0 + r (r of this lane's rows) of ml and po
    auto add = [&](const float2* ml, const float* po, size_t at0, int r_off) {
      float f1[2], f2[2];
      const float4* src[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t at = at0 + min(rows[i], R - 1) - r_off;
        const float2 v = ml[at];
        src[i] = reinterpret_cast<const float4*>(po + at * D + c * (D / 4));
        const float mx = fmaxf(m[i], v.x);
        f1[i] = m[i] == -INFINITY ? 0.f : uno::ex2(m[i] - mx);
        f2[i] = uno::ex2(v.x - mx);
        // a side without a finite maximum still carries its NaN
        l[i] = (l[i] != l[i] ? l[i] : l[i] * f1[i]) + (v.y != v.y ? v.y : v.y * f2[i]);
        m[i] = mx;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)  // columns DN (2 c + q)..
#pragma unroll
          for (int e = 0; e < DN / 4; ++e) {
            const float4 v = src[i][q * (DN / 4) + e];
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              o[4 * e + x][2 * i + q] = fmaf(w[x], f2[i], o[4 * e + x][2 * i + q] * f1[i]);
          }
    };
    for (int cp = kw; cp < a.copies; cp += KW)
      add(a.item_ml, a.item_o,
          ((static_cast<size_t>(b) * a.Hkv + h) * a.copies + cp) * (static_cast<size_t>(a.T) * a.G),
          0);
    for (int k = kw; k < a.copies * more.y; k += KW)
      add(a.cta_ml, a.cta_o,
          static_cast<size_t>(more.x + k / a.copies) * kRows + k % a.copies * lanes_per_copy,
          rt * kRows);
  }
  if constexpr (KW > 1) {
    if (kw > 0) {
#pragma unroll
      for (int j = 0; j < DN; ++j)
        s_sum[kw - 1][j][lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      s_sum[kw - 1][DN][lane] = make_float4(m[0], m[1], l[0], l[1]);
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll 1
    for (int k = 0; k < KW - 1; ++k) {
      const float4 ml = s_sum[k][DN][lane];
      const float m2[2] = {ml.x, ml.y}, l2[2] = {ml.z, ml.w};
      float f1[2], f2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mx = fmaxf(m[i], m2[i]);
        f1[i] = m[i] == -INFINITY ? 0.f : uno::ex2(m[i] - mx);
        f2[i] = m2[i] == -INFINITY ? 0.f : uno::ex2(m2[i] - mx);
        l[i] = (l[i] != l[i] ? l[i] : l[i] * f1[i]) + (l2[i] != l2[i] ? l2[i] : l2[i] * f2[i]);
        m[i] = mx;
      }
#pragma unroll
      for (int j = 0; j < DN; ++j) {
        const float4 v = s_sum[k][j][lane];
        o[j][0] = fmaf(v.x, f2[0], o[j][0] * f1[0]);
        o[j][1] = fmaf(v.y, f2[0], o[j][1] * f1[0]);
        o[j][2] = fmaf(v.z, f2[1], o[j][2] * f1[1]);
        o[j][3] = fmaf(v.w, f2[1], o[j][3] * f1[1]);
      }
    }
  }
  if (sq.bad || lost) l[0] = l[1] = quiet_nan();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (rows[i] >= R) continue;
    const float inv = 1.f / l[i];
    uint4* dst = reinterpret_cast<uint4*>(a.out + q_at(i) + c * (D / 4));
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < DN / 8; ++k) {
        const int j = 8 * k, e = 2 * i + q;
        dst[q * (DN / 8) + k] =
            make_uint4(pack_bf16(o[j][e] * inv, o[j + 1][e] * inv),
                       pack_bf16(o[j + 2][e] * inv, o[j + 3][e] * inv),
                       pack_bf16(o[j + 4][e] * inv, o[j + 5][e] * inv),
                       pack_bf16(o[j + 6][e] * inv, o[j + 7][e] * inv));
      }
  }
}

// ---- host side ------------------------------------------------------------------

// Failure-path test hook (uno_attention_test_hook); zero: normal operation.
std::atomic<uint32_t> g_test_query_segments{0};

int copies_for(long long rows) {
  return rows <= kFewRows ? 1 : rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

struct Layout {
  size_t item_ml, item_o, cta_ml, cta_o, bytes;
};

Layout layout(int B, int T, int Hq, int Hkv, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const long long rows = static_cast<long long>(T) * (Hq / Hkv);
  const size_t items = static_cast<size_t>(B) * Hkv * rows * copies_for(rows);
  const size_t lanes = static_cast<size_t>(kMaxCtas) * kRows;
  Layout w;
  w.item_ml = up(sizeof(int2) * static_cast<size_t>(B) * Hkv * ((rows + kRows - 1) / kRows));
  w.item_o = w.item_ml + up(sizeof(float2) * items);
  w.cta_ml = w.item_o + up(sizeof(float) * items * D);
  w.cta_o = w.cta_ml + up(sizeof(float2) * lanes);
  w.bytes = w.cta_o + sizeof(float) * lanes * D;
  return w;
}

bool cache_map(CUtensorMap* map, const void* codes, long long rows, int D, int unit) {
  auto enc = uno_host::tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(unit)};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename... Args>
int launch(K kern, unsigned grid, int threads, int smem, bool early, cudaStream_t st,
           const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = early;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  return UNO_OK;
}

template <int D, int COPIES, int FEW = 0>
int launch_cached(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                  cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // devices with the shared-memory opt-in
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return UNO_ERR_CUDA;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (!bit || !(attr_done.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(cached_kernel<D, COPIES, FEW>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<D, FEW>::kBytes) != cudaSuccess)
      return UNO_ERR_CUDA;
    attr_done.fetch_or(bit, std::memory_order_relaxed);
  }
  // a CTA per unit at most, as far as the host can know
  const long long rts = (static_cast<long long>(a.T) * a.G + kRows - 1) / kRows;
  const long long tiles = (static_cast<long long>(a.width) * a.page + kTile - 1) / kTile;
  long long ctas = std::min<long long>(a.B * rts, kMaxCtas) * a.Hkv;
  ctas = std::min<long long>(ctas, kMaxCtas) * std::min<long long>(tiles, kMaxCtas);
  ctas = std::max<long long>(std::min<long long>(ctas, kMaxCtas), 1);
  return launch(cached_kernel<D, COPIES, FEW>, static_cast<unsigned>(ctas), threads(COPIES),
                Plan<D, FEW>::kBytes, true, st, mk, mv, a);
}

template <int D>
int launch_all(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, bool cached,
               cudaStream_t st) {
  if (cached) {
    const int rows = a.T * a.G;
    const int rc = rows <= 4       ? launch_cached<D, 2, 4>(mk, mv, a, st)
                   : rows <= 8     ? launch_cached<D, 3, 8>(mk, mv, a, st)
                   : rows <= kFewRows ? launch_cached<D, 3, kFewRows>(mk, mv, a, st)
                   : a.copies == 4 ? launch_cached<D, 4>(mk, mv, a, st)
                   : a.copies == 2 ? launch_cached<D, 2>(mk, mv, a, st)
                                   : launch_cached<D, 1>(mk, mv, a, st);
    if (rc != UNO_OK) return rc;
  }
  // (finish_kernel reads its inputs before it waits for the launch before it: it may
  // start early only behind cached_kernel, which has waited for what wrote them)
  // four warps per 16 rows while that leaves the GPU room, one when there are many
  const long long items =
      static_cast<long long>(a.B) * a.Hkv * ((static_cast<long long>(a.T) * a.G + 15) / 16);
  if (items <= 4 * kMaxCtas)
    return launch(finish_kernel<D, 4>, static_cast<unsigned>(items), 128, 0, cached, st, a);
  return launch(finish_kernel<D, 1>, static_cast<unsigned>((items + 3) / 4), 128, 0, cached, st, a);
}

bool sizes_ok(int B, int T, int Hq, int Hkv, int D, int page, int width, int num_pages) {
  return uno_host::cache_sizes_ok(B, T, Hkv, D, page, width, num_pages) && T <= kMaxT &&
         Hq >= Hkv && Hq % Hkv == 0 && Hq <= 16384 &&
         static_cast<long long>(B) * Hkv * ((static_cast<long long>(T) * (Hq / Hkv) + 15) / 16) <=
             0x7FFFFFFFll &&
         static_cast<long long>(num_pages) * Hkv * page <= 0x7FFFFFFFll;
}

}  // namespace

namespace uno_host {

int attention_fault_flags(bool clear, unsigned* flags) {
  if (cudaMemcpyFromSymbol(flags, g_attn_fault, sizeof(unsigned)) != cudaSuccess)
    return UNO_ERR_CUDA;
  const unsigned zero = 0;
  if (clear && cudaMemcpyToSymbol(g_attn_fault, &zero, sizeof(unsigned)) != cudaSuccess)
    return UNO_ERR_CUDA;
  return UNO_OK;
}

}  // namespace uno_host

extern "C" int uno_attention_test_hook(uint32_t query_segments) {
  g_test_query_segments.store(query_segments);
  return UNO_OK;
}

extern "C" size_t uno_block_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  if (!sizes_ok(B, T, Hq, Hkv, D, 64, 0, 0)) return 0;
  return layout(B, T, Hq, Hkv, D).bytes;
}

extern "C" int uno_block_attention(const void* q, const void* k_new, const void* v_new,
                                   const int32_t* lens, const int32_t* parent,
                                   const int32_t* num_new, float scale, int B, int T, int Hq,
                                   int Hkv, int D, int page, const int32_t* page_table, int width,
                                   int num_pages, const void* k_codes, const void* v_codes,
                                   const float* k_scale, const float* v_scale, void* out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(B, T, Hq, Hkv, D, page, width, num_pages)) return UNO_ERR_SIZE;
  if (!(scale > -INFINITY && scale < INFINITY)) return UNO_ERR_SIZE;
  if (B == 0 || T == 0) return UNO_OK;
  for (const void* p : {q, k_new, v_new, static_cast<const void*>(out)}) {
    if (!p) return UNO_ERR_NULL;
    if (!uno_host::aligned(p, 16)) return UNO_ERR_ALIGN;
  }
  if (!lens) return UNO_ERR_NULL;
  const bool cached = width > 0 && num_pages > 0;  // else every length has to be 0
  if (cached && (!page_table || !k_codes || !v_codes || !k_scale || !v_scale)) return UNO_ERR_NULL;
  if (!uno_host::aligned(k_codes, 16) || !uno_host::aligned(v_codes, 16)) return UNO_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(parent),
                        static_cast<const void*>(num_new), static_cast<const void*>(page_table),
                        static_cast<const void*>(k_scale), static_cast<const void*>(v_scale)})
    if (!uno_host::aligned(p, 4)) return UNO_ERR_ALIGN;
  const Layout w = layout(B, T, Hq, Hkv, D);
  if (!workspace || workspace_bytes < w.bytes) return UNO_ERR_WORKSPACE;
  if (!uno_host::aligned(workspace, 16)) return UNO_ERR_ALIGN;
  const int dev = uno_host::check_device();
  if (dev != UNO_OK) return dev;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.out = static_cast<uint16_t*>(out);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = page_table;
  a.lens = lens;
  a.parent = parent;
  a.num_new = num_new;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.page = page;
  a.width = cached ? width : 0;
  a.num_pages = num_pages;
  a.scale = scale;
  const uint32_t segments = g_test_query_segments.load();
  a.query_segments = segments && segments < 0x7FFFFFFFu ? static_cast<int>(segments) : 0x7FFFFFFF;
  char* ws = static_cast<char*>(workspace);
  a.item_ctas = reinterpret_cast<int2*>(ws);
  a.item_ml = reinterpret_cast<float2*>(ws + w.item_ml);
  a.item_o = reinterpret_cast<float*>(ws + w.item_o);
  a.cta_ml = reinterpret_cast<float2*>(ws + w.cta_ml);
  a.cta_o = reinterpret_cast<float*>(ws + w.cta_o);
  a.copies = copies_for(static_cast<long long>(T) * (Hq / Hkv));
  CUtensorMap mk{}, mv{};
  if (cached) {
    const long long map_rows = static_cast<long long>(num_pages) * Hkv * page;
    const int unit = std::min(page, kTile);
    if (!cache_map(&mk, k_codes, map_rows, D, unit) || !cache_map(&mv, v_codes, map_rows, D, unit))
      return UNO_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch_all<128>(mk, mv, a, cached, st) : launch_all<64>(mk, mv, a, cached, st);
}
