// Attention of a drafted block (or tree) over a paged 8-bit cache.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i . k_j)
//
// over the sequence's cached tokens (all of them) and its new tokens: j <= i
// of a block, or i's ancestors of a tree. Cached keys and values are e4m3 codes
// with a scale per page and head; the new ones are bfloat16.
//
// Bound. A cached token costs 2 D bytes per KV head and 4 D flops per query row
// (rows = new tokens x query heads per KV head). With few rows the stream of
// codes bounds the call (HBM), past some 60 rows the products do.
//
// Split. The work items are (sequence, KV head, tile of query rows), each a list
// of 64-token tiles of the cache and one unit for the new tokens. The units of
// all items form one line that the CTAs share out evenly, whatever the lengths
// of the sequences: a CTA's part starts and ends inside items, at most two of
// its items are shared with other CTAs, and those leave their partial sums in
// the workspace for the combine launch. (Lengths are on the device, so a split
// planned on the host would have to assume the longest.)
//
// Arithmetic. mma.sync m16n8k16 with float32 accumulation. Codes are decoded to
// half precision in registers (exact: e4m3 is a subset), queries are scaled per
// row by a power of two into its range (bfloat16's 8 bits fit its 11). The value
// scales go into the exponent: t = score log2(e) + log2(v_scale), the running
// maximum is taken over t, and p = 2^(t - max) is at most 1 and rounded to half
// (2^-11); the normaliser sums p / v_scale in float32. New tokens use bfloat16
// products on the raw rows (p rounded to 2^-9).
//
// Layout. One thread's fragment of a contraction needs no particular order of
// the contracted index, so the index is permuted until a thread's share is
// contiguous: lane (g, c) (g = lane / 4, c = lane % 4) reads key bytes
// [c D/4, (c + 1) D/4) of token g, and for values the D/8 bytes from g D/8
// of the four tokens whose weights it already holds from the score
// fragment. So codes go from TMA's swizzled tiles to registers in 16-byte
// loads without bank conflicts and without a transpose.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "sm100.cuh"
#include "uno.h"
#include "uno_device.cuh"
#include "uno_host.h"

namespace {

constexpr int kTile = 64;      // cached tokens per unit
constexpr int kStages = 5;     // tiles in shared memory
constexpr int kProducers = 2;  // TMA warps, alternating tiles
constexpr int kMaxCtas = 2 * 148;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

enum : unsigned { kFaultProducer = 8u, kFaultConsumer = 16u };
__device__ unsigned int g_attn_fault;

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
  float scale;            // softmax scale
  struct Head* head;      // workspace
  struct Desc* desc;      // [grid]
  float2* part_ml;        // [grid][2][ROWS] running maximum and normaliser
  float* part_o;          // [grid][2][ROWS][D]
};

struct Head {
  long long units;
  int ctas;  // CTAs that have a part
};

// The item that a CTA's part starts in.
struct Desc {
  long long start, end;  // its units
  int b, h, rt, pad;
};

// A sequence's share of the line of units.
struct Seq {
  int len;    // cached tokens (0 when invalid)
  int nn;     // new tokens
  int tiles;  // units per item
  int rts;    // row tiles
  bool bad;   // length outside the page table: the rows come out as NaN
  long long units;
};

template <int ROWS>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  s.len = a.lens[b];
  s.bad = s.len < 0 || s.len > a.width * a.page;
  if (s.bad) s.len = 0;
  s.nn = a.num_new ? min(max(a.num_new[b], 0), a.T) : a.T;
  s.tiles = (s.len + kTile - 1) / kTile + 1;
  s.rts = (s.nn * a.G + ROWS - 1) / ROWS;
  s.units = static_cast<long long>(a.Hkv) * s.rts * s.tiles;
  return s;
}

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ bool nonfinite2(uint32_t w) {  // either bfloat16 of a pair
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Shared-memory plan of a variant.
template <int D, int RW, int KW>
struct Plan {
  static constexpr int kRows = 16 * RW;
  static constexpr int kConsumers = RW * KW;
  static constexpr int kThreads = 32 * (kConsumers + kProducers);
  static constexpr int kStage = 2 * kTile * D;  // keys, values
  static constexpr int kScales = kStages * kStage;               // float4 [stage][4 groups]
  static constexpr int kMerge = kScales + kStages * 64;          // (KW - 1) warps' O, then m and l
  static constexpr int kMergeWarp = 16 * D * 4 + 32 * 16;
  static constexpr int kBars = kMerge + (KW - 1) * RW * kMergeWarp;
  static constexpr int kBytes = kBars + 2 * kStages * 8 + 1024;  // + alignment
  static constexpr int kCtasPerSm = kConsumers <= 4 ? 2 : 1;
};

template <int D, int RW, int KW>
__global__ void __launch_bounds__(Plan<D, RW, KW>::kThreads, Plan<D, RW, KW>::kCtasPerSm)
    attn_kernel(const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const AttnArgs a) {
  using P = Plan<D, RW, KW>;
  constexpr int ROWS = P::kRows;
  constexpr int KS = D / 16;       // k-steps of a score, 4 contiguous codes of a thread each
  constexpr int DN = D / 8;        // output column tiles
  constexpr int NT = 8 / KW;       // token n-tiles per warp and tile
  constexpr int NG = NT / 2;       // groups of 16 tokens per warp and tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float4* s_scale = reinterpret_cast<float4*>(smem + P::kScales);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t* empty = full + kStages;
  __shared__ long long s_u0, s_u1, s_base;
  __shared__ int s_b;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&empty[s], P::kConsumers);
    }
    s_abort = 0;
    sm100::fence_mbar_init();
  }
  uno::launch_dependents();
  uno::grid_dependency_wait();

  // This CTA's part [u0, u1) of the line, and the sequence it starts in.
  if (warp == 0) {
    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long long n = b0 + lane < a.B ? seq_of<ROWS>(a, b0 + lane).units : 0;
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
    if (u0 < u1) {
      for (int b0 = 0;; b0 += 32) {  // ends: u0 < total
        const long long n = b0 + lane < a.B ? seq_of<ROWS>(a, b0 + lane).units : 0;
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
    }
    if (lane == 0) {
      s_u0 = u0;
      s_u1 = u1;
      s_base = base;
      s_b = at;
      if (i == 0) *a.head = Head{total, ctas};
    }
  }
  __syncthreads();
  const long long u0 = s_u0, u1 = s_u1;

  // A segment: the part of one item that this CTA does.
  struct Segment {
    Seq s;
    int b, h, rt, t0, t1;  // units [t0, t1) of the item
    long long start;       // the item's first unit
  };
  long long base = s_base;
  int b = s_b;
  auto segment_at = [&](long long u) {
    Segment g;
    g.s = seq_of<ROWS>(a, b);
    while (u >= base + g.s.units) {
      base += g.s.units;
      g.s = seq_of<ROWS>(a, ++b);
    }
    g.b = b;
    const int item = static_cast<int>((u - base) / g.s.tiles);
    g.start = base + static_cast<long long>(item) * g.s.tiles;
    g.t0 = static_cast<int>(u - g.start);
    g.t1 = static_cast<int>(min(u1 - g.start, static_cast<long long>(g.s.tiles)));
    g.h = item / g.s.rts;
    g.rt = item - g.h * g.s.rts;
    return g;
  };

  if (warp >= P::kConsumers) {
    // ---- producers: tiles of the cache, alternating ----
    const int pr = warp - P::kConsumers;
    const int unit = min(a.page, kTile);  // tokens per TMA copy
    const int per = kTile / unit;         // copies per tile (and of keys and values each)
    int it = 0;                           // tiles of this CTA so far, over all segments
    int mine = -1;                        // this warp's last tile
    bool ok = true;
    for (long long u = u0; u < u1 && ok;) {
      const Segment g = segment_at(u);
      const int end = min(g.t1, g.s.tiles - 1);  // the last unit is the new tokens
      const int n = max(end - g.t0, 0);
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
        const float lv = vs != vs ? vs : log2f(vc);
        const int row = static_cast<int>(at) * a.page + pos % a.page;
        for (int k = 0; k < batch && j0 + k * kProducers < n; ++k) {
          const int i = it + j0 + k * kProducers;
          const int s = i % kStages;
          bool bad = i >= kStages && !sm100::mbar_wait(&empty[s], ((i / kStages) - 1) & 1, kWaitNs);
          if (bad) {
            atomicOr(&g_attn_fault, kFaultProducer);
            s_abort = 1;
          }
          if (__any_sync(0xFFFFFFFFu, bad || s_abort)) {
            ok = false;
            break;
          }
          const bool turn = lane / per == k;
          if (turn) {
            const int first = lane % per * (unit / 16);
            for (int e = 0; e < unit / 16; ++e)
              s_scale[s * 4 + first + e] = make_float4(ks, lv, 1.f / vc, 0.f);
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
      u = g.start + g.t1;
    }
    // No copy may still be landing when the CTA exits: wait for this warp's
    // among the last kStages tiles (the consumers have done so too, unless
    // they have given up).
    for (int i = max((ok ? it : mine + 1) - kStages, 0); i <= mine; ++i)
      if (i % kProducers == pr) sm100::mbar_wait(&full[i % kStages], (i / kStages) & 1, kWaitNs);
  } else {
    // ---- consumers: warp (rw, kw) has rows 16 rw.. and every KW-th share of a tile's tokens ----
    const int rw = warp % RW, kw = warp / RW;
    const int g = lane >> 2, c = lane & 3;
    bool ok = true;
    int it = 0;
    for (long long u = u0; u < u1;) {
      const Segment sg = segment_at(u);
      const int R = sg.s.nn * a.G;           // rows of the sequence and head
      const int r0 = sg.rt * ROWS + rw * 16; // this warp's first row
      const int rows[2] = {r0 + g, r0 + g + 8};
      // query row r: token r / G, head h * G + r % G
      size_t q_at[2];
      int tok[2];
      uint32_t qa[KS][4];
      float qf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = min(rows[i], R - 1);  // rows past the end repeat the last one, unstored
        tok[i] = r / a.G;
        q_at[i] = ((static_cast<size_t>(sg.b) * a.T + tok[i]) * a.Hq + sg.h * a.G + r % a.G) * D;
      }
      const bool live = r0 < R;  // warp-uniform
      auto load_q = [&](int i, uint32_t* w) {
        const uint4* p = reinterpret_cast<const uint4*>(a.q + q_at[i] + c * (D / 4));
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint4 v = __ldg(p + k);
          w[4 * k] = v.x;
          w[4 * k + 1] = v.y;
          w[4 * k + 2] = v.z;
          w[4 * k + 3] = v.w;
        }
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[D / 8];
        load_q(i, w);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // the row's largest magnitude moves to [2^13, 2^14)
        const int sh = min(13 + 127 - static_cast<int>(top >> 7), 120);
        const float f = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
        qf[i] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qa[k][i] = pack_f16(bf_lo(w[2 * k]) * f, bf_hi(w[2 * k]) * f);
          qa[k][i + 2] = pack_f16(bf_lo(w[2 * k + 1]) * f, bf_hi(w[2 * k + 1]) * f);
        }
      }
      float o[DN][4];
#pragma unroll
      for (int i = 0; i < DN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      // New reference for t[n][..] (n n-tiles): weights in place, o and l rescaled.
      auto rescale = [&](float (*t)[4], int n) {
        float mx[2] = {m[0], m[1]};
        for (int j = 0; j < n; ++j) {
          mx[0] = fmaxf(mx[0], fmaxf(t[j][0], t[j][1]));
          mx[1] = fmaxf(mx[1], fmaxf(t[j][2], t[j][3]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
        }
        const bool up = mx[0] > m[0] || mx[1] > m[1];
        if (__any_sync(0xFFFFFFFFu, up)) {
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
        for (int j = 0; j < n; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[j][e] = uno::ex2(t[j][e] - ref[e >> 1]);
      };

      // ---- cached tokens ----
      const int end = min(sg.t1, sg.s.tiles - 1);
      for (int ti = sg.t0; ti < end; ++ti, ++it) {
        const int s = it % kStages;
        if (ok && !sm100::mbar_wait(&full[s], (it / kStages) & 1, kWaitNs)) {
          if (lane == 0) atomicOr(&g_attn_fault, kFaultConsumer);
          s_abort = 1;
          ok = false;  // go on without waiting: the results are abandoned
        }
        if (live) {
          const uint8_t* sk = smem + s * P::kStage;
          const uint8_t* sv = sk + kTile * D;
          const int left = sg.s.len - ti * kTile;  // tokens of the tile that exist
          float t[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int tr = (kw * NT + n) * 8 + g;
            uint32_t w[D / 16];
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(sk + tr * 128 + (((2 * c) ^ g) << 4));
              const uint4 y =
                  *reinterpret_cast<const uint4*>(sk + tr * 128 + (((2 * c + 1) ^ g) << 4));
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
              w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
            } else {
              const uint4 x =
                  *reinterpret_cast<const uint4*>(sk + tr * 64 + ((c ^ ((g >> 1) & 3)) << 4));
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) t[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
              mma_f16(t[n], qa[k], halves(w[k] & 0xFFFFu), halves(w[k] >> 16));
          }
          float iv[NG];
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float4 sc = s_scale[s * 4 + kw * NG + i];
            iv[i] = sc.z;
            const float f0 = qf[0] * sc.x, f1 = qf[1] * sc.x;
#pragma unroll
            for (int n = 2 * i; n < 2 * i + 2; ++n) {
              t[n][0] = fmaf(t[n][0], f0, sc.y);
              t[n][1] = fmaf(t[n][1], f0, sc.y);
              t[n][2] = fmaf(t[n][2], f1, sc.y);
              t[n][3] = fmaf(t[n][3], f1, sc.y);
            }
          }
          if (left < kTile) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((kw * NT + n) * 8 + 2 * c + (e & 1) >= left) t[n][e] = -INFINITY;
          }
          rescale(t, NT);
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float* x = t[2 * i];
            const float* y = t[2 * i + 1];
            l[0] = fmaf(iv[i], (x[0] + x[1]) + (y[0] + y[1]), l[0]);
            l[1] = fmaf(iv[i], (x[2] + x[3]) + (y[2] + y[3]), l[1]);
            const uint32_t pa[4] = {pack_f16(x[0], x[1]), pack_f16(x[2], x[3]),
                                    pack_f16(y[0], y[1]), pack_f16(y[2], y[3])};
            const int tb = (kw * NG + i) * 16 + 2 * c;
            uint32_t w[4][D / 32];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tk = tb + (e & 1) + (e >> 1) * 8;
              if constexpr (D == 128) {
                const uint4 z =
                    *reinterpret_cast<const uint4*>(sv + tk * 128 + ((g ^ (tk & 7)) << 4));
                w[e][0] = z.x, w[e][1] = z.y, w[e][2] = z.z, w[e][3] = z.w;
              } else {
                const uint2 z = *reinterpret_cast<const uint2*>(
                    sv + tk * 64 + (((g >> 1) ^ ((tk >> 1) & 3)) << 4) + (g & 1) * 8);
                w[e][0] = z.x, w[e][1] = z.y;
              }
              // slots behind the sequence may hold anything, NaN too
              if (left < kTile && tk >= left) {
#pragma unroll
                for (int k = 0; k < D / 32; ++k) w[e][k] = 0u;
              }
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              const uint32_t a0 = __byte_perm(w[0][k], w[1][k], 0x5140);
              const uint32_t a1 = __byte_perm(w[0][k], w[1][k], 0x7362);
              const uint32_t b0 = __byte_perm(w[2][k], w[3][k], 0x5140);
              const uint32_t b1 = __byte_perm(w[2][k], w[3][k], 0x7362);
              mma_f16(o[4 * k], pa, halves(a0 & 0xFFFFu), halves(b0 & 0xFFFFu));
              mma_f16(o[4 * k + 1], pa, halves(a0 >> 16), halves(b0 >> 16));
              mma_f16(o[4 * k + 2], pa, halves(a1 & 0xFFFFu), halves(b1 & 0xFFFFu));
              mma_f16(o[4 * k + 3], pa, halves(a1 >> 16), halves(b1 >> 16));
            }
          }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&empty[s]);
      }

      // ---- new tokens: groups of 16, from the last one any row sees down ----
      if (live && sg.t1 == sg.s.tiles) {
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
        const int32_t* par = a.parent ? a.parent + static_cast<size_t>(sg.b) * a.T : nullptr;
        int cur[2] = {tok[0], tok[1]};  // the next ancestor to mark (trees)
        const int last = min(r0 + 15, R - 1) / a.G;
        for (int gi = last / 16; gi >= 0; --gi) {
          // rows see columns (bits) of this group
          uint32_t see[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (par) {
              see[i] = 0u;
              while (cur[i] >= gi * 16) {
                see[i] |= 1u << (cur[i] - gi * 16);
                const int up = __ldg(par + cur[i]);
                cur[i] = up < cur[i] ? up : -1;  // parents come before their children
              }
            } else {
              const int n = tok[i] - gi * 16 + 1;
              see[i] = n >= 16 ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
            }
          }
          if (gi % KW != kw) continue;
          float t[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int col = min(gi * 16 + n * 8 + g, last);
            const uint4* p = reinterpret_cast<const uint4*>(
                a.k_new + ((static_cast<size_t>(sg.b) * a.T + col) * a.Hkv + sg.h) * D +
                c * (D / 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) t[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              const uint4 v = __ldg(p + k);
              mma_bf16(t[n], qa[2 * k], v.x, v.y);
              mma_bf16(t[n], qa[2 * k + 1], v.z, v.w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              t[n][e] = (see[e >> 1] >> (n * 8 + 2 * c + (e & 1))) & 1u ? t[n][e] * f : -INFINITY;
          }
          rescale(t, 2);
          l[0] += (t[0][0] + t[0][1]) + (t[1][0] + t[1][1]);
          l[1] += (t[0][2] + t[0][3]) + (t[1][2] + t[1][3]);
          uint32_t w[4][D / 16];
          bool odd = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tk = min(gi * 16 + 2 * c + (e & 1) + (e >> 1) * 8, last);
            const uint4* p = reinterpret_cast<const uint4*>(
                a.v_new + ((static_cast<size_t>(sg.b) * a.T + tk) * a.Hkv + sg.h) * D +
                g * (D / 8));
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
              const uint4 v = __ldg(p + k);
              w[e][4 * k] = v.x, w[e][4 * k + 1] = v.y;
              w[e][4 * k + 2] = v.z, w[e][4 * k + 3] = v.w;
              odd |= nonfinite2(v.x) || nonfinite2(v.y) || nonfinite2(v.z) || nonfinite2(v.w);
            }
          }
          if (__any_sync(0xFFFFFFFFu, odd)) {
            // An infinity or NaN among the values: rows that do not see its token
            // must not meet it (0 times infinity), so this group goes row by row.
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
                  a.v_new + ((static_cast<size_t>(sg.b) * a.T + gi * 16 + tk) * a.Hkv + sg.h) * D;
#pragma unroll
              for (int j = 0; j < DN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if ((see[e >> 1] >> tk) & 1u)
                    o[j][e] = fmaf(pr[e >> 1],
                                   uno::bf16_bits_to_float(p[(2 * c + (e & 1)) * DN + j]), o[j][e]);
            }
          } else {
            const uint32_t pa[4] = {pack_bf16(t[0][0], t[0][1]), pack_bf16(t[0][2], t[0][3]),
                                    pack_bf16(t[1][0], t[1][1]), pack_bf16(t[1][2], t[1][3])};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              mma_bf16(o[2 * k], pa, __byte_perm(w[0][k], w[1][k], 0x5410),
                       __byte_perm(w[2][k], w[3][k], 0x5410));
              mma_bf16(o[2 * k + 1], pa, __byte_perm(w[0][k], w[1][k], 0x7632),
                       __byte_perm(w[2][k], w[3][k], 0x7632));
            }
          }
        }
      }

      // ---- the segment's sums ----
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      }
      if constexpr (KW > 1) {
        // the token shares of a row meet in shared memory
        constexpr int kConsumerThreads = 32 * P::kConsumers;
        auto slot = [&](int k) { return smem + P::kMerge + ((k - 1) * RW + rw) * P::kMergeWarp; };
        if (kw > 0) {
          float4* so = reinterpret_cast<float4*>(slot(kw));
#pragma unroll
          for (int j = 0; j < DN; ++j)
            so[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
          so[DN * 32 + lane] = make_float4(m[0], m[1], l[0], l[1]);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kConsumerThreads) : "memory");
        if (kw == 0) {
          for (int k = 1; k < KW; ++k) {
            const float4* so = reinterpret_cast<const float4*>(slot(k));
            const float4 ml = so[DN * 32 + lane];
            const float m2[2] = {ml.x, ml.y}, l2[2] = {ml.z, ml.w};
            float f1[2], f2[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mx = fmaxf(m[i], m2[i]);
              f1[i] = m[i] == -INFINITY ? 0.f : uno::ex2(m[i] - mx);
              f2[i] = m2[i] == -INFINITY ? 0.f : uno::ex2(m2[i] - mx);
              // a share without a finite maximum still carries its NaN
              l[i] = (l[i] != l[i] ? l[i] : l[i] * f1[i]) + (l2[i] != l2[i] ? l2[i] : l2[i] * f2[i]);
              m[i] = mx;
            }
#pragma unroll
            for (int j = 0; j < DN; ++j) {
              const float4 v = so[j * 32 + lane];
              o[j][0] = fmaf(v.x, f2[0], o[j][0] * f1[0]);
              o[j][1] = fmaf(v.y, f2[0], o[j][1] * f1[0]);
              o[j][2] = fmaf(v.z, f2[1], o[j][2] * f1[1]);
              o[j][3] = fmaf(v.w, f2[1], o[j][3] * f1[1]);
            }
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kConsumerThreads) : "memory");
      }
      if (kw == 0 && live) {
        if (sg.s.bad) l[0] = l[1] = __uint_as_float(0x7FC00000u);
        const bool whole = sg.t0 == 0 && sg.t1 == sg.s.tiles;
        const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + (sg.t0 > 0 ? 0 : 1)) * ROWS;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (rows[i] >= R) continue;
          if (whole) {
            const float inv = 1.f / l[i];
            uint4* dst = reinterpret_cast<uint4*>(a.out + q_at[i] + c * (D / 4));
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int k = 0; k < DN / 8; ++k) {
                const int j = 8 * k, e = 2 * i + n;
                dst[n * (DN / 8) + k] = make_uint4(
                    pack_bf16(o[j][e] * inv, o[j + 1][e] * inv),
                    pack_bf16(o[j + 2][e] * inv, o[j + 3][e] * inv),
                    pack_bf16(o[j + 4][e] * inv, o[j + 5][e] * inv),
                    pack_bf16(o[j + 6][e] * inv, o[j + 7][e] * inv));
              }
          } else {
            const size_t row = part + rw * 16 + g + 8 * i;
            float4* dst = reinterpret_cast<float4*>(a.part_o + row * D + c * (D / 4));
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int k = 0; k < DN / 4; ++k) {
                const int j = 4 * k, e = 2 * i + n;
                dst[n * (DN / 4) + k] = make_float4(o[j][e], o[j + 1][e], o[j + 2][e], o[j + 3][e]);
              }
            if (c == 0) a.part_ml[row] = make_float2(m[i], l[i]);
          }
        }
      }
      if (u == u0 && threadIdx.x == 0)
        a.desc[blockIdx.x] = Desc{sg.start, sg.start + sg.s.tiles, sg.b, sg.h, sg.rt, 0};
      u = sg.start + sg.t1;
    }
  }
}

// Items shared by several CTAs: block (i, .) handles the item that CTA i starts
// in the middle of, when i is the first such CTA of the item. A warp per row.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) combine_kernel(const AttnArgs a) {
  uno::launch_dependents();
  uno::grid_dependency_wait();
  const Head hd = *a.head;
  const int i = static_cast<int>(blockIdx.x) + 1;
  if (i >= hd.ctas) return;
  auto first_unit = [&](int j) { return hd.units * j / hd.ctas; };
  const Desc d = a.desc[i];
  if (first_unit(i) <= d.start || first_unit(i - 1) > d.start) return;
  const int lane = threadIdx.x & 31;
  const int rt_row = static_cast<int>(blockIdx.y) * 4 + (threadIdx.x >> 5);  // row of the tile
  const int nn = a.num_new ? min(max(a.num_new[d.b], 0), a.T) : a.T;
  const int r = d.rt * ROWS + rt_row;
  if (r >= nn * a.G) return;
  // CTA i - 1 began the item (its part's last piece), CTAs i.. go on (their first)
  int n = 1;
  while (i - 1 + n < hd.ctas && first_unit(i - 1 + n) < d.end) ++n;
  auto slot = [&](int k) {
    return (static_cast<size_t>(i - 1 + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + rt_row;
  };
  constexpr int E = D / 32;  // columns of a lane
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float mx = -INFINITY;
  for (int k = lane; k < n; k += 32) mx = fmaxf(mx, a.part_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  float l = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    float f = 0.f;
    if (k0 + lane < n) {
      const float2 ml = a.part_ml[slot(k0 + lane)];
      f = ml.x == -INFINITY ? 0.f : uno::ex2(ml.x - mx);
      l += ml.y != ml.y ? ml.y : ml.y * f;  // NaN stays, whatever its reference
    }
    const int m = min(32, n - k0);
    for (int k = 0; k < m; ++k) {
      const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
      const float* src = a.part_o + slot(k0 + k) * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(v.x, fk, acc[0]);
        acc[1] = fmaf(v.y, fk, acc[1]);
        acc[2] = fmaf(v.z, fk, acc[2]);
        acc[3] = fmaf(v.w, fk, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(v.x, fk, acc[0]);
        acc[1] = fmaf(v.y, fk, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  const float inv = 1.f / l;
  uint16_t* dst = a.out +
                  ((static_cast<size_t>(d.b) * a.T + r / a.G) * a.Hq + d.h * a.G + r % a.G) * D +
                  lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv),
                                                pack_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
}

// ---- host side ------------------------------------------------------------------

// Rows per CTA: all of a sequence's rows for one KV head where one tile holds
// them (in steps of the variants below), else tiles of 128.
int rows_for(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 80 ? 80 : 128; }

struct Layout {
  size_t desc, ml, o, bytes;
};

Layout layout(int rows, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout w;
  w.desc = 256;
  w.ml = w.desc + up(sizeof(Desc) * kMaxCtas);
  w.o = w.ml + up(sizeof(float2) * 2 * kMaxCtas * static_cast<size_t>(rows));
  w.bytes = w.o + sizeof(float) * 2 * kMaxCtas * static_cast<size_t>(rows) * D;
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

template <int D, int RW, int KW>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, cudaStream_t st) {
  using P = Plan<D, RW, KW>;
  static std::atomic<uint64_t> attr_done{0};  // devices with the shared-memory opt-in
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return UNO_ERR_CUDA;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (!bit || !(attr_done.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(attn_kernel<D, RW, KW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             P::kBytes) != cudaSuccess)
      return UNO_ERR_CUDA;
    attr_done.fetch_or(bit, std::memory_order_relaxed);
  }
  // a CTA per unit at most, as far as the host can know
  const long long rts = (static_cast<long long>(a.T) * a.G + P::kRows - 1) / P::kRows;
  const long long tiles = (static_cast<long long>(a.width) * a.page + kTile - 1) / kTile + 1;
  long long ctas = std::min<long long>(a.B * rts, kMaxCtas) * a.Hkv;
  ctas = std::min<long long>(ctas, kMaxCtas) * std::min<long long>(tiles, kMaxCtas);
  ctas = std::min<long long>(ctas, kMaxCtas / 2 * P::kCtasPerSm);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_kernel<D, RW, KW>, mk, mv, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  if (ctas == 1) return UNO_OK;  // nothing is shared
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), P::kRows / 4);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, combine_kernel<D, P::kRows>, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  return UNO_OK;
}

template <int D>
int launch_rows(int rows, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                cudaStream_t st) {
  switch (rows) {
    case 16: return launch<D, 1, 4>(mk, mv, a, st);
    case 32: return launch<D, 2, 2>(mk, mv, a, st);
    case 64: return launch<D, 4, 1>(mk, mv, a, st);
    case 80: return launch<D, 5, 1>(mk, mv, a, st);
    default: return launch<D, 8, 1>(mk, mv, a, st);
  }
}

bool sizes_ok(int B, int T, int Hq, int Hkv, int D, int page, int width, int num_pages) {
  return uno_host::cache_sizes_ok(B, T, Hkv, D, page, width, num_pages) && T <= 4096 &&
         Hq >= Hkv && Hq % Hkv == 0 && Hq <= 16384 &&
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

extern "C" size_t uno_block_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  if (!sizes_ok(B, T, Hq, Hkv, D, 64, 0, 0)) return 0;
  return layout(rows_for(static_cast<long long>(T) * (Hq / Hkv)), D).bytes;
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
  const int rows = rows_for(static_cast<long long>(T) * (Hq / Hkv));
  const Layout w = layout(rows, D);
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
  char* ws = static_cast<char*>(workspace);
  a.head = reinterpret_cast<Head*>(ws);
  a.desc = reinterpret_cast<Desc*>(ws + w.desc);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  CUtensorMap mk{}, mv{};
  if (cached) {
    const long long map_rows = static_cast<long long>(num_pages) * Hkv * page;
    const int unit = std::min(page, kTile);
    if (!cache_map(&mk, k_codes, map_rows, D, unit) || !cache_map(&mv, v_codes, map_rows, D, unit))
      return UNO_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch_rows<128>(rows, mk, mv, a, st) : launch_rows<64>(rows, mk, mv, a, st);
}
