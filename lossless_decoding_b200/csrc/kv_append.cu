// Rows of new keys and values into a paged 8-bit cache with a scale per page
// and KV head.
//
// A page holds `page` tokens of every head, head by head: [Hkv][page][D] e4m3
// codes; a code stands for code * scale[page][head]. Scales are powers of two,
// the smallest with max|x| <= 448 scale over the page's tokens: e4m3 is a
// floating-point format, so a power of two costs no precision, x / scale
// is exact, and when a later token makes the scale grow the earlier codes
// move by whole binades (exact but for codes that become subnormal). The
// page's codes therefore hardly depend on how its tokens were cut into calls.
//
// Bound by HBM: rows come in once (2 bytes) and codes go out once (1 byte);
// earlier tokens are touched only when the scale grows. One CTA per (touched
// page, head, K or V) holds the page's new rows in registers between the
// maximum and the conversion, eight 16-byte pieces per thread at most.
#include <cstdint>
#include <cuda_runtime.h>

#include "uno.h"
#include "uno_device.cuh"
#include "uno_host.h"

namespace {

struct AppendArgs {
  const uint16_t* x[2];   // new keys, new values [B][T][Hkv][D] bf16
  uint8_t* codes[2];      // [num_pages][Hkv][page][D]
  float* scales[2];       // [num_pages][Hkv]
  const int32_t* table;   // [B][width] page ids
  const int32_t* start;   // [B] first position
  const int32_t* count;   // [B] tokens, or null (n each)
  const int32_t* rows;    // [B][n] row of x of each appended token, or null (token j = row j)
  int T, n, Hkv, D, page, width, num_pages, pages_per_seq;
};

constexpr int kPieces = 8;  // 16-byte pieces of new rows per thread

// The smallest power of two s with v <= 448 s (v finite, > 0), at least 2^-126.
__device__ __forceinline__ float scale_for(float v) {
  int e;
  const float m = frexpf(v, &e);  // v = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
  e = max(m <= 0.875f ? e - 9 : e - 8, -126);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_max[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = static_cast<int>(blockIdx.x) / a.pages_per_seq;
  const int pi = static_cast<int>(blockIdx.x) % a.pages_per_seq;
  const int head = blockIdx.y, kv = blockIdx.z;
  uno::launch_dependents();
  uno::grid_dependency_wait();
  const int start = a.start[b];
  const int count = a.count ? min(max(a.count[b], 0), a.n) : a.n;
  if (start < 0 || start > a.width * a.page) return;
  const int page_no = start / a.page + pi;
  // this page's tokens: appended tokens [t0, t1), slots t0 + start - page_no * page onwards
  const int t0 = max(page_no * a.page - start, 0);
  const int t1 = min((page_no + 1) * a.page - start, count);
  if (t0 >= t1 || page_no >= a.width) return;
  const int id = a.table[static_cast<size_t>(b) * a.width + page_no];
  if (id < 0 || id >= a.num_pages) return;
  const int slot0 = start + t0 - page_no * a.page;
  // 16-byte pieces: 2^lv of a row; a thread's pieces are `step` rows apart
  const int lv = a.D == 128 ? 4 : 3;
  const int step = static_cast<int>(blockDim.x) >> lv;
  const int first = tid >> lv, d = (tid - (first << lv)) * 8;
  const size_t stride = static_cast<size_t>(a.Hkv) * a.D;  // from token to token
  const uint16_t* x = a.x[kv] + static_cast<size_t>(b) * a.T * stride + head * a.D + d;
  uint4 v[kPieces];
  uint32_t top = 0;
  const int n = t1 - t0 - first;  // tokens from this thread's first one on
  if (a.rows) {
    const int32_t* rows = a.rows + static_cast<size_t>(b) * a.n + t0 + first;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int row = i * step < n ? rows[i * step] : 0;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i * step < n)
        v[i] = row < 0 || row >= a.T
                   ? make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u)
                   : *reinterpret_cast<const uint4*>(x + row * stride);
    }
  } else {
    const uint16_t* src = x + (t0 + first) * stride;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i * step < n) v[i] = *reinterpret_cast<const uint4*>(src + i * step * stride);
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k)  // bf16 magnitudes order like their bits
      top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
  if (top >= 0x7F80u) {  // infinities and NaN drop out
    top = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) top = max(top, lo);
        if (hi < 0x7F80u) top = max(top, hi);
      }
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) s_max[warp] = top;
  // the page's scale is read before the barrier that orders its one writer after every reader
  float* scale = a.scales[kv] + static_cast<size_t>(id) * a.Hkv + head;
  const float old = slot0 > 0 ? *scale : 0.f;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu,
                          lane < static_cast<int>(blockDim.x) / 32 ? s_max[lane] : 0u);
  const float amax = uno::bf16_bits_to_float(top);
  const float now = fmaxf(old, amax > 0.f ? scale_for(amax) : 0.f);
  if (tid == 0) *scale = now;
  uint8_t* codes =
      a.codes[kv] + (static_cast<size_t>(id) * a.Hkv + head) * a.page * static_cast<size_t>(a.D);
  const float inv = now > 0.f ? 1.f / now : 1.f;
  if (now > old) {  // the page's earlier tokens move to the larger scale
    const float grow = old / now;
    uint2* c = reinterpret_cast<uint2*>(codes);
    for (int p = tid; p < slot0 << lv; p += static_cast<int>(blockDim.x)) {
      const uint2 w = c[p];
      uint32_t o[2];
      const uint32_t in[2] = {w.x, w.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 f0 = from_e4m3x2(in[k] & 0xFFFFu), f1 = from_e4m3x2(in[k] >> 16);
        o[k] = e4m3x2(f0.x * grow, f0.y * grow) | (e4m3x2(f1.x * grow, f1.y * grow) << 16);
      }
      c[p] = make_uint2(o[0], o[1]);
    }
  }
  uint8_t* dst = codes + (slot0 + first) * a.D + d;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (i * step < n) {
      float f[8];
      uno::LogitRow<uint16_t>::unpack(v[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= inv;
      *reinterpret_cast<uint2*>(dst + i * step * a.D) =
          make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16),
                     e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
    }
  }
}

}  // namespace

extern "C" int uno_kv_append(const void* k_new, const void* v_new, const int32_t* start,
                             const int32_t* count, const int32_t* rows, int B, int T, int n,
                             int Hkv, int D, int page, const int32_t* page_table, int width,
                             int num_pages, void* k_codes, void* v_codes, float* k_scale,
                             float* v_scale, void* stream) {
  if (!uno_host::cache_sizes_ok(B, T, Hkv, D, page, width, num_pages) || n < 0 || n > (1 << 20))
    return UNO_ERR_SIZE;
  if (!rows && n > T) return UNO_ERR_SIZE;
  // tokens touch at most this many pages of a sequence, whatever slot they start at
  const long long per_seq = n == 0 ? 0 : (n + page - 2) / page + 1;
  if (per_seq * B > 0x7FFFFFFFll) return UNO_ERR_SIZE;
  // (of an empty pool or table no token is written, wherever it would go)
  if (B == 0 || n == 0 || T == 0 || width == 0 || num_pages == 0) return UNO_OK;
  for (const void* p : {k_new, v_new, static_cast<const void*>(k_codes),
                        static_cast<const void*>(v_codes)}) {
    if (!p) return UNO_ERR_NULL;
    if (!uno_host::aligned(p, 16)) return UNO_ERR_ALIGN;
  }
  for (const void* p : {static_cast<const void*>(start), static_cast<const void*>(page_table),
                        static_cast<const void*>(k_scale), static_cast<const void*>(v_scale)})
    if (!p) return UNO_ERR_NULL;
  for (const void* p : {static_cast<const void*>(start), static_cast<const void*>(count),
                        static_cast<const void*>(rows), static_cast<const void*>(page_table),
                        static_cast<const void*>(k_scale), static_cast<const void*>(v_scale)})
    if (!uno_host::aligned(p, 4)) return UNO_ERR_ALIGN;
  const int dev = uno_host::check_device();
  if (dev != UNO_OK) return dev;
  AppendArgs a{};
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.scales[0] = k_scale;
  a.scales[1] = v_scale;
  a.table = page_table;
  a.start = start;
  a.count = count;
  a.rows = rows;
  a.T = T;
  a.n = n;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.width = width;
  a.num_pages = num_pages;
  a.pages_per_seq = static_cast<int>(per_seq);
  // a page's new rows in kPieces pieces per thread: min(n, page) rows of D / 8 pieces
  const int pieces = (n < page ? n : page) * (D / 8);
  const int warps = (pieces + 32 * kPieces - 1) / (32 * kPieces);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(per_seq * B), static_cast<unsigned>(Hkv), 2);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv_append_kernel, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  return UNO_OK;
}
