// Rows to 8-bit integers with one scale each, alone or after a residual
// addition and an RMS norm: what an 8-bit projection reads.
//
//   h = x + residual                    (rounded to the rows' type)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   scale = max|y| / 127, q = rint(y / scale)
//
// Bound by HBM, and at 2 bytes in and 1 out nearly by issue slots: x (and the
// residual) come in once, h and q go out once, a row stays in registers between
// its loads and its stores, and an element costs few instructions (a rounding is
// one fma onto 1.5 * 2^23, whose low byte is then the integer). Measured, to
// q: norm with residual 1 x 4096 6 us, 1088 x 4096 12 us, 8192 x 4096 57 us; quantiser
// 8192 x 12288 46 us (6.6 TB/s). Widths that are not multiples of 8 go element by
// element: 8192 x 4095 133 us (norm) and 76 us (quantiser, 23 us at 4096). The row factor
// r = rsqrt(..) scales every |h w| alike, so max|y| = r max|h w| and
// q = rint(h w * (127 / max|h w|)): the sum of squares and the maximum are one
// block reduction, not two with the row read again between them.
//
// Maxima keep NaN and are compared as bit patterns across threads (NaN above
// infinity above every finite number), so that a non-finite row is seen: it
// stores scale = NaN and q = 0.
#include <cstdint>
#include <cuda_runtime.h>

#include "uno.h"
#include "uno_device.cuh"
#include "uno_host.h"

namespace {

constexpr int kMaxD = 32768;  // 1024 threads x 32 register-held values

struct RowArgs {
  const void* x;
  const void* residual;  // or null
  const void* w;         // null: no norm
  float eps;
  int M, d;
  void* h;      // or null
  void* y;      // or null
  int8_t* q;    // or null
  float* scale;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) {
  return uno::bf16_bits_to_float(v);
}
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return uno::float_to_bf16_bits(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// V consecutive elements: V = 8 in 16-byte vectors, V = 1 by themselves.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* f) {
  if constexpr (V == 1) {
    f[0] = to_f32<T>(*p);
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += uno::LogitRow<T>::kVec)
      uno::LogitRow<T>::unpack(*reinterpret_cast<const uint4*>(p + k), f + k);
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  if constexpr (V == 1) {
    *p = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]),
                                              bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// max(m, |v|) that keeps a NaN of either.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// The integers in the low bytes of V words to memory.
template <int V>
__device__ __forceinline__ void store_q(int8_t* p, const uint32_t* q) {
  if constexpr (V == 1) {
    *p = static_cast<int8_t>(q[0]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = __byte_perm(__byte_perm(q[4 * k], q[4 * k + 1], 0x0040),
                         __byte_perm(q[4 * k + 2], q[4 * k + 3], 0x0040), 0x5410);
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// f + r in the rows' type: written to h (where given) and read back from it.
template <typename T, int V>
__device__ __forceinline__ void add_rows(float* f, const float* r, T* h) {
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] += r[k];
  if constexpr (V == 8 && sizeof(T) == 2) {
    const uint4 w = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]),
                               bf16x2(f[6], f[7]));
    uno::LogitRow<T>::unpack(w, f);
    if (h) *reinterpret_cast<uint4*>(h) = w;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f32<T>(from_f32<T>(f[k]));
    if (h) store_v<T, V>(h, f);
  }
}

// Onto it a float32 rounds to an integer, to nearest even, that is then its low bits.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
constexpr float kLift = 0x1p64f;      // of rows whose 127 / max passes float32 (maxima below 2^-121)

// 127 / max of a row, infinite where it passes float32. Rounded up: a value of half the
// maximum is 63.5 steps and has to become 64 (nearest even), which it does if the product
// is 63.5 or a little more, and does not (for about half of all maxima) if it is a
// little less. Of bfloat16 rows every other value is right too: 127 x / max lies on a half,
// then 127 / max is exact, or at least 2^-17 x from one, 2^6 times the quotient's error.
__device__ __forceinline__ float steps_per_unit(float amax) {
  const float inv = 127.f / amax;
  // one step up where it is below the quotient (the remainder's sign is exact)
  return __uint_as_float(__float_as_uint(inv) + (fmaf(inv, amax, -127.f) < 0.f));
}

// One row per group of `warps` warps (rows_per_cta groups in a CTA; a group
// of one warp needs no shared memory). Each thread holds ITER pieces of V
// elements, a group's pieces interleaved so that its loads are coalesced.
template <typename T, int V, int ITER, bool NORM>
__global__ void __launch_bounds__(1024, 1) row_quant_kernel(const RowArgs a, int warps) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = static_cast<int>(blockDim.x) / 32 / warps;  // 1 when warps > 1
  const int row = static_cast<int>(blockIdx.x) * rows + warp / warps;
  const int tid = threadIdx.x - (warp / warps) * warps * 32;
  const int step = warps * 32 * V;
  uno::launch_dependents();
  uno::grid_dependency_wait();
  if (row >= a.M) return;  // whole warps (a group of several warps is a whole CTA)
  const size_t at = static_cast<size_t>(row) * a.d;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + at : nullptr;
  const T* w = static_cast<const T*>(a.w);
  float f[ITER][V];
  bool in[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int e = tid * V + i * step;
    in[i] = e < a.d;
#pragma unroll
    for (int k = 0; k < V; ++k) f[i][k] = 0.f;
    if (in[i]) load_v<T, V>(x + e, f[i]);
  }
  if (NORM) {
    T* h = static_cast<T*>(a.h);
    if (res) {
      float r[ITER][V];
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (in[i]) load_v<T, V>(res + tid * V + i * step, r[i]);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (in[i]) add_rows<T, V>(f[i], r[i], h ? h + at + tid * V + i * step : nullptr);
    } else if (h) {
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (in[i]) store_v<T, V>(h + at + tid * V + i * step, f[i]);
    }
  }
  float sum = 0.f, big = 0.f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (NORM) {
#pragma unroll
      for (int k = 0; k < V; ++k) sum = fmaf(f[i][k], f[i][k], sum);
      if (in[i]) {
        float g[V];
        load_v<T, V>(w + tid * V + i * step, g);
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] *= g[k];
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) big = max_abs(big, f[i][k]);
  }
  uint32_t top = __float_as_uint(big);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (NORM) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  if (warps > 1) {
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = top;
    }
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? s_max[lane] : 0u);
    if (NORM) {
      sum = lane < warps ? s_sum[lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
  }
  const float rstd = NORM ? 1.f / sqrtf(sum / static_cast<float>(a.d) + a.eps) : 1.f;
  if (NORM && a.y) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!in[i]) continue;
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = f[i][k] * rstd;
      store_v<T, V>(static_cast<T*>(a.y) + at + tid * V + i * step, v);
    }
  }
  if (!a.q) return;
  const float amax = __uint_as_float(top);
  const bool bad = top >= 0x7F800000u || !(sum < INFINITY) || !(rstd < INFINITY);
  const float inv = bad ? 0.f : steps_per_unit(amax);
  int8_t* dst = a.q + at + tid * V;
  if (inv < INFINITY) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!in[i]) continue;
      uint32_t q[V];
#pragma unroll
      for (int k = 0; k < V; ++k)
        q[k] = bad ? 0u : __float_as_uint(fmaf(f[i][k], inv, kRound));
      store_q<V>(dst + i * step, q);
    }
  } else {  // amax = 0, or lifted
    const float lifted = amax > 0.f ? steps_per_unit(amax * kLift) : 0.f;
#pragma unroll 1
    for (int i = 0; i < ITER; ++i) {
      if (tid * V + i * step >= a.d) break;
      uint32_t q[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < ITER; ++j)
          if (j == i) v = f[j][k];
        q[k] = __float_as_uint(fmaf(v * kLift, lifted, kRound));
      }
      store_q<V>(dst + i * step, q);
    }
  }
  if (tid == 0) a.scale[row] = bad ? __uint_as_float(0x7FC00000u) : amax * rstd / 127.f;
}

template <typename T, int V, int ITER, bool NORM>
int launch(const RowArgs& a, int warps, cudaStream_t st) {
  const int rows = warps == 1 ? 4 : 1;  // one-warp rows: four to a CTA
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.M + rows - 1) / rows));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps * rows));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, row_quant_kernel<T, V, ITER, NORM>, a, warps) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  return UNO_OK;
}

// uno_quantize_rows of bfloat16 rows in 16-byte pieces: the row stays packed in
// registers (half of what its float32 values would take, so that twice the rows
// are in flight), its maximum is taken two at a time over the bit patterns.
template <int ITER, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) quant_bf16_kernel(const RowArgs a) {
  __shared__ uint32_t s_max[THREADS / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int step = static_cast<int>(blockDim.x) * 8;
  uno::launch_dependents();
  uno::grid_dependency_wait();
  const size_t at = static_cast<size_t>(blockIdx.x) * a.d + tid * 8;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + at;
  uint4 v[ITER];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid * 8 + i * step < a.d) v[i] = *reinterpret_cast<const uint4*>(x + i * step);
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu,
                          lane < static_cast<int>(blockDim.x) / 32 ? s_max[lane] : 0u);
  const float amax = uno::bf16_bits_to_float(top);
  const bool bad = top >= 0x7F80u;
  const bool tiny = amax < 0x1p-120f;
  const float inv = bad || top == 0 ? 0.f : steps_per_unit(tiny ? amax * kLift : amax);
  int8_t* dst = a.q + at;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (tid * 8 + i * step >= a.d) continue;
    float f[8];
    uno::LogitRow<uint16_t>::unpack(v[i], f);
    uint32_t q[8];
    if (tiny) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= kLift;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      q[k] = bad ? 0u : __float_as_uint(fmaf(f[k], inv, kRound));
    store_q<8>(dst + i * step, q);
  }
  if (tid == 0) a.scale[blockIdx.x] = bad ? __uint_as_float(0x7FC00000u) : amax / 127.f;
}

template <int ITER, int THREADS>
int launch_quant_bf16(const RowArgs& a, int warps, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.M));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, quant_bf16_kernel<ITER, THREADS>, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return UNO_ERR_CUDA;
  }
  return UNO_OK;
}

template <typename T, bool NORM>
int run(const RowArgs& a, cudaStream_t st) {
  // 16-byte pieces when every row starts on a 16-byte boundary; any other
  // width goes element by element
  if (a.d % 8 == 0) {
    const int pieces = a.d / 8;
    // Few rows: one piece per thread, so that a row's latency is one round of
    // loads. Many rows: four, so that more rows are in flight on an SM.
    if (pieces <= 32 || (pieces <= 1024 && a.M <= 296))
      return launch<T, 8, 1, NORM>(a, (pieces + 31) / 32, st);
    if constexpr (sizeof(T) == 2 && !NORM) {
      if (pieces <= 2048) return launch_quant_bf16<4, 512>(a, (pieces + 127) / 128, st);
    }
    // (float32's would not fit 64 registers; with more, fewer rows are in flight)
    if (sizeof(T) == 4 && pieces <= 2048) return launch<T, 8, 2, NORM>(a, (pieces + 63) / 64, st);
    return launch<T, 8, 4, NORM>(a, (pieces + 127) / 128, st);
  }
  if (a.d <= 8192) return launch<T, 1, 8, NORM>(a, (a.d + 255) / 256, st);
  return launch<T, 1, 32, NORM>(a, (a.d + 1023) / 1024, st);
}

int check(const RowArgs& a, int dtype) {
  if (dtype != UNO_BF16 && dtype != UNO_F32) return UNO_ERR_DTYPE;
  if (a.M < 0 || a.M > (1 << 24) || a.d < 1 || a.d > kMaxD) return UNO_ERR_SIZE;
  if (a.M == 0) return UNO_OK;
  if (!a.x || (a.q && !a.scale) || (!a.q && !a.y)) return UNO_ERR_NULL;
  for (const void* p : {a.x, a.residual, a.w, static_cast<const void*>(a.h),
                        static_cast<const void*>(a.y), static_cast<const void*>(a.q)})
    if (!uno_host::aligned(p, 16)) return UNO_ERR_ALIGN;
  if (!uno_host::aligned(a.scale, 4)) return UNO_ERR_ALIGN;
  return 1;
}

}  // namespace

extern "C" int uno_rms_norm(const void* x, const void* residual, const void* w, float eps, int M,
                            int d, int dtype, void* h, void* y, int8_t* q, float* scale,
                            void* stream) {
  const RowArgs a{x, residual, w, eps, M, d, h, y, q, scale};
  if (!(eps >= 0.f) || !(eps < INFINITY)) return UNO_ERR_SIZE;
  const int chk = check(a, dtype);
  if (chk != 1) return chk;
  if (!w) return UNO_ERR_NULL;
  const int dev = uno_host::check_device();
  if (dev != UNO_OK) return dev;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == UNO_BF16 ? run<uint16_t, true>(a, st) : run<float, true>(a, st);
}

extern "C" int uno_quantize_rows(const void* x, int M, int d, int dtype, int8_t* q, float* scale,
                                 void* stream) {
  const RowArgs a{x, nullptr, nullptr, 0.f, M, d, nullptr, nullptr, q, scale};
  const int chk = check(a, dtype);
  if (chk != 1) return chk;
  if (!q) return UNO_ERR_NULL;
  const int dev = uno_host::check_device();
  if (dev != UNO_OK) return dev;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == UNO_BF16 ? run<uint16_t, false>(a, st) : run<float, false>(a, st);
}
