// quantize_fp8_block.cu -- E4M3 codes with one fp32 scale per block of
// 128 x 128 elements (a weight) or 1 x 128 (an activation's token).
//
//   s[I, J] = max(max |x| over the block / 448, 1e-8)
//   q       = E4M3(fl32(x / s))   (round to nearest even, saturating)
//
// Bound by HBM: 2 (4) bytes read and 1 written per element, 4 per block.  A
// CTA of 256 threads owns a 128 x 128 tile and holds it in registers between
// the maximum and the codes, so the input is read once: 16 lanes x 8 elements
// cover a row's 128 columns (one 16-byte load per lane for 16-bit inputs), 16
// rows per step, 8 steps, all eight loads in flight before the first use.  For
// 1 x 128 blocks four lanes hold a row's block, so that its maximum takes two
// shuffles.  The quotient is a multiplication by 1 / s and Markstein's
// correction (a division per element was 262 us).  bf16: 28672 x 8192 in 128 x
// 128 blocks 119 us on an input used over and over, 5.9 TB/s, 132 on new ones; 2048 x
// 11008 in 1 x 128 blocks 16 us, of which half is the launch.
#include <cuda_fp8.h>

#include "kernels.h"
#include "qmath.cuh"

namespace wq {
namespace fp8b {

constexpr int THREADS = 256;
constexpr int STEPS = 8;  // 16 rows each

// Eight elements of a row, as loaded.  absmax: the largest magnitude, non-finite
// if one of them is.
template <typename T>
struct Row8 {  // 16-bit
  static constexpr int CTAS = 4;
  uint4 v;
  __device__ void load(const T* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ uint32_t absmax(uint32_t m) const {
    m = absmax2<T>(m, v.x);
    m = absmax2<T>(m, v.y);
    m = absmax2<T>(m, v.z);
    return absmax2<T>(m, v.w);
  }
  static __device__ float value(uint32_t m) {
    float a, b;
    unpack2<T>(m & 0x7FFF7FFFu, a, b);
    return a > b || a != a ? a : b;
  }
  __device__ void get(float (&x)[8]) const {
    unpack2<T>(v.x, x[0], x[1]);
    unpack2<T>(v.y, x[2], x[3]);
    unpack2<T>(v.z, x[4], x[5]);
    unpack2<T>(v.w, x[6], x[7]);
  }
};
template <>
struct Row8<float> {
  static constexpr int CTAS = 2;
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ uint32_t absmax(uint32_t m) const {
    float x[8];
    get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    return m;
  }
  static __device__ float value(uint32_t m) { return __uint_as_float(m); }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// The larger of two magnitudes (>= 0, infinite or NaN): a NaN's pattern is the
// largest.
__device__ __forceinline__ float max_mag(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// max(a / 448, 1e-8); of a block with a non-finite element, that.
__device__ __forceinline__ float scale_of(float a, bool& bad) {
  if (__float_as_uint(a) < 0x7F800000u) return fmaxf(div_rn(a, 448.f), 1e-8f);
  bad = true;
  return a;
}

// Eight codes of x / s, from inv = fl(1 / s).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 r = make_float2(quot_rn(x[2 * j], s, inv), quot_rn(x[2 * j + 1], s, inv));
    h[j] = __nv_cvt_float2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// ROWS = 128: scales [ceil(R / 128), KB].  ROWS = 1: scales [R, KB], or
// [KB, ld] with `transposed` (the layout the product reads).  `counters`
// (nullable): n_counters words of the product's workspace set to zero.
template <typename T, int ROWS>
__global__ void __launch_bounds__(THREADS, Row8<T>::CTAS)
    quantize_fp8_block_kernel(const T* __restrict__ X, int64_t R, int64_t K, uint8_t* __restrict__ q,
                              float* __restrict__ scales, int64_t ld, bool transposed,
                              int* __restrict__ counters, int n_counters, int* status) {
  // (for the product, which waits for this kernel before it reads its results; a
  // caller's own next kernel starts when this one is over)
  if (transposed) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[THREADS / 32];
  const int KB = int((K + 127) / 128);
  const int64_t tile = blockIdx.x;
  const int kb = int(tile % KB);
  const int64_t r0 = (tile / KB) * 128;
  // row and column of piece i
  const int64_t row0 = r0 + (ROWS == 1 ? threadIdx.x >> 2 : threadIdx.x >> 4);
  const int64_t k0 = int64_t(kb) * 128 + (ROWS == 1 ? threadIdx.x & 3 : threadIdx.x & 15) * 8;
  auto row_of = [&](int i) { return row0 + (ROWS == 1 ? (i >> 2) * 64 : i * 16); };
  auto col_of = [&](int i) { return k0 + (ROWS == 1 ? (i & 3) * 32 : 0); };
  for (int64_t i = tile * THREADS + threadIdx.x; i < n_counters; i += int64_t(gridDim.x) * THREADS)
    counters[i] = 0;

  Row8<T> v[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (row_of(i) < R && col_of(i) < K)
      v[i].load(X + row_of(i) * K + col_of(i));
    else
      v[i].zero();
  }
  bool bad = false;
  float s[2], inv[2];  // of pieces 0 to 3 and 4 to 7
  if (ROWS == 128) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) a = v[i].absmax(a);
    float f = Row8<T>::value(a);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f = max_mag(f, __shfl_xor_sync(0xffffffffu, f, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) f = max_mag(f, red[w]);
    s[0] = s[1] = scale_of(f, bad);
    if (threadIdx.x == 0) scales[(r0 / 128) * KB + kb] = s[0];
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) a = v[4 * j + i].absmax(a);
      float f = Row8<T>::value(a);
#pragma unroll
      for (int o = 2; o > 0; o >>= 1) f = max_mag(f, __shfl_xor_sync(0xffffffffu, f, o));
      s[j] = scale_of(f, bad);
      const int64_t r = row_of(4 * j);
      if ((threadIdx.x & 3) == 0 && r < R)
        scales[transposed ? int64_t(kb) * ld + r : r * ld + kb] = s[j];
    }
  }
  inv[0] = __frcp_rn(s[0]);
  inv[1] = ROWS == 128 ? inv[0] : __frcp_rn(s[1]);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (row_of(i) >= R || col_of(i) >= K) continue;
    float x[8];
    v[i].get(x);
    *reinterpret_cast<uint2*>(q + row_of(i) * K + col_of(i)) = codes8(x, s[i >> 2], inv[i >> 2]);
  }
  if (bad) record_error(status, WQ_ERR_NONFINITE);
}

}  // namespace fp8b
}  // namespace wq

namespace wq_host {

template <typename T>
static int launch_t(const void* X, int64_t R, int64_t K, int rows, void* q, float* scales,
                    int64_t ld, bool transposed, int* counters, int n_counters, cudaStream_t s) {
  const int64_t tiles = ((R + 127) / 128) * ((K + 127) / 128);
  if (tiles > 0x7fffffff) return WQ_ERR_UNSUPPORTED;
  const T* x = static_cast<const T*>(X);
  uint8_t* codes = static_cast<uint8_t*>(q);
  if (rows == 128)
    wq::fp8b::quantize_fp8_block_kernel<T, 128><<<unsigned(tiles), wq::fp8b::THREADS, 0, s>>>(
        x, R, K, codes, scales, ld, transposed, counters, n_counters, status_ptr());
  else
    wq::fp8b::quantize_fp8_block_kernel<T, 1><<<unsigned(tiles), wq::fp8b::THREADS, 0, s>>>(
        x, R, K, codes, scales, ld, transposed, counters, n_counters, status_ptr());
  WQ_LAUNCH_CHECK("quantize_fp8_block_kernel");
  return WQ_OK;
}

int launch_quantize_fp8_block(const void* X, int dtype, int64_t R, int64_t K, int rows, void* q,
                              float* scales, int64_t ld, bool transposed, int* counters,
                              int n_counters, cudaStream_t s) {
  switch (dtype) {
    case WQ_F32: return launch_t<float>(X, R, K, rows, q, scales, ld, transposed, counters, n_counters, s);
    case WQ_BF16: return launch_t<__nv_bfloat16>(X, R, K, rows, q, scales, ld, transposed, counters, n_counters, s);
    case WQ_F16: return launch_t<__half>(X, R, K, rows, q, scales, ld, transposed, counters, n_counters, s);
  }
  return WQ_ERR_ARG;
}

}  // namespace wq_host
