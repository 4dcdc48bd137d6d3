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
// rows per step, 8 steps, all eight loads in flight before the first use.
#include <cuda_fp8.h>

#include "kernels.h"
#include "qmath.cuh"

namespace wq {
namespace fp8b {

constexpr int THREADS = 256;
constexpr int STEPS = 8;  // 16 rows each

template <typename T>
struct Row8;
template <>
struct Row8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <typename T>
struct Row8 {
  uint4 v;
  __device__ void load(const T* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[8]) const {
    unpack2<T>(v.x, x[0], x[1]);
    unpack2<T>(v.y, x[2], x[3]);
    unpack2<T>(v.z, x[4], x[5]);
    unpack2<T>(v.w, x[6], x[7]);
  }
};

// Largest |x| of 8 elements, NaN skipped; `bad` is raised by any non-finite one.
__device__ __forceinline__ float absmax8(const float (&x)[8], bool& bad) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m = fmaxf(m, fabsf(x[e]));
    bad |= !(fabsf(x[e]) <= 3.4028234663852886e38f);
  }
  return m;
}

// Eight codes of x / s.  The quotients come from one reciprocal
// (quot_e4m3: the IEEE quotient's code, the division itself near half-way).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = make_float2(quot_e4m3(x[2 * j], s, inv), quot_e4m3(x[2 * j + 1], s, inv));
    h[j] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// ROWS = 128: scales [ceil(R / 128), KB].  ROWS = 1: scales [R, KB], or
// [KB, ld] with `transposed` (the layout the product reads).  `counters`
// (nullable): n_counters words of the product's workspace set to zero.
template <typename T, int ROWS>
__global__ void __launch_bounds__(THREADS)
    quantize_fp8_block_kernel(const T* __restrict__ X, int64_t R, int64_t K, uint8_t* __restrict__ q,
                              float* __restrict__ scales, int64_t ld, bool transposed,
                              int* __restrict__ counters, int n_counters, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[THREADS / 32];
  const int KB = int((K + 127) / 128);
  const int64_t tile = blockIdx.x;
  const int kb = int(tile % KB);
  const int64_t r0 = (tile / KB) * 128;
  const int c8 = (threadIdx.x & 15) * 8;
  const int64_t k = int64_t(kb) * 128 + c8;
  const int64_t row = r0 + (threadIdx.x >> 4);
  for (int i = int(tile) * THREADS + threadIdx.x; i < n_counters; i += int(gridDim.x) * THREADS)
    counters[i] = 0;

  Row8<T> v[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t r = row + 16 * i;
    if (r < R && k < K)
      v[i].load(X + r * K + k);
    else
      v[i].zero();
  }
  bool bad = false;
  float m[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    float x[8];
    v[i].get(x);
    m[i] = absmax8(x, bad);
  }
  if (ROWS == 128) {
    float a = m[0];
#pragma unroll
    for (int i = 1; i < STEPS; ++i) a = fmaxf(a, m[i]);
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) a = fmaxf(a, red[w]);
    const float s = fmaxf(div_rn(a, 448.f), 1e-8f);
    if (threadIdx.x == 0) scales[(r0 / 128) * KB + kb] = s;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) m[i] = s;
  } else {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
      m[i] = fmaxf(div_rn(m[i], 448.f), 1e-8f);
      const int64_t r = row + 16 * i;
      if ((threadIdx.x & 15) == 0 && r < R)
        scales[transposed ? int64_t(kb) * ld + r : r * ld + kb] = m[i];
    }
  }
  float inv = ROWS == 128 ? rcp_approx(m[0]) : 0.f;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t r = row + 16 * i;
    if (r >= R || k >= K) continue;
    float x[8];
    v[i].get(x);
    if (ROWS == 1) inv = rcp_approx(m[i]);
    *reinterpret_cast<uint2*>(q + r * K + k) = codes8(x, m[i], inv);
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
