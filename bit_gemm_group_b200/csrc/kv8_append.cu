// kv8_append.cu -- write new key and value rows into the paged 8-bit cache,
// keys rotated by their position on the way.
//
// For each (page, head) that receives rows, keys and values apart:
//   s' = max(max |x| of the new rows / qmax, 1e-8), and at least the block's
//        scale s where the page already holds older rows of the sequence
//   older codes c -> round(c s / s') where s' > s;  new codes round(x / s')
// qmax = 127 (int8) or 448 (E4M3).
//
// Bound by HBM: 2 (4) bytes read and 1 written per element.  One CTA per
// (sequence, touched page, head, keys or values) holds the page's new rows in
// registers between the maximum and the codes, so a block is read once and its
// scale is written by one CTA, with no atomics.  A thread's piece is 16
// elements of a row that rotate with one another (8 and their 8 partners), so
// that nothing is read twice; the loads of its four pieces are in flight
// together.  In a decode step a CTA has one row; older codes are read only when
// the new row raises the maximum.
//
// 7107 rows of 8 heads of 128 in four sequences: 18 us (their 44 MB at the copy
// rate are 6.7), bound by a CTA's chain of table, rows, maximum and codes, about 5
// us four times over, and by instructions: the quotients in packed pairs and one
// test for all of a thread's non-finite elements took it from 23.  Half as many
// elements in twice the threads: 16 us, but a step of 64 sequences with one row
// each 9.2 us in place of 8.2.
#include "kv8.cuh"

namespace wq {
namespace kv8 {

constexpr int STEPS = 4;  // 16-element pieces per thread; T D / 64 threads

// (a, b) -> (a c - b s, b c + a s), every product and sum rounded (the packed
// multiplication and addition come out fused: one bit off)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = u;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(512)
    kv8_append_kernel(const T* __restrict__ K, const T* __restrict__ V, int64_t ldk, int64_t ldv,
                      int D, Cache c, Batch bt, Rope rp, int slots, int* status) {
  constexpr float TOP = FMT == WQ_W8_INT8 ? 127.f : 448.f;
  __shared__ float red[16];
  int64_t id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int h = int(id % c.heads);
  id /= c.heads;
  const int j = int(id % slots), b = int(id / slots);

  const int T_ = 1 << c.tshift;
  int r0;
  const int n = seq_rows(bt, b, &r0, status);
  if (n == 0) return;
  const int len = __ldg(bt.lens + b), start = len - n;
  if (start < 0) {
    if (threadIdx.x == 0) record_error(status, WQ_ERR_ARG);
    return;
  }
  const int col = (start >> c.tshift) + j;
  // (in 64 bits: the end of a page near 2^31 is no int)
  const int64_t begin = int64_t(col) << c.tshift;
  if (begin >= len) return;
  const int p0 = max(start, int(begin)), p1 = int(min(int64_t(len), begin + T_));
  const int64_t page = col < bt.width ? __ldg(bt.table + int64_t(b) * bt.width + col) : -1;
  if (page < 0 || page >= c.pages || (rp.cos != nullptr && p1 > rp.max_pos)) {
    if (threadIdx.x == 0) record_error(status, WQ_ERR_ARG);
    return;
  }
  const int slot0 = p0 & (T_ - 1), rows = p1 - p0;
  const int per = D >> 4;                       // pieces per row
  const int piece = int(threadIdx.x) % per;
  const int first = int(threadIdx.x) / per, rstep = int(blockDim.x) / per;
  // the piece's two runs of 8 elements, and where its angles are
  const int half = rp.rot >> 1;
  const bool turns = !is_v && rp.cos != nullptr && piece * 16 < rp.rot;
  const bool split = turns && !rp.interleaved;
  const int d0 = split ? piece * 8 : piece * 16, d1 = split ? d0 + half : d0 + 8;
  const T* src = (is_v ? V : K) + int64_t(r0 + (p0 - start)) * (is_v ? ldv : ldk) + int64_t(h) * D;
  const int64_t ld = is_v ? ldv : ldk;
  const int64_t blk = c.block(page, h);
  uint8_t* codes = (is_v ? c.vq : c.kq) + (blk << c.tshift) * D;
  float* sp = (is_v ? c.vs : c.ks) + blk;

  // the new rows (beyond the last, that one again), in pairs of elements
  uint64_t x[STEPS][8];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const T* row = src + int64_t(min(first + i * rstep, rows - 1)) * ld;
    float a[8] = {}, b8[8] = {};
    if (i * rstep < rows) {
      load8(row + d0, a);
      load8(row + d1, b8);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[i][e] = two(a[2 * e], a[2 * e + 1]);
      x[i][4 + e] = two(b8[2 * e], b8[2 * e + 1]);
    }
  }
  if (turns) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (i * rstep >= rows) break;
      const int64_t at = int64_t(p0 + min(first + i * rstep, rows - 1)) * half + piece * 8;
      float cs[8], sn[8];
      load8(rp.cos + at, cs);
      load8(rp.sin + at, sn);
      // pair e: elements e and e + 8 of the piece, or 2 e and 2 e + 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a[2], b[2];
        if (split) {
          split_two(x[i][e], a[0], a[1]);
          split_two(x[i][4 + e], b[0], b[1]);
        } else {
          split_two(x[i][2 * e], a[0], b[0]);
          split_two(x[i][2 * e + 1], a[1], b[1]);
        }
        turn(a[0], b[0], cs[2 * e], sn[2 * e]);
        turn(a[1], b[1], cs[2 * e + 1], sn[2 * e + 1]);
        if (split) {
          x[i][e] = two(a[0], a[1]);
          x[i][4 + e] = two(b[0], b[1]);
        } else {
          x[i][2 * e] = two(a[0], b[0]);
          x[i][2 * e + 1] = two(a[1], b[1]);
        }
      }
    }
  }
  // the largest magnitude; x 0 summed is no number where an element is not finite
  float m = 0.f;
  uint64_t odd = 0;
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, b;
      split_two(x[i][e], a, b);
      m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
      odd = fma_two(x[i][e], 0, odd);
    }
  float odd0, odd1;
  split_two(odd, odd0, odd1);
  const bool bad = odd0 != 0.f || odd1 != 0.f;
  if (bad) {  // of the finite ones; NaN as 0, infinities keep their sign and saturate
    m = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v[2];
        split_two(x[i][e], v[0], v[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (fabsf(v[k]) <= 3.4028234663852886e38f) m = fmaxf(m, fabsf(v[k]));
          if (v[k] != v[k]) v[k] = 0.f;
        }
        x[i][e] = two(v[0], v[1]);
      }
  }
  const float old = slot0 ? *sp : 0.f;
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();  // also: `old` has been read by every thread
  for (int w = 0; w < int(blockDim.x >> 5); ++w) m = fmaxf(m, red[w]);
  float s = fmaxf(div_rn(m, TOP), 1e-8f);
  if (slot0) s = fmaxf(s, old);
  if (threadIdx.x == 0) *sp = s;
  if (slot0 && s != old) {
    const float ratio = div_rn(old, s);
    for (int i = int(threadIdx.x) * 4; i < slot0 * D; i += int(blockDim.x) * 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + i);
      uint32_t o = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t byte = (w >> (8 * e)) & 0xFFu;
        uint32_t y;
        if (FMT == WQ_W8_INT8) {
          const float v = rintf(float(int8_t(byte)) * ratio);
          y = uint32_t(int(fminf(fmaxf(v, -127.f), 127.f))) & 0xFFu;
        } else {
          __nv_fp8_e4m3 f;
          f.__x = __nv_fp8_storage_t(byte);
          y = __nv_cvt_float_to_fp8(float(f) * ratio, __NV_SATFINITE, __NV_E4M3);
        }
        o |= y << (8 * e);
      }
      *reinterpret_cast<uint32_t*>(codes + i) = o;
    }
  }
  if (bad) {
    // (s TOP may round above the largest number)
    const float top = fminf(s * TOP, 3.4028234663852886e38f);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a, b;
        split_two(x[i][e], a, b);
        x[i][e] = two(fminf(fmaxf(a, -top), top), fminf(fmaxf(b, -top), top));
      }
  }
  // (a finite element is within half a unit of s TOP's last place, whose code is TOP)
  const float inv = __frcp_rn(s);
  const uint64_t s2 = two(s, s), minus_inv = two(-inv, -inv);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int r = first + i * rstep;
    if (r >= rows) break;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint64_t v[2] = {minus_quot_rn_two(x[i][2 * k], s2, minus_inv),
                       minus_quot_rn_two(x[i][2 * k + 1], s2, minus_inv)};
      float f[4];
      if (FMT == WQ_W8_INT8) {
        // the low byte of 1.5 2^23 - v is -v rounded half to even
        const uint64_t magic = two(12582912.f, 12582912.f), minus_one = two(-1.f, -1.f);
        v[0] = fma_two(v[0], minus_one, magic);
        v[1] = fma_two(v[1], minus_one, magic);
      }
      split_two(v[0], f[0], f[1]);
      split_two(v[1], f[2], f[3]);
      if (FMT == WQ_W8_INT8) {
        o[k] = low_bytes4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
      } else {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
        o[k] = (a | (b << 16)) ^ 0x80808080u;
      }
    }
    uint8_t* dst = codes + int64_t(slot0 + r) * D;
    *reinterpret_cast<uint2*>(dst + d0) = make_uint2(o[0], o[1]);
    *reinterpret_cast<uint2*>(dst + d1) = make_uint2(o[2], o[3]);
  }
  if (bad) record_error(status, WQ_ERR_NONFINITE);
}

}  // namespace kv8
}  // namespace wq

namespace wq_host {

int launch_kv8_append(const void* K, const void* V, int dtype, int64_t ldk, int64_t ldv,
                      const Kv8& a, int max_pos, cudaStream_t s) {
  using namespace wq::kv8;
  const int T = a.page;
  int tshift = 0;
  while ((1 << tshift) < T) ++tshift;
  const Cache c{static_cast<uint8_t*>(a.kq), a.ks, static_cast<uint8_t*>(a.vq), a.vs, a.pages,
                int(a.kv_heads), tshift};
  const Batch bt{a.table, a.cu, a.lens, int(a.B), int(a.width), int(a.rows), int(a.max_new)};
  const Rope rp{a.cos, a.sin, int(a.rot), max_pos, a.interleaved};
  const int slots = int((a.max_new + T - 2) / T + 1);
  const int64_t blocks = int64_t(a.B) * slots * a.kv_heads * 2;
  if (blocks > 0x7fffffff) return WQ_ERR_UNSUPPORTED;
  const int threads = int(T * a.D / 64) < 32 ? 32 : int(T * a.D / 64);
  const unsigned grid = unsigned(blocks);
#define WQ_APPEND(TYPE, FMT)                                                              \
  kv8_append_kernel<TYPE, FMT><<<grid, threads, 0, s>>>(                                  \
      static_cast<const TYPE*>(K), static_cast<const TYPE*>(V), ldk, ldv, int(a.D), c, bt, rp, \
      slots, status_ptr())
  const bool i8 = a.fmt == WQ_W8_INT8;
  if (dtype == WQ_F32) {
    if (i8) WQ_APPEND(float, WQ_W8_INT8);
    else WQ_APPEND(float, WQ_W8_E4M3);
  } else if (dtype == WQ_BF16) {
    if (i8) WQ_APPEND(__nv_bfloat16, WQ_W8_INT8);
    else WQ_APPEND(__nv_bfloat16, WQ_W8_E4M3);
  } else {
    if (i8) WQ_APPEND(__half, WQ_W8_INT8);
    else WQ_APPEND(__half, WQ_W8_E4M3);
  }
#undef WQ_APPEND
  WQ_LAUNCH_CHECK("kv8_append_kernel");
  return WQ_OK;
}

}  // namespace wq_host
