// kv8.cuh -- the paged 8-bit KV cache shared by its append and its attention.
//
// Codes of one (page, kv head) are a contiguous [T, D] block, int8 or E4M3;
// its keys and its values each have one fp32 scale.  Position p of sequence b
// is slot p % T of page table[b, p / T].
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"
#include "qmath.cuh"

namespace wq {
namespace kv8 {

struct Cache {
  uint8_t* kq;
  float* ks;
  uint8_t* vq;
  float* vs;
  int64_t pages;
  int heads, tshift;  // kv heads; T = 1 << tshift tokens per page
  __device__ __forceinline__ int64_t block(int64_t page, int h) const { return page * heads + h; }
};

// What the tokens of a call are: sequence b has the rows [cu[b], cu[b + 1]) and
// `lens[b]` positions in all, its rows being the last of them.
struct Batch {
  const int* table;
  const int* cu;
  const int* lens;
  int B, width, rows, max_new;
};

struct Rope {
  const float* cos;  // [max_pos, rot / 2], nullptr for no rotation
  const float* sin;
  int rot, max_pos;
  bool interleaved;
};

// Rows of sequence b, or 0 (and an error recorded) where cu is not usable.
__device__ __forceinline__ int seq_rows(const Batch& bt, int b, int* first, int* status) {
  const int r0 = __ldg(bt.cu + b), r1 = __ldg(bt.cu + b + 1);
  *first = r0;
  if (r0 < 0 || r1 < r0 || r1 > bt.rows || r1 - r0 > bt.max_new) {
    record_error(status, WQ_ERR_ARG);
    return 0;
  }
  return r1 - r0;
}

// 8 consecutive elements as fp32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  unpack2<T>(v.x, x[0], x[1]);
  unpack2<T>(v.y, x[2], x[3]);
  unpack2<T>(v.z, x[4], x[5]);
  unpack2<T>(v.w, x[6], x[7]);
}

// Elements [d, d + 8) of a head row after the rotation by position `pos`:
// pair (a, b) becomes (a cos - b sin, b cos + a sin), each product and sum
// rounded to fp32.  Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) when
// interleaved; elements from rot on stay.  rot % 16 == 0, so the eight
// elements are of one kind.
template <typename T>
__device__ __forceinline__ void rotated8(const T* row, int d, int pos, const Rope& rp,
                                         float (&x)[8]) {
  load8(row + d, x);
  if (rp.cos == nullptr || d >= rp.rot) return;
  const int half = rp.rot >> 1;
  const int64_t at = int64_t(pos) * half;
  if (rp.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(rp.cos + at + (d >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(rp.sin + at + (d >> 1)));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = __fsub_rn(__fmul_rn(a, cc[j]), __fmul_rn(b, ss[j]));
      x[2 * j + 1] = __fadd_rn(__fmul_rn(b, cc[j]), __fmul_rn(a, ss[j]));
    }
    return;
  }
  const bool upper = d >= half;
  const int i = upper ? d - half : d;
  float y[8], c[8], s[8];
  load8(row + (upper ? d - half : d + half), y);
  load8(rp.cos + at + i, c);
  load8(rp.sin + at + i, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = __fmul_rn(x[j], c[j]), q = __fmul_rn(y[j], s[j]);
    x[j] = upper ? __fadd_rn(p, q) : __fsub_rn(p, q);
  }
}

// The one-pass softmax of both attention kernels (its scheme: attn_kv8.cu).
constexpr float LAG = 8.f;  // how far a maximum may grow before the sums are rescaled
constexpr float OFF = 6.f;  // weights are kept 2^OFF above their exponential

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Units [u0, u1) of worker w: [w U / W, (w + 1) U / W).
__device__ __forceinline__ int64_t run_start(int64_t w, int64_t U, int64_t W) { return w * U / W; }
__device__ __forceinline__ int64_t run_owner(int64_t u, int64_t U, int64_t W) {
  return ((u + 1) * W - 1) / U;
}
// Workers in use: no run is shorter than two units (a cut run costs a part in
// the workspace, about a unit's bytes).
__device__ __forceinline__ int64_t workers(int64_t U, int64_t W) {
  const int64_t w = (U + 1) / 2;
  return w < W ? w : W;
}

}  // namespace kv8
}  // namespace wq
