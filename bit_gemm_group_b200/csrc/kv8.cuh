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

// Whether a row's maximum m must move for a score mx: asked of the exponent that mx would
// get, so that no weight passes 2^(LAG + OFF) whatever m + LAG or OFF - m round to (at 2^27
// a unit is 16).  False where there is no score.
__device__ __forceinline__ bool moves(float mx, float m) { return mx + (OFF - m) > LAG + OFF; }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 0x80 in each byte of a word that is an E4M3 NaN (0x7F or 0xFF).  The products
// multiply a weight of 0 by every value of a block that some row sees only in part,
// and 0 NaN is no 0: there NaN codes are taken as 0, and the rows that do see one
// are given their NaN at the end (a look at the codes again, for caches that hold
// one only).
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
// The word with its NaN codes, as e4m3_nans marks them, zeroed.
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t nans) {
  return w & ~((nans >> 7) * 0xFFu);
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// a / b for a >= 0, b > 0 (32-bit where both fit: a quarter of the instructions)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// U units in equal runs for up to `most` workers: the first `rem` runs have
// base + 1 units, the others base.  There are no more runs than make two units each, but
// for one of an odd U (a cut run costs a part in the workspace, about a unit's bytes).
struct Runs {
  int64_t base;
  int workers, rem;
  __device__ __forceinline__ Runs(int64_t U, int64_t most) {
    const int64_t w = (U + 1) >> 1;
    workers = int(w < most ? w : most);
    base = workers ? quotient(U, workers) : 0;
    rem = int(U - base * workers);
  }
  __device__ __forceinline__ int64_t start(int w) const { return w * base + min(w, rem); }
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t longer = rem * (base + 1);
    return u < longer ? int(quotient(u, base + 1)) : rem + int(quotient(u - longer, base));
  }
};

// Exclusive prefix sum of `mine` over the block's threads (NW warps); *total gets
// the sum.  Ends with a barrier of the block after `sums` has been read.
template <int NW>
__device__ __forceinline__ int64_t block_scan(int64_t mine, int64_t* sums, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return before + inc - mine;
}

// ------------------------------------------------------------------- joining
// What run w (w > 0) says about its start: whether that cuts a segment (first_run
// >= 0), which, and the runs first_run .. last_run that have parts of it.  A run's
// first segment is its part 0; only the first run can have begun with an earlier
// one, and then holds this one as its part 1.
struct __align__(16) Cut {
  int first_run, last_run, first_part, rows;  // rows: row block (row tile) of the segment
  int n, q0, h, pad;                          // of its sequence; kv head
};

// Written by one thread for each run, cutting or not.  The segment's units are
// `begin` and on, `extra` of them for its start and then `tiles`.
__device__ __forceinline__ void write_cut(Cut* cut, bool cuts, const Runs& runs, int64_t begin,
                                          int extra, int tiles, int rows, int n, int q0, int h) {
  int4 a = make_int4(-1, 0, 0, 0), b = make_int4(0, 0, 0, 0);
  if (cuts) {
    const int wa = runs.owner(begin + extra);
    a = make_int4(wa, runs.owner(begin + extra + tiles - 1), runs.start(wa) < begin ? 1 : 0, rows);
    b = make_int4(n, q0, h, 0);
  }
  reinterpret_cast<int4*>(cut)[0] = a;
  reinterpret_cast<int4*>(cut)[1] = b;
}

// A block of 8 warps at the start of run w.  The blocks of a segment's cuts share
// the work on 8 of its rows: `split` of them (a power of two up to 8) take part,
// block i the 8 / split rows from i * 8 / split on, with `split` warps per row.
struct JoinShare {
  int row, group, groups;  // this warp's row of the 8, its share of the parts
};
__device__ __forceinline__ bool join_share(int w, const Cut& c, JoinShare* js) {
  if (c.first_run < 0) return false;
  const int cuts = c.last_run - c.first_run, i = w - 1 - c.first_run;
  const int split = cuts >= 8 ? 8 : cuts >= 4 ? 4 : cuts >= 2 ? 2 : 1;
  if (i >= split) return false;
  const int warp = threadIdx.x >> 5, rows = 8 / split;
  js->row = i * rows + warp / split;
  js->group = warp % split;
  js->groups = split;
  return true;
}

// The sum of a row's parts of the runs first + group, first + group + groups, ...
// in order (l and, in lane e' of each 32, elements e 32 + e' of o), then of the
// groups in order through shared memory; true in the warp that holds the row.
// `row` of `rows` is the row's place in a part.
template <int D>
__device__ __forceinline__ bool join_row(const JoinShare& js, const Cut& cut, int rows, int row,
                                         const float* parts, const float* part_ml, float* l_out,
                                         float (&o)[D / 32]) {
  constexpr int PER = D / 32, BATCH = D == 256 ? 2 : 4;
  __shared__ float sm[8][2], so[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -__int_as_float(0x7f800000), l = 0.f;
  const float none = m;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int w0 = cut.first_run + js.group; w0 <= cut.last_run; w0 += js.groups * BATCH) {
    float pm[BATCH], pl[BATCH], po[BATCH][PER];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {  // (all in flight before the first is used)
      const int w = w0 + k * js.groups;
      pm[k] = none, pl[k] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) po[k][e] = 0.f;
      if (w <= cut.last_run) {
        const int64_t r = int64_t(w * 2 + (w == cut.first_run ? cut.first_part : 0)) * rows + row;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml + r * 2));
        pm[k] = ml.x, pl[k] = ml.y;
#pragma unroll
        for (int e = 0; e < PER; ++e) po[k][e] = __ldcg(parts + r * D + e * 32 + lane);
      }
    }
    float now = m;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) now = fmaxf(now, pm[k]);
    if (now == none) now = 0.f;
    const float a = exp2_approx(m - now);
    m = now;
    l *= a;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= a;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float x = exp2_approx(pm[k] - now);
      l = fmaf(pl[k], x, l);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(po[k][e], x, o[e]);
    }
  }
  if (js.groups > 1) {
    if (lane == 0) sm[warp][0] = m, sm[warp][1] = l;
#pragma unroll
    for (int e = 0; e < PER; ++e) so[warp][e * 32 + lane] = o[e];
    __syncthreads();
    if (js.group != 0) return false;
    float now = none;
    for (int k = 0; k < js.groups; ++k) now = fmaxf(now, sm[warp + k][0]);
    if (now == none) now = 0.f;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    for (int k = 0; k < js.groups; ++k) {
      const float x = exp2_approx(sm[warp + k][0] - now);
      l = fmaf(sm[warp + k][1], x, l);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(so[warp + k][e * 32 + lane], x, o[e]);
    }
  }
  *l_out = l;
  return true;
}

}  // namespace kv8
}  // namespace wq
