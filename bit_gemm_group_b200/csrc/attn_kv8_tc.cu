// attn_kv8_tc.cu -- causal attention over the paged 8-bit cache for more than 32
// rows to a (sequence, kv head): prompts, chunks of prompts, long drafts.
//
// The mathematics of attn_kv8.cu on the fifth-generation tensor cores.  One CTA
// per SM; 128 rows (query, head) are one tensor-core tile, 64 positions a block:
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, a row per thread: scores
//                   from tensor memory, weights back to it as f16, over the scores
//   warps 8-11      converters of keys: a block's codes from the pages to f16
//                   (exactly) in shared memory, two blocks' loads ahead
//   warps 12-15     converters of values, into the same 128-byte swizzled layout
//                   (the product's sum runs along their rows: MN-major)
//   warps 16, 17    issue, a warp per tile, tcgen05.mma kind::f16: scores Q K^T
//                   (both operands in shared memory), then weights (tensor
//                   memory) times V; the scores run two blocks ahead
//   warps 18, 19    no work (registers are given in groups of four warps)
//
// PAIR: the two tiles are 256 rows of one (sequence, head) and share every
// converted block, which halves the conversion work: prompts.  Otherwise both
// tiles are the same 128 rows and take the blocks in turn, each with sums of its
// own that are joined at the end: drafts (while one tile's softmax runs the
// tensor cores work for the other), and fp16 inputs, whose queries are two f16
// terms (rounded, and what that left) so that a result is good to fp16.
//
// Two chunks, 3245 queries of 32 heads over 8 kv heads of 128, 9974 positions in
// all (E4M3): 314 us on inputs used over and over, 750 TFLOP/s of products; 322 on new
// ones.  Bound by the hand-offs: a
// block took a tile 2600 cycles at 431 us, of which its two products are 690
// (45 to 52 cycles per m128 n64 k16 score step, 60 to 68 per m128 n128 k16 value
// step) and its exponentials 512 of the special-function units.  Leaving one
// part out at a time, at 431 us, says that none of them is the limit by itself: no
// exponentials 399 us, no converter stores 419, no converter loads either 409, no
// sums 416; part of the exponentials as polynomials on the fma pipe 430 at best.
// (Not repeated since.)  The steps from there to 302 were the queries, which a row
// per lane fetched from L2 several times over, the weight of an item's start in the
// division of work, and waits (one that is over already costs 150 cycles): one less
// per block, the others where nothing waits for them.  What a row does not see although
// it is no number, and scores beyond 2^16, cost the 12 us from 302 to 314.
// Two score buffers of 64 positions per tile let the tensor cores run while the
// softmax works on the other.
//
// Items (row tile, head) are cut into blocks and numbered; each CTA takes an equal
// run of blocks, with START more for each item, and joins cut items as attn_kv8.cu
// does.
#include <math_constants.h>

#include <mutex>
#include <type_traits>

#include "kv8.cuh"
#include "tc.cuh"

namespace wq {
namespace kv8 {
namespace tcore {

// 20 warps of 96 registers at launch; the softmax keeps a block's 64 words of
// weights and takes 128, the converters 80, the issuers' four warps 64
constexpr int WARPS = 20, THREADS = WARPS * 32;
constexpr int REGS_SOFTMAX = 128, REGS_CONVERT = 80, REGS_ISSUE = 64;
static_assert(2 * REGS_SOFTMAX + 2 * REGS_CONVERT + REGS_ISSUE <= 5 * 96, "registers");
constexpr int TK = 64;      // positions per block
constexpr int STAGES = 4;   // blocks of keys and of values in shared memory
constexpr int SCALES = 8;   // blocks whose scales are kept
// Units that an item's queries, its first blocks' growing maxima and its results
// count, so that CTAs with many items end with the others (two prompt chunks: 354
// us with 4, 343 with 8, 335 with 11, 338 with 14; 36 rows over 2 x 4096 45 us with
// 4, 38 with 7 and with 11).
constexpr int START = 11;

// An item's (sequence, row tile) and how many blocks it has.
struct Item {
  int b, r, h;
  int n, q0, len, R, tiles;
  int hidden;  // first position that some query of the row tile does not see
  __device__ __forceinline__ void load(const Batch& bt, int tshift, int G, int rows, int* status) {
    n = seq_rows(bt, b, &q0, status);
    len = __ldg(bt.lens + b);
    const int64_t most = int64_t(bt.width) << tshift;
    if (len < 0 || len > most) {
      record_error(status, WQ_ERR_ARG);
      len = len < 0 ? 0 : int(most);
    }
    R = int((int64_t(n) * G + rows - 1) / rows);
    row_tile(G, rows);
  }
  __device__ __forceinline__ void row_tile(int G, int rows) {
    int64_t i = (int64_t(r + 1) * rows - 1) / G;  // the tile's last query
    if (i > n - 1) i = n - 1;
    int seen = len - n + int(i) + 1;
    seen = seen > len ? len : seen;
    tiles = seen > 0 ? (seen + TK - 1) / TK : 1;
    hidden = len - n + int(int64_t(r) * rows / G) + 1;
    hidden = hidden < 0 ? 0 : hidden < len ? hidden : len;
  }
  __device__ __forceinline__ bool valid() const { return n > 0 && r < R; }
};

// Walks over the work of a CTA's run: the item and its blocks [t0, t1).
struct Walk {
  Item it;
  int64_t begin, u0, u1;  // first unit of the item; the run
  int t0, t1;
  __device__ __forceinline__ void clip() {
    const int64_t a = u0 - begin - START, e = u1 - begin - START;
    t0 = a > 0 ? int(a) : 0;
    t1 = e < it.tiles ? int(e) : it.tiles;
  }
  // the next item with blocks in the run; false at its end
  __device__ __forceinline__ bool next(const Batch& bt, int heads, int tshift, int G, int rows) {
    while (true) {
      begin += it.tiles + START;
      if (begin >= u1) return false;
      if (++it.h == heads) {
        it.h = 0;
        if (++it.r < it.R) {
          it.row_tile(G, rows);
        } else {
          it.r = 0;
          do {
            if (++it.b >= bt.B) return false;
            it.load(bt, tshift, G, rows, nullptr);
          } while (it.n == 0);
        }
      }
      clip();
      if (t1 > t0) return true;
    }
  }
};

template <int D>
struct Smem {
  static constexpr int TILE = 128 * D * 2;  // 128 rows of f16
  static constexpr int BLOCK = TK * D * 2;
  static constexpr int BLOCKS = 2 * TILE + 2 * STAGES * BLOCK;  // Q 2, K, V
  struct Ctrl {
    uint64_t kfull[STAGES], kempty[STAGES], vfull[STAGES], vempty[STAGES], qfull;
    // per tile: two rounds in turn (a wait tells a round from the one two before,
    // which is known to be over, but not from the one in between)
    uint64_t sfull[2][2], pfull[2][2], odone[2][2];
    // An item of one block gives tile 1's issuer no round, so that nothing else says
    // that it has seen the item's queries: two items on, the parity of `qfull` would
    // tell it the wrong phase.
    uint64_t idle;
    uint64_t mfull, mfree, drain[2];
    // per block and 16 positions: ks, log2 vs, 1 / vs, written before the block's
    // keys are announced, read after the scores that waited for them are (a barrier
    // of their own cost the softmax 150 cycles a block).  A slot is written again 8
    // blocks later, when the scores 4 blocks later are done, whose predecessors 2
    // blocks back have been through the softmax.
    float4 scale[SCALES][TK / 16];
    float m[128], l[128];   // of tile 1, where both tiles are the same rows
    int64_t sum[WARPS], start_off;
    // every warp's place in the work (in registers it would be spilled, and local
    // memory comes back from L2 here)
    Walk walk[WARPS];
    int start_p, tmem_base, abort_flag;
    // set by the converters: a value's code or a scale that is no number where the rows
    // of an item differ in what they see (written before the block is announced, read
    // after its product is done)
    volatile int nans;
  };
  static constexpr size_t BYTES = 1024 + BLOCKS + sizeof(Ctrl);
};

constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (8u << 24);
}
// MN-major operand in 128-byte swizzled rows of 64 elements: groups of 64
// elements `lbo` bytes apart, groups of 8 rows (positions) 1024.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= uint64_t((addr & 0x3FFFFu) >> 4);
  d |= uint64_t(lbo >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Four codes of a word as two f16 pairs (see attn_kv8.cu).
template <int FMT>
__device__ __forceinline__ void expand(uint32_t w, uint32_t& a, uint32_t& b) {
  if (FMT == WQ_W8_INT8) {
    const uint32_t x = w ^ 0x80808080u;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(x, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(x, 0x64646464u, 0x4342)), "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
  }
}

__device__ __forceinline__ float as_f(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ uint64_t u32x2(uint32_t a, uint32_t b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
  return v;
}
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  return u32x2(__float_as_uint(a), __float_as_uint(b));
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

struct TcArgs {
  int64_t ldq;
  int heads, G, most_r;  // query heads, heads per kv head, row tiles of the longest sequence
  float scale_log2;
  float* parts;     // [2 W][ROWS][D]
  float* part_ml;   // [2 W][ROWS][2]
  Cut* cuts;        // [W] the items that the runs' starts cut
};

// Stages 32 rows of queries, row0 and on of the item's `total`, at dst (rows of 128
// bytes, planes of 64 elements `plane` bytes apart), and gives lane i row i's factor
// back.  D / 8 lanes share a row (a row per lane fetched every sector several times:
// a megabyte from L2 for 256 rows), each with two runs of four elements that rotate
// with one another, so that four rows' loads are on their way in 48 registers.
// Rounded as rotated8.  `parity` >= 0: only every second group of rows is written.
// TWO: `term` 1 writes what the rounding to f16 left.
template <typename TQ, int D, bool TWO>
__device__ __forceinline__ void stage_queries(const TQ* __restrict__ Q, const TcArgs& ar,
                                              const Rope& rp, const Item& it, int row0, int total,
                                              uint32_t dst, int plane, int parity, int term,
                                              float& fq, int* status) {
  constexpr int P = D / 8, RPP = 32 / P, BATCH = 4;
  const int lane = threadIdx.x & 31, p = lane % P, sub = lane / P;
  const int half = rp.rot >> 1;
  const bool turns = rp.max_pos > 0 && 8 * p < rp.rot, split = turns && !rp.interleaved;
  const int e0 = split ? 4 * p : 8 * p, e1 = split ? e0 + half : e0 + 4;
  const TQ* q0 = Q + int64_t(it.q0) * ar.ldq + int64_t(it.h) * ar.G * D;
  const uint32_t d0 = dst + (e0 / 64) * plane + (e0 & 4) * 2, d1 = dst + (e1 / 64) * plane + (e1 & 4) * 2;
#pragma unroll 1
  for (int s0 = 0; s0 < P; s0 += BATCH) {
    uint2 lo[BATCH], hi[BATCH];
    float4 c[BATCH], sn[BATCH];
    uint32_t plain = 0;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int qr = row0 + (s0 + k) * RPP + sub;
      const int row = qr < total ? qr : total - 1;  // (rows behind the last become zeros)
      const int i = row / ar.G, pos = it.len - it.n + i;
      const TQ* src = q0 + int64_t(i) * ar.ldq + (row - i * ar.G) * D;
      lo[k] = __ldg(reinterpret_cast<const uint2*>(src + e0));
      hi[k] = __ldg(reinterpret_cast<const uint2*>(src + e1));
      c[k] = make_float4(1.f, 1.f, 1.f, 1.f), sn[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rp.cos != nullptr && pos >= rp.max_pos) record_error(status, WQ_ERR_ARG);
      if (!turns || pos < 0 || pos >= rp.max_pos) {
        plain |= 1u << k;
      } else {
        c[k] = __ldg(reinterpret_cast<const float4*>(rp.cos + int64_t(pos) * half + 4 * p));
        sn[k] = __ldg(reinterpret_cast<const float4*>(rp.sin + int64_t(pos) * half + 4 * p));
      }
      if (qr >= total) lo[k] = hi[k] = make_uint2(0, 0);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      float v[8];
      unpack2<TQ>(lo[k].x, v[0], v[1]);
      unpack2<TQ>(lo[k].y, v[2], v[3]);
      unpack2<TQ>(hi[k].x, v[4], v[5]);
      unpack2<TQ>(hi[k].y, v[6], v[7]);
      if (!(plain >> k & 1)) {
        const float cc[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
        const float ss[4] = {sn[k].x, sn[k].y, sn[k].z, sn[k].w};
        // pair e: elements e and e + 4 of the eight, or 2 e and 2 e + 1
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = split ? v[e] : v[2 * e], b = split ? v[4 + e] : v[2 * e + 1];
          x[e] = __fsub_rn(__fmul_rn(a, cc[e]), __fmul_rn(b, ss[e]));
          x[4 + e] = __fadd_rn(__fmul_rn(b, cc[e]), __fmul_rn(a, ss[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = split ? x[e] : x[(e & 1) * 4 + (e >> 1)];
      }
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(v[e]));
#pragma unroll
      for (int o = P / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      // a power of two brings the row's largest element to [2^14, 2^15)
      int ex = (a > 0.f && a <= 3.4028234663852886e38f) ? 141 - int(__float_as_uint(a) >> 23) : 0;
      ex = ex > 100 ? 100 : ex;
      const float up = __uint_as_float(uint32_t(127 + ex) << 23);
      const int s = s0 + k;
      const float back = __shfl_sync(0xffffffffu, __uint_as_float(uint32_t(127 - ex) << 23),
                                     (lane % RPP) * P);
      if (lane / RPP == s) fq = back;
      if (parity >= 0 && (s & 1) != parity) continue;
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = v[2 * e] * up, z = v[2 * e + 1] * up;
        if (TWO && term == 1) {
          y -= __half2float(__float2half_rn(y));
          z -= __half2float(__float2half_rn(z));
        }
        h[e] = f16x2(y, z);
      }
      const int w = s * RPP + sub;
      sts64(d0 + w * 128 + ((((e0 & 63) >> 3) ^ (w & 7)) << 4), h[0], h[1]);
      sts64(d1 + w * 128 + ((((e1 & 63) >> 3) ^ (w & 7)) << 4), h[2], h[3]);
    }
  }
}

template <typename T>
__device__ __forceinline__ T nan_of() {
  if constexpr (std::is_same<T, __half>::value)
    return __float2half_rn(CUDART_NAN_F);
  else
    return __float2bfloat16_rn(CUDART_NAN_F);
}

// Beyond 2^16 what a fused v mul - m leaves over is no longer small against an exponent
// (2^95 at 1e36): for such a row scores are rounded before the maximum is taken off.
__device__ __forceinline__ bool is_far(float m) {
  return fabsf(m) > 65536.f && fabsf(m) <= 3.4028234663852886e38f;
}
// The weights of a block (its scores at `st`) against the maximum m, stored over the scores,
// and their sum, for a warp with such a row; the others as in the kernel's loop.
// Positions from `lim` on are not seen.  (In the loop: two prompt chunks 336 us back to
// back where this takes 313.)
__device__ __noinline__ float far_weights(uint32_t st, const float4* scl, float fq, float m,
                                          int lim) {
  const bool far = is_far(m);
  const float off = OFF - (m == -CUDART_INF_F ? 0.f : m);
  float sum = 0.f;
#pragma unroll 1
  for (int g = 0; g < TK / 16; ++g) {  // (weights take half the columns of their scores)
    uint32_t v[16], p[8];
    tc::tmem_ld_x16(st + g * 16, v);
    tc::tmem_wait_ld();
    const float4 f = scl[g];
    const float mul = fmaxf(fq * f.x, 1e-37f);
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float s = g * 16 + e >= lim ? -CUDART_INF_F : as_f(v[e]);
      const float x = exp2_approx(far ? fmaf(s, mul, f.y) + off : fmaf(s, mul, f.y + off));
      part[e & 3] += x;
      if (e & 1)
        p[e / 2] = f16x2(as_f(v[e - 1]), x);
      else
        v[e] = __float_as_uint(x);
    }
    sum = fmaf((part[0] + part[2]) + (part[1] + part[3]), f.z, sum);
    tc::tmem_st_x8(st + g * 8, p);
  }
  return sum;
}

template <typename TQ, int FMT, int D, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    attn_kv8_tc_kernel(const TQ* __restrict__ Q, TQ* __restrict__ O, Cache c, Batch bt, Rope rp,
                       TcArgs ar, int* status, uint64_t limit_ns) {
  using S = Smem<D>;
  constexpr int ROWS = PAIR ? 256 : 128;
  constexpr bool TWO = !PAIR && std::is_same<TQ, __half>::value;  // queries in two terms
  constexpr int PLANE = 128 * 128, KVPLANE = TK * 128;  // 128 (64) rows of 64 f16
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  auto& sm = *reinterpret_cast<typename S::Ctrl*>(base + S::BLOCKS);
  const uint32_t qs = tc::smem_u32(base), ksm = qs + 2 * S::TILE, vsm = ksm + STAGES * S::BLOCK;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T_ = 1 << c.tshift;

  // ------------------------------------------------ the run of this CTA
  const int P = bt.B * ar.most_r;
  auto units_at = [&](int p, int* st) {
    if (p >= P) return int64_t(0);
    Item it;
    it.b = p / ar.most_r;
    it.r = p - it.b * ar.most_r;
    it.load(bt, c.tshift, ar.G, ROWS, st);
    return it.valid() ? int64_t(it.tiles + START) * c.heads : int64_t(0);
  };
  const bool one = P <= THREADS;  // looked at once
  int64_t U = 0, part = 0, first = 0, units = 0;
  for (int p0 = 0; p0 < P; p0 += THREADS) {
    units = units_at(p0 + int(threadIdx.x), status);
    first = U + block_scan<WARPS>(units, sm.sum, &part);
    U += part;
  }
  const Runs runs(U, gridDim.x);
  if (int(blockIdx.x) >= runs.workers) {
    if (threadIdx.x == 0) write_cut(ar.cuts + blockIdx.x, false, runs, 0, 0, 0, 0, 0, 0, 0);
    return;
  }
  const int64_t u0 = runs.start(blockIdx.x), u1 = runs.start(blockIdx.x + 1);
  int64_t done = 0;
  for (int p0 = 0; p0 < P; p0 += THREADS) {
    if (!one) {
      units = units_at(p0 + int(threadIdx.x), nullptr);
      first = done + block_scan<WARPS>(units, sm.sum, &part);
      done += part;
    }
    if (units > 0 && u0 >= first && u0 < first + units) {
      sm.start_p = p0 + int(threadIdx.x);
      sm.start_off = u0 - first;
    }
  }
  __syncthreads();
  Walk wk;
  wk.u0 = u0, wk.u1 = u1;
  wk.it.b = sm.start_p / ar.most_r;
  wk.it.r = sm.start_p - wk.it.b * ar.most_r;
  wk.it.load(bt, c.tshift, ar.G, ROWS, nullptr);
  wk.it.h = int(quotient(sm.start_off, wk.it.tiles + START));
  wk.begin = u0 - (sm.start_off - int64_t(wk.it.h) * (wk.it.tiles + START));
  wk.clip();
  if (threadIdx.x == 0)
    write_cut(ar.cuts + blockIdx.x, wk.t0 > 0, runs, wk.begin, START, wk.it.tiles, wk.it.r,
              wk.it.n, wk.it.q0, wk.it.h);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      tc::mbar_init(&sm.kfull[i], 4);
      tc::mbar_init(&sm.vfull[i], 4);
      tc::mbar_init(&sm.kempty[i], PAIR ? 2 : 1);
      tc::mbar_init(&sm.vempty[i], PAIR ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) {
        tc::mbar_init(&sm.sfull[i][k], 1);
        tc::mbar_init(&sm.pfull[i][k], 4);
        tc::mbar_init(&sm.odone[i][k], 1);
      }
      tc::mbar_init(&sm.drain[i], 1);
    }
    tc::mbar_init(&sm.idle, 1);
    tc::mbar_init(&sm.mfull, 4);
    tc::mbar_init(&sm.mfree, 4);
    tc::mbar_init(&sm.qfull, 8);
    sm.abort_flag = 0;
    sm.nans = 0;
    tc::fence_mbar_init();
  }
  if (warp == 16) {
    tc::tmem_alloc(reinterpret_cast<uint32_t*>(&sm.tmem_base), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uint32_t(sm.tmem_base);
  // (the limit starts again with every item: a call may take longer than one wait)
  tc::Watchdog wd{tc::globaltimer_ns() + limit_ns, &sm.abort_flag, status};
  bool more = wk.t1 > wk.t0 || wk.next(bt, c.heads, c.tshift, ar.G, ROWS);
  if (lane == 0) sm.walk[warp] = wk;
  __syncwarp();
  const Walk& place = sm.walk[warp];
  const Item& it = place.it;
  auto step = [&]() {
    Walk w = place;
    const bool m = w.next(bt, c.heads, c.tshift, ar.G, ROWS);
    __syncwarp();
    if (lane == 0) sm.walk[warp] = w;
    __syncwarp();
    wd.deadline_ns = tc::globaltimer_ns() + limit_ns;
    return m;
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int x = warp >> 2;                       // tile
    const int row = (warp & 3) * 32 + lane;        // of the tile
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    // scores, and weights over them: two buffers of 64 columns, taken in turn
    const uint32_t st0 = tmem + lanes + uint32_t(x) * 128;
    const uint32_t ot = tmem + lanes + 256 + uint32_t(x) * 128;  // result
    uint32_t op = 0;  // tensor-core rounds of this tile so far
    bool ok = true, first_seg = true;
    uint32_t block = 0, seg = 0;  // blocks and items of the CTA so far
    uint32_t idles = 0;           // items without a round of this tile
    for (; more && ok; more = step(), ++seg) {
      const int rr = it.r * ROWS + (PAIR ? x * 128 : 0) + row;
      const bool live = rr < it.n * ar.G;
      const int i = live ? rr / ar.G : 0;
      const int pos = it.len - it.n + i;
      // (a row of no query takes part as zeros, and asks for no masking)
      const int lim = live ? min(it.len, pos + 1) : 0x7fffffff;
      // -------- the warp's 32 rows of queries, as f16 in the swizzled operand layout
      float fq = 0.f;
      {
        const uint32_t dst = qs + ((PAIR || TWO) ? x * S::TILE : 0) + (warp & 3) * 32 * 128;
        const int row0 = it.r * ROWS + (PAIR ? x * 128 : 0) + (warp & 3) * 32;
        // with one tile of one term each group of warps writes half of it; two terms:
        // group 0 the rounded query, group 1 what that left
        const int parity = !PAIR && !TWO ? x : -1;
        stage_queries<TQ, D, TWO>(Q, ar, rp, it, row0, it.n * ar.G, dst, PLANE, parity, x, fq,
                                  status);
        fq *= ar.scale_log2;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.qfull);
      }

      float m = -CUDART_INF_F, l = 0.f;
      const int t0 = place.t0, J = place.t1 - t0;
      int done = 0;  // of this tile in this segment
      bool far = false;   // a row of the warp has a maximum beyond 2^16
      bool seen = false;  // the block's scores were complete when the last one's weights were
      for (int j = PAIR ? 0 : x; j < J; j += PAIR ? 1 : 2, ++op, ++done) {
        const uint32_t b = block + uint32_t(j);
        const uint32_t buf = op & 1u, st = st0 + buf * TK;
        if (!seen && !(ok = tc::wait_warp(&sm.sfull[x][buf], (op >> 1) & 1u, wd))) break;
        tc::fence_after_sync();
        const int tok0 = (t0 + j) * TK;
        const float4* scl = sm.scale[b % SCALES];
        // -------- weights against the maximum so far; where a score is more than
        // LAG above it the maximum moves and they are computed again
        const bool edge = __any_sync(0xffffffffu, tok0 + TK > lim);
        uint32_t p[TK / 2];
        float sum;
        while (true) {
          const float off = OFF - (m == -CUDART_INF_F ? 0.f : m);
          float mx = -CUDART_INF_F;
          sum = 0.f;
          uint32_t s[2][32];
          tc::tmem_ld_x32(st, s[0]);
#pragma unroll
          for (int c = 0; c < TK / 32; ++c) {
            tc::tmem_wait_ld();
            if (c + 1 < TK / 32) tc::tmem_ld_x32(st + (c + 1) * 32, s[(c + 1) & 1]);
            uint32_t(&v)[32] = s[c & 1];
            if (edge)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (tok0 + c * 32 + e >= lim) v[e] = 0xFF800000u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 positions, of one page
              const float4 f = scl[2 * c + h];
              const float mul = fmaxf(fq * f.x, 1e-37f);
              // (a tree of maxima of three)
              float a[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                a[k] = fmaxf(fmaxf(as_f(v[16 * h + 4 * k]), as_f(v[16 * h + 4 * k + 1])),
                             fmaxf(as_f(v[16 * h + 4 * k + 2]), as_f(v[16 * h + 4 * k + 3])));
              mx = fmaxf(mx, fmaf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), mul, f.y));
              const uint64_t mul2 = f32x2(mul, mul), add2 = f32x2(f.y + off, f.y + off);
              uint64_t part[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                uint64_t t = u32x2(v[16 * h + 2 * e], v[16 * h + 2 * e + 1]);
                asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(t) : "l"(mul2), "l"(add2));
                const float x0 = exp2_approx(as_f(uint32_t(t)));
                const float x1 = exp2_approx(as_f(uint32_t(t >> 32)));
                const uint64_t y = f32x2(x0, x1);
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(part[e & 1]) : "l"(y));
                p[c * 16 + h * 8 + e] = f16x2(x0, x1);
              }
              asm("add.rn.f32x2 %0, %0, %1;" : "+l"(part[0]) : "l"(part[1]));
              sum = fmaf(as_f(uint32_t(part[0])) + as_f(uint32_t(part[0] >> 32)), f.z, sum);
            }
          }
          if (!__any_sync(0xffffffffu, moves(mx, m))) break;
          const float now = fmaxf(m, mx);
          const float al = now == m ? 1.f : exp2_approx(m - now);
          m = now;
          far = __any_sync(0xffffffffu, is_far(m));
          l *= al;
          if (done) {
            // the products that add to the result so far are complete
            if (!(ok = tc::wait_warp(&sm.odone[x][(op - 1) & 1u], ((op - 1) >> 1) & 1u, wd))) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tc::tmem_ld_x16(ot + q * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc::tmem_st_x16(ot + q * 16, o);
            }
          }
        }
        if (!ok) break;
        seen = j + (PAIR ? 1 : 2) < J &&
               tc::mbar_test(&sm.sfull[x][(op + 1) & 1u], ((op + 1) >> 1) & 1u);
        if (far)
          sum = far_weights(st, scl, fq, m, lim - tok0);
        else
          tc::tmem_st_x32(st, p);
        l += sum;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        // (a release: the block's scales have been read, and may be written over)
        if (lane == 0) tc::mbar_arrive(&sm.pfull[x][buf]);
        seen = __all_sync(0xffffffffu, seen);
      }
      if (!ok) break;
      if (done) {
        if (!(ok = tc::wait_warp(&sm.odone[x][(op - 1) & 1u], ((op - 1) >> 1) & 1u, wd))) break;
        tc::fence_after_sync();
      } else if (!PAIR) {
        if (!(ok = tc::wait_warp(&sm.idle, idles++ & 1u, wd))) break;
      }
      // -------- results
      const bool whole = place.t0 == 0 && place.t1 == it.tiles;
      const int64_t part = int64_t(blockIdx.x) * 2 + (first_seg ? 0 : 1);
      float w0 = 1.f, w1 = 0.f;
      bool both = false;
      if (!PAIR) {
        // tile 1's sums join tile 0's
        if (x == 1) {
          sm.m[row] = m, sm.l[row] = l;
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.mfull);
        } else {
          if (!(ok = tc::wait_warp(&sm.mfull, seg & 1u, wd))) break;
          tc::fence_after_sync();
          const float m1 = sm.m[row], l1 = sm.l[row], now = fmaxf(m, m1);
          both = J > 1;
          if (now != -CUDART_INF_F) {
            w0 = exp2_approx(m - now);
            w1 = exp2_approx(m1 - now);
            l = l * w0 + l1 * w1;
            m = now;
          }
        }
      }
      if (PAIR || x == 0) {
        const int prow = (PAIR ? x * 128 : 0) + row;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        TQ* dst = O + (int64_t(it.q0 + i) * ar.heads + it.h * ar.G + (rr - i * ar.G)) * D;
        float* pd = ar.parts + (part * ROWS + prow) * D;
        if (!whole) {
          __stcg(ar.part_ml + (part * ROWS + prow) * 2, m);
          __stcg(ar.part_ml + (part * ROWS + prow) * 2 + 1, l);
        }
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t a[16], b[16];
          tc::tmem_ld_x16(ot + q * 16, a);
          if (both) tc::tmem_ld_x16(ot + 128 + q * 16, b);
          tc::tmem_wait_ld();
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] = __uint_as_float(a[e]) * w0;
            if (both) v[e] = fmaf(__uint_as_float(b[e]), w1, v[e]);
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              __stcg(reinterpret_cast<float4*>(pd + q * 16 + e),
                     make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
          } else if (live) {
#pragma unroll
            for (int e0 = 0; e0 < 16; e0 += 8) {
              union {
                uint4 u;
                TQ e[8];
              } y;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if constexpr (std::is_same<TQ, __half>::value)
                  y.e[e] = __float2half_rn(v[e0 + e] * inv);
                else
                  y.e[e] = __float2bfloat16_rn(v[e0 + e] * inv);
              }
              *reinterpret_cast<uint4*>(dst + q * 16 + e0) = y.u;
            }
          }
        }
      }
      if (sm.nans != 0 && live && (PAIR || x == 0)) {
        // what the row does see of what its blocks left out, over the results
        const bool to_part = !whole;
        const int64_t prow = part * ROWS + (PAIR ? x * 128 : 0) + row;
        TQ* dst = O + (int64_t(it.q0 + i) * ar.heads + it.h * ar.G + (rr - i * ar.G)) * D;
        const int end = min(lim, place.t1 * TK);
#pragma unroll 1
        for (int p = max(t0, it.hidden / TK) * TK; p < end; ++p) {
          const int page = __ldg(bt.table + int64_t(it.b) * bt.width + (p >> c.tshift));
          if (page < 0 || page >= c.pages) continue;
          const int64_t blk = c.block(page, it.h);
          const bool all = !(__ldg(c.ks + blk) + __ldg(c.vs + blk) < CUDART_INF_F);
          const uint8_t* v = c.vq + ((blk << c.tshift) + (p & (T_ - 1))) * D;
          if (FMT != WQ_W8_E4M3 && !all) continue;
#pragma unroll 1
          for (int e0 = 0; e0 < D; e0 += 4) {
            const uint32_t b =
                all ? 0x80808080u : e4m3_nans(__ldg(reinterpret_cast<const uint32_t*>(v + e0)));
            if (b == 0) continue;
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              if (!(b >> (8 * e) & 0x80u)) continue;
              if (to_part)
                __stcg(ar.parts + prow * D + e0 + e, CUDART_NAN_F);
              else
                dst[e0 + e] = nan_of<TQ>();
            }
          }
        }
      }
      tc::fence_before_sync();
      if (!PAIR) {
        // tile 1's result, m and l have been read
        __syncwarp();
        if (x == 1)
          ok = tc::wait_warp(&sm.mfree, seg & 1u, wd);
        else if (lane == 0)
          tc::mbar_arrive(&sm.mfree);
        tc::fence_after_sync();
      }
      first_seg = false;
      block += J;
    }
    if (!ok) sm.abort_flag = 1;
  } else if (warp < 16) {
    // ------------------------------------------------------------- converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CONVERT));
    // a thread's pieces: 16 codes of rows tr, tr + STEP, ... of the block
    constexpr int PER = D / 16, STEP = 128 / PER, N = TK / STEP;  // N pieces of a block
    const bool values = warp >= 12;
    const uint8_t* src = values ? c.vq : c.kq;
    const uint32_t region = values ? vsm : ksm;
    uint64_t* const full = values ? sm.vfull : sm.kfull;
    uint64_t* const empty = values ? sm.vempty : sm.kempty;
    const int ct = int(threadIdx.x) & 127, piece = ct % PER, tr = ct / PER;
    // a piece is two 16-byte parts of a row of 64 f16; lanes of the upper
    // half planes store them in the other order (bank conflicts)
    const int plane = piece / 4, part0 = (piece & 3) * 2, swap = plane & 1;
    uint32_t block = 0;
    bool ok = true;
    for (; more && ok; more = step()) {
      const int t0 = place.t0, J = place.t1 - t0, len = it.len;
      // Lane g of a warp looks after positions 16 g to 16 g + 15 of a block (one
      // page): table entry two blocks ahead, address and (first warp) scales one
      // block ahead, so that nothing here waits for the load before it.
      auto entry = [&](int j) {
        const int tok = (t0 + j) * TK + lane * 16;
        return lane < TK / 16 && j < J && tok < len
                   ? __ldg(bt.table + int64_t(it.b) * bt.width + (tok >> c.tshift))
                   : -2;
      };
      auto from = [&](int page, int j) {  // of the group's first code, -1 where it has no page
        if (page < 0 || page >= c.pages) {
          if (page != -2) record_error(status, WQ_ERR_ARG);
          return int64_t(-1);
        }
        return ((c.block(page, it.h) << c.tshift) + (((t0 + j) * TK + lane * 16) & (T_ - 1))) * D;
      };
      auto load = [&](uint4 (&w)[N], int j, int64_t at, bool whole) {
        const uint8_t* mine = src + (tr & 15) * D + piece * 16;
        if (whole) {
          int64_t o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = __shfl_sync(0xffffffffu, at, (tr + i * STEP) >> 4);
#pragma unroll
          for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(mine + o[i]));
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int r = tr + i * STEP;
            const int64_t o = __shfl_sync(0xffffffffu, at, r >> 4);
            w[i] = make_uint4(0, 0, 0, 0);
            if (o >= 0 && (t0 + j) * TK + r < len)
              w[i] = __ldg(reinterpret_cast<const uint4*>(mine + o));
          }
        }
      };
      auto is_full = [&](int j, int64_t at) {
        return (t0 + j + 1) * TK <= len && __all_sync(0xffffffffu, lane >= TK / 16 || at >= 0);
      };
      auto store = [&](const uint4 (&w)[N], uint32_t dst) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = tr + i * STEP;
          uint32_t h[8];
          expand<FMT>(w[i].x, h[0], h[1]);
          expand<FMT>(w[i].y, h[2], h[3]);
          expand<FMT>(w[i].z, h[4], h[5]);
          expand<FMT>(w[i].w, h[6], h[7]);
          const uint32_t p0 = dst + plane * KVPLANE + r * 128 + ((part0 ^ (r & 7)) << 4);
          const uint32_t p1 = p0 ^ 16;
          if (swap) {
            sts128(p1, h[4], h[5], h[6], h[7]);
            sts128(p0, h[0], h[1], h[2], h[3]);
          } else {
            sts128(p0, h[0], h[1], h[2], h[3]);
            sts128(p1, h[4], h[5], h[6], h[7]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      };
      // the codes of two blocks are on their way (or a block's being expanded)
      uint4 w0[N], w1[N];
      float ks0 = 1.f, vs0 = -1.f, ks1 = 1.f, vs1 = -1.f;
      int next = entry(0);
      auto fetch = [&](uint4 (&w)[N], float& ks, float& vs, int j) {
        const int64_t at = from(next, j);
        next = entry(j + 1);
        ks = 1.f, vs = -1.f;
        if (warp == 8 && at >= 0) {
          const int64_t blk = (at / D) >> c.tshift;
          ks = __ldg(c.ks + blk), vs = __ldg(c.vs + blk);
        }
        if (j < J) load(w, j, at, is_full(j, at));
      };
      auto convert = [&](uint4 (&w)[N], float& ks, float& vs, int j) {
        const uint32_t s = block % STAGES;
        if (!(ok = tc::wait_warp(&empty[s], ((block / STAGES) & 1u) ^ 1u, wd))) return;
        const bool hides = (t0 + j + 1) * TK > it.hidden;  // some row does not see all of it
        if (warp == 8) {
          // A scale that is no number, or infinite, makes the rows that see it NaN: by its
          // logarithm here, or at the end where some rows do not see it.
          const float v = fmaxf(vs, 1e-30f);
          float lv = vs < 0.f ? -CUDART_INF_F : fmaf(ks, 0.f, __log2f(vs < 1e-30f ? 1e-30f : vs));
          float rv = vs < 0.f ? 0.f : __fdividef(1.f, v);
          if (hides && !(lv < CUDART_INF_F)) lv = -CUDART_INF_F, rv = 0.f, sm.nans = 1;
          if (lane < TK / 16)
            sm.scale[block % SCALES][lane] = make_float4(fmaxf(ks, 1e-30f), lv, rv, 0.f);
        }
        if (FMT == WQ_W8_E4M3 && values && hides) {
          uint32_t any = 0;
          auto clean = [&](uint32_t& x) {
            const uint32_t b = e4m3_nans(x);
            any |= b;
            x = without(x, b);
          };
#pragma unroll
          for (int i = 0; i < N; ++i) clean(w[i].x), clean(w[i].y), clean(w[i].z), clean(w[i].w);
          if (any) sm.nans = 1;
        }
        store(w, region + s * S::BLOCK);
        if (lane == 0) tc::mbar_arrive(&full[s]);
        ++block;
        fetch(w, ks, vs, j + 2);
      };
      fetch(w0, ks0, vs0, 0);
      fetch(w1, ks1, vs1, 1);
      for (int j = 0; j < J && ok; j += 2) {
        convert(w0, ks0, vs0, j);
        if (j + 1 < J && ok) convert(w1, ks1, vs1, j + 1);
      }
    }
    if (!ok) sm.abort_flag = 1;
  } else {
    // ------------------------------------------------------------- MMA issuer
    // (the whole warp walks the loop and one lane issues, so that operand
    // addresses stay in uniform registers)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
    constexpr uint32_t idesc_s = idesc_f16(TK, false), idesc_o = idesc_f16(D, true);
    // Each tile has a warp of its own.  A tile's rounds so far: scores issued,
    // weights taken.
    const int x = warp & 1;
    uint32_t block = 0, seg = 0, sc = 0, pv = 0;
    bool ok = warp < 18;
    for (; more && ok; more = step(), ++seg) {
      const int J = place.t1 - place.t0, N = PAIR ? J : (J + 1 - x) >> 1;
      ok = tc::wait_warp(&sm.qfull, seg & 1u, wd);
      if (!PAIR && N == 0 && lane == 0) tc::mbar_arrive(&sm.idle);
      tc::fence_after_sync();
      const uint64_t dq = tc::sdesc_k_sw128(qs + (PAIR ? x * S::TILE : 0));
      auto keys = [&](int i) {
        const uint32_t b = block + (PAIR ? i : 2 * i + x);
        return tc::wait_warp(&sm.kfull[b % STAGES], (b / STAGES) & 1u, wd);
      };
      auto scores = [&](int i) {
        const uint32_t b = block + (PAIR ? i : 2 * i + x), s = b % STAGES, buf = sc & 1u;
        tc::fence_after_sync();
        ++sc;
        const uint64_t dk = tc::sdesc_k_sw128(ksm + s * S::BLOCK);
        if (tc::elect_one()) {
#pragma unroll
          for (int term = 0; term < (TWO ? 2 : 1); ++term)
#pragma unroll
            for (int k16 = 0; k16 < D / 16; ++k16) {
              const uint32_t qat = ((k16 / 4) * PLANE + (k16 & 3) * 32) >> 4;
              const uint32_t kat = ((k16 / 4) * KVPLANE + (k16 & 3) * 32) >> 4;
              tc::mma_f16_ss(tmem + x * 128 + buf * TK, dq + uint64_t(term * (S::TILE >> 4) + qat),
                             dk + uint64_t(kat), idesc_s, (term | k16) != 0);
            }
          tc::mma_commit(&sm.sfull[x][buf]);
          tc::mma_commit(&sm.kempty[s]);
        }
        __syncwarp();
      };
      // the scores are two rounds ahead of their weights
      for (int i = 0; i < 2 && i < N && ok; ++i)
        if ((ok = keys(i))) scores(i);
      for (int i = 0; i < N && ok; ++i) {
        const uint32_t b = block + (PAIR ? i : 2 * i + x), s = b % STAGES, buf = pv & 1u;
        // (the weights last: what follows them is what the softmax waits for)
        if (!(ok = tc::wait_warp(&sm.vfull[s], (b / STAGES) & 1u, wd))) break;
        if (i + 2 < N && !(ok = keys(i + 2))) break;
        if (!(ok = tc::wait_warp(&sm.pfull[x][buf], (pv >> 1) & 1u, wd))) break;
        ++pv;
        tc::fence_after_sync();
        const uint64_t dv = sdesc_mn_sw128(vsm + s * S::BLOCK, KVPLANE);
        if (tc::elect_one()) {
#pragma unroll
          for (int k16 = 0; k16 < TK / 16; ++k16)
            tc::mma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + buf * TK + k16 * 8,
                           dv + uint64_t(k16 * 128), idesc_o, i > 0 || k16 != 0);
          tc::mma_commit(&sm.odone[x][buf]);
          tc::mma_commit(&sm.vempty[s]);
        }
        __syncwarp();
        if (i + 2 < N) scores(i + 2);
      }
      block += J;
    }
    if (!ok && warp < 18) sm.abort_flag = 1;
    if (warp < 18 && tc::elect_one()) {
      tc::mma_commit(&sm.drain[x]);
      tc::wait_until(&sm.drain[x], 0, tc::globaltimer_ns() + tc::kDrainNs);
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of cut items: blocks as in attn_kv8.cu, for each 8 rows.
template <typename TQ, int D, bool PAIR>
__global__ void __launch_bounds__(256, 5) attn_kv8_tc_join_kernel(TQ* __restrict__ O, TcArgs ar) {
  constexpr int ROWS = PAIR ? 256 : 128;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = 1 + int(blockIdx.x) / (ROWS / 8), oct = int(blockIdx.x) % (ROWS / 8);
  const Cut cut = ar.cuts[w];
  JoinShare js;
  if (cut.rows * int64_t(ROWS) + oct * 8 >= int64_t(cut.n) * ar.G || !join_share(w, cut, &js)) return;
  const int row = oct * 8 + js.row, rr = cut.rows * ROWS + row;
  float l, o[D / 32];
  if (!join_row<D>(js, cut, ROWS, row, ar.parts, ar.part_ml, &l, o) || rr >= cut.n * ar.G) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int i = rr / ar.G;
  TQ* dst = O + (int64_t(cut.q0 + i) * ar.heads + cut.h * ar.G + (rr - i * ar.G)) * D;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    if constexpr (std::is_same<TQ, __half>::value)
      dst[e * 32 + (threadIdx.x & 31)] = __float2half_rn(o[e] * inv);
    else
      dst[e * 32 + (threadIdx.x & 31)] = __float2bfloat16_rn(o[e] * inv);
  }
}

}  // namespace tcore
}  // namespace kv8
}  // namespace wq

namespace wq_host {

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct TcWs {
  size_t ml, cuts, bytes;
};
TcWs tc_ws(int64_t D, bool pair) {
  const size_t rows = pair ? 256 : 128, w2 = size_t(sm_count()) * 2;
  TcWs s;
  s.ml = up256(w2 * rows * size_t(D) * 4);
  s.cuts = s.ml + up256(w2 * rows * 8);
  s.bytes = s.cuts + w2 / 2 * sizeof(wq::kv8::Cut);
  return s;
}

template <typename TQ, int FMT, int D, bool PAIR>
int launch_tc(const void* Q, int64_t ldq, int64_t heads, const Kv8& a, int max_pos, float scale,
              void* out, uint8_t* ws, cudaStream_t s) {
  using namespace wq::kv8;
  using namespace wq::kv8::tcore;
  auto kern = attn_kv8_tc_kernel<TQ, FMT, D, PAIR>;
  constexpr size_t smem = Smem<D>::BYTES;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  WQ_CUDA_CHECK(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      WQ_CUDA_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
      if (dev < 64) done[dev] = true;
    }
  }
  constexpr int64_t ROWS = PAIR ? 256 : 128;
  int tshift = 0;
  while ((int64_t(1) << tshift) < a.page) ++tshift;
  const int G = int(heads / a.kv_heads);
  const int64_t most_r = (a.max_new * G + ROWS - 1) / ROWS;
  if (a.B * most_r > 0x7fffffff) return WQ_ERR_UNSUPPORTED;
  const Cache c{static_cast<uint8_t*>(a.kq), a.ks, static_cast<uint8_t*>(a.vq), a.vs, a.pages,
                int(a.kv_heads), tshift};
  const Batch bt{a.table, a.cu, a.lens, int(a.B), int(a.width), int(a.rows), int(a.max_new)};
  const Rope rp{a.cos, a.sin, int(a.rot), max_pos, a.interleaved};
  const TcWs w = tc_ws(D, PAIR);
  const TcArgs ar{ldq, int(heads), G, int(most_r), scale * 1.4426950408889634f,
                  reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + w.ml),
                  reinterpret_cast<Cut*>(ws + w.cuts)};
  const int grid = sm_count();
  TQ* o = static_cast<TQ*>(out);
  kern<<<grid, THREADS, smem, s>>>(static_cast<const TQ*>(Q), o, c, bt, rp, ar, status_ptr(),
                                   wait_limit_ns());
  WQ_LAUNCH_CHECK("attn_kv8_tc_kernel");
  if (grid < 2) return WQ_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((grid - 1) * (ROWS / 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  WQ_CUDA_CHECK(cudaLaunchKernelEx(&cfg, attn_kv8_tc_join_kernel<TQ, D, PAIR>, o, ar));
  return WQ_OK;
}

template <int FMT, int D>
int launch_tc_by_type(const void* Q, int dtype, int64_t ldq, int64_t heads, const Kv8& a,
                      int max_pos, float scale, void* out, uint8_t* ws, cudaStream_t s) {
  if (dtype == WQ_F16)
    return launch_tc<__half, FMT, D, false>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
  if (attn_kv8_pairs(dtype, heads, a.kv_heads, a.max_new))
    return launch_tc<__nv_bfloat16, FMT, D, true>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
  return launch_tc<__nv_bfloat16, FMT, D, false>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
}

}  // namespace

// Whether the tensor-memory kernel takes the call: more than 32 rows to a
// (sequence, kv head).  The other kernel reads the codes once for each 8 rows, this
// one once for 128 (its time hardly depends on the rows).  Measured, the other and
// this, over 4 x 32768 positions of 8 kv heads of 128: 16 rows 117 and 176 us, 24
// 163 and 176, 32 198 and 176, 40 235 and 176, 64 363 and 178; over 64 x 2048 32
// rows 206 and 215, 40 247 and 217; heads of 64, 32 rows 135 and 141, 40 165 and
// 141; over 4 x 1024 40 rows 29 and 33.  Heads of 256 are not built here: their results
// for two tiles do not fit in tensor memory beside the scores (for one they would).
bool attn_kv8_on_tc(int64_t heads, int64_t kv_heads, int64_t D, int64_t max_q) {
  return D <= 128 && max_q * (heads / kv_heads) > 32;
}
// Two row tiles that share the converted blocks: where there are two, and the queries
// are one term (160 rows over 4 x 32768: 223 us, and 336 one tile after the other; two
// terms of two tiles do not fit in shared memory beside four stages of blocks).
bool attn_kv8_pairs(int dtype, int64_t heads, int64_t kv_heads, int64_t max_q) {
  return dtype == WQ_BF16 && max_q * (heads / kv_heads) > 128;
}

size_t attn_kv8_tc_workspace_bytes(int64_t heads, int64_t kv_heads, int64_t D,
                                   int64_t max_q) {
  const int64_t rows = max_q * (heads / kv_heads);
  return tc_ws(D, rows > 128).bytes;  // (pairs of row tiles need the more)
}

int launch_attn_kv8_tc(const void* Q, int dtype, int64_t ldq, int64_t heads, const Kv8& a,
                       int max_pos, float scale, void* out, void* ws, cudaStream_t s) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool i8 = a.fmt == WQ_W8_INT8;
  if (a.D == 64)
    return i8 ? launch_tc_by_type<WQ_W8_INT8, 64>(Q, dtype, ldq, heads, a, max_pos, scale, out, w, s)
              : launch_tc_by_type<WQ_W8_E4M3, 64>(Q, dtype, ldq, heads, a, max_pos, scale, out, w, s);
  return i8 ? launch_tc_by_type<WQ_W8_INT8, 128>(Q, dtype, ldq, heads, a, max_pos, scale, out, w, s)
            : launch_tc_by_type<WQ_W8_E4M3, 128>(Q, dtype, ldq, heads, a, max_pos, scale, out, w, s);
}

}  // namespace wq_host
