// attn_kv8.cu -- causal attention over the paged 8-bit cache, few queries per
// sequence (decode, verification of drafts).
//
//   row (i, g) of kv head h: query i of the sequence, head h G + g, G = Hq / Hkv
//   s_j = scale (rope(q) . kq_j) ks(page of j),  j <= len - n + i
//   o   = sum_j softmax(s)_j vq_j vs(page of j)
//
// Bound by HBM up to 8 rows to a kv head: every code is read once per block of 8
// rows, 2 D bytes per position and head.  64 sequences of 277580 positions in all,
// 64 heads of 128 over 8 kv heads, one new token each (int8): 119 us with the
// join on inputs used over and over, 4.8 TB/s; 128 on new ones.
// Each further block of 8 rows reads the codes again (from L2, mostly) and expands
// them again: 40 us per 4 x 32768 positions and 8 kv heads.  A block walks over all
// positions of its sequence, those behind its last row's too (up to the call's rows).
//
// The codes go to f16 (exactly: int8 and E4M3 are subsets) and through mma.sync
// m16n8k16.  The scores' products have 16 rows for 8 queries: rows 0 to 7 hold the
// rotated query rounded to f16, rows 8 to 15 what that rounding left, so that the
// query counts with 22 bits at no cost.  A decode step needs about a third of the
// mma.sync rate while it streams at the copy rate, so tensor memory would add
// hand-offs and no speed.
//
// Work is cut into units of TK positions of one (sequence, head, row block),
// numbered with the position fastest, and every warp of the grid takes an equal
// run of them, whatever the sequences' lengths: no warp waits for another.  A
// segment (all units of a row block) counts two units more, for its queries and
// its result: a unit takes a warp 2.6 us in a full decode step, a segment's start
// and end about 5, and without that the warps that got many short sequences ended
// a quarter later than the rest.  A run's whole segments are written out directly;
// cut ones go to the workspace and attn_kv8_join_kernel adds them in a fixed order
// (10 us of those 119; its launch overlaps the end of the main kernel).
// (Units of 16 positions for heads of 128: 147 us where these took 131.)
//
// Softmax in one pass, in base 2, with the value scale folded into the
// exponent: t = s log2(e) + log2(vs), p' = 2^(t - m), so that p' is at most
// 2^LAG whatever the pages' scales; the sum takes p' / vs.  m and the sums are
// fp32, p' goes to the tensor cores as f16 (half a step 2^-11, against 2^-8
// of a bf16 result) with LAG + OFF = 14 binades above one and 24 + 14 below
// the row's maximum.
#include <math_constants.h>

#include <mutex>
#include <type_traits>

#include "kv8.cuh"

namespace wq {
namespace kv8 {

constexpr int MAX_WARPS = 12;
constexpr int RB = 8;      // rows per block
constexpr int START = 2;   // units that a segment's queries and result count

template <int D_>
struct Shape {
  static constexpr int D = D_;
  static constexpr int TK = D == 256 ? 16 : 32;    // positions per unit
  // a 256-wide head's sums need the registers of 8 warps per SM
  static constexpr int WARPS = D == 256 ? 8 : MAX_WARPS;
  static constexpr int STAGES = D == 128 ? 2 : 3;
  // rows of 128 bytes and more are kept as 16-byte pieces XORed with the row
  // (conflict-free fragment reads); 64-byte value rows are 80 bytes apart
  static constexpr int KP = D, VP = D == 64 ? 80 : D;
  static constexpr int KBYTES = TK * KP, VBYTES = TK * VP;
  static constexpr int STAGE = KBYTES + VBYTES + 32;  // + scales of up to two pages
  static constexpr int QP = 2 * D + 8;                // halves per staged query row
  static constexpr int WARP_BYTES = STAGES * STAGE + 4 * QP * 2;
};

__device__ __forceinline__ int swz(int D, int row, int piece) {
  return D == 64 ? piece : piece ^ (row & 7);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the same, or 16 zero bytes
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// Codes as f16 pairs, exactly.
// Keys: int8 as u = c + 128 in the subnormals (u 2^-24); the score of -128
//   ones is where a row's sum starts.  E4M3 through the hardware conversion.
// Values: int8 as 0x6400 | u, which is 1024 + u, minus 1152 (a bias of 128 per
//   weight would swamp a long sum whose values cancel).
template <int FMT>
struct Code;
template <>
struct Code<WQ_W8_INT8> {
  static constexpr float KEY = 16777216.f, BIAS = 128.f / 16777216.f;
  // codes 0, 1 (a) and 2, 3 (b) of a word of keys
  static __device__ __forceinline__ void key(uint32_t w, uint32_t& a, uint32_t& b) {
    const uint32_t x = w ^ 0x80808080u;
    a = __byte_perm(x, 0, 0x4140);
    b = __byte_perm(x, 0, 0x4342);
  }
  // codes 2 e and 2 e + 1 of two words of values, each as a pair
  static __device__ __forceinline__ void value(uint32_t w0, uint32_t w1, int e, uint32_t& a,
                                               uint32_t& b) {
    const uint32_t u = (__byte_perm(w0, w1, 0x4400 + 0x2222 * e) & 0x00FF00FFu) ^ 0x64806480u;
    const uint32_t v = (__byte_perm(w0, w1, 0x5511 + 0x2222 * e) & 0x00FF00FFu) ^ 0x64806480u;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(a) : "r"(u), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(b) : "r"(v), "r"(0x64806480u));
  }
};
template <>
struct Code<WQ_W8_E4M3> {
  static constexpr float KEY = 1.f, BIAS = 0.f;
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
  }
  static __device__ __forceinline__ void key(uint32_t w, uint32_t& a, uint32_t& b) {
    pairs(w, a, b);
  }
  static __device__ __forceinline__ void value(uint32_t w0, uint32_t w1, int e, uint32_t& a,
                                               uint32_t& b) {
    pairs(__byte_perm(w0, w1, 0x5140 + 0x2222 * e), a, b);
  }
};

// D (+)= A B, one warp: A 16 x 16, B 16 x 8, f16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Zeroes the NaN codes of a unit's staged values (at vb); whether there were any.  (Out
// of the loop: 4 x 5 drafts over 32768 in fp16 90.7 us, 91.2 as a part of it, 89.1
// without the check.)
template <int D>
__device__ __noinline__ bool zero_nans(uint32_t vb) {
  constexpr int PER = D / 16, STEP = 32 / PER;
  const int lane = threadIdx.x & 31;
  bool any = false;
#pragma unroll 1
  for (int r = lane / PER; r < Shape<D>::TK; r += STEP) {
    const uint32_t at = vb + r * Shape<D>::VP + swz(D, r, lane % PER) * 16;
    const uint4 v = lds128(at);
    const uint4 b = make_uint4(e4m3_nans(v.x), e4m3_nans(v.y), e4m3_nans(v.z), e4m3_nans(v.w));
    if (b.x | b.y | b.z | b.w) {
      any = true;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(without(v.x, b.x)),
                   "r"(without(v.y, b.y)), "r"(without(v.z, b.z)), "r"(without(v.w, b.w))
                   : "memory");
    }
  }
  any = __any_sync(0xffffffffu, any);
  __syncwarp();
  return any;
}

// A sequence as this kernel sees it, and a position in the numbering of units.
struct Cursor {
  int b, h, rb, tile;           // sequence, kv head, row block, unit of positions
  int n, q0, len, tiles, nrb;   // of sequence b
  int at;                       // unit of the run (a segment's first unit is its start)

  __device__ __forceinline__ void load(const Batch& bt, int tshift, int G, int TK, int* status) {
    n = seq_rows(bt, b, &q0, status);
    len = __ldg(bt.lens + b);
    const int64_t most = int64_t(bt.width) << tshift;
    if (len < 0 || len > most) {
      record_error(status, WQ_ERR_ARG);
      len = len < 0 ? 0 : int(most);
    }
    nrb = int((int64_t(n) * G + RB - 1) / RB);
    tiles = len > 0 ? (len + TK - 1) / TK : 1;
  }
  __device__ __forceinline__ int64_t units(int heads) const {
    return n > 0 ? int64_t(nrb) * heads * (tiles + START) : 0;
  }
};

struct Args {
  int64_t ldq;
  int heads, G;  // query heads, heads per kv head
  float scale_log2;
  float* parts;      // [2 W][RB][D]
  float* part_ml;    // [2 W][RB][2]
  Cut* cuts;         // [W] the segments that the runs' starts cut
};

template <typename TQ, int FMT, int D>
__global__ void __launch_bounds__(Shape<D>::WARPS * 32, 1)
    attn_kv8_kernel(const TQ* __restrict__ Q, TQ* __restrict__ O, Cache c, Batch bt, Rope rp,
                    Args ar, int* status) {
  using S = Shape<D>;
  constexpr int WARPS = S::WARPS, TK = S::TK, NT = TK / 8, MT = D / 16;
  constexpr int KS = D / 16;  // steps of the product over D
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t warp_sum[WARPS], start_at[WARPS], run_at[WARPS];
  __shared__ Cursor start_seq[WARPS];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int T_ = 1 << c.tshift;

  // ------------------------------------------------ which units are this warp's
  constexpr int NT_ = WARPS * 32;
  auto units_at = [&](Cursor& s, int b, int* st) {
    s.b = b;
    if (b >= bt.B) return int64_t(0);
    s.load(bt, c.tshift, ar.G, TK, st);
    return s.units(c.heads);
  };
  // (up to 384 sequences are looked at once)
  const bool one = bt.B <= NT_;
  Cursor mine;
  int64_t U = 0, part = 0, first = 0, units = 0;
  for (int b0 = 0; b0 < bt.B; b0 += NT_) {
    units = units_at(mine, b0 + int(threadIdx.x), status);
    first = U + block_scan<WARPS>(units, warp_sum, &part);
    U += part;
  }
  const Runs runs(U, int64_t(gridDim.x) * WARPS);
  if (threadIdx.x < WARPS) {
    const int id = int(threadIdx.x) * gridDim.x + blockIdx.x;
    run_at[threadIdx.x] = id < runs.workers ? runs.start(id) : -1;
  }
  __syncthreads();
  int64_t done = 0;
  for (int b0 = 0; b0 < bt.B; b0 += NT_) {
    if (!one) {
      units = units_at(mine, b0 + int(threadIdx.x), nullptr);
      first = done + block_scan<WARPS>(units, warp_sum, &part);
      done += part;
    }
    // the sequence that holds a warp's first unit
    if (units > 0)
      for (int w = 0; w < WARPS; ++w) {
        const int64_t u = run_at[w];
        if (u >= first && u < first + units) {
          start_seq[w] = mine;
          start_at[w] = u - first;
        }
      }
  }
  __syncthreads();
  const int id = warp * gridDim.x + blockIdx.x;
  if (id >= runs.workers) {
    if (lane == 0) write_cut(ar.cuts + id, false, runs, 0, 0, 0, 0, 0, 0, 0);
    return;
  }
  const int64_t u0 = run_at[warp];
  const int count = int(runs.start(id + 1) - u0);
  Cursor me = start_seq[warp];
  const int64_t at_seq = start_at[warp], seg = quotient(at_seq, me.tiles + START);
  const int64_t seg_begin = u0 - (at_seq - seg * (me.tiles + START));
  me.tile = int(u0 - seg_begin) - START;
  me.at = me.tile < 0 ? -me.tile : 0;  // units of the segment's start
  if (me.tile < 0) me.tile = 0;
  me.h = int(quotient(seg, me.nrb));
  me.rb = int(seg - int64_t(me.h) * me.nrb);
  const bool cuts = me.tile > 0;
  const int cut_tiles = me.tiles, cut_rb = me.rb, cut_n = me.n, cut_q0 = me.q0, cut_h = me.h;
  auto advance = [&](Cursor& s) {
    ++s.at;
    if (++s.tile < s.tiles) return;
    s.at += START;
    s.tile = 0;
    if (++s.rb < s.nrb) return;
    s.rb = 0;
    if (++s.h < c.heads) return;
    s.h = 0;
    do {
      ++s.b;
      if (s.b >= bt.B) return;
      s.load(bt, c.tshift, ar.G, TK, nullptr);
    } while (s.n == 0);
  };

  uint8_t* wbase = smem + size_t(warp) * S::WARP_BYTES;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(wbase));
  __half* qs = reinterpret_cast<__half*>(wbase + S::STAGES * S::STAGE);
  const uint32_t qbase = base + S::STAGES * S::STAGE;

  // ------------------------------------------------ the copies, a few units ahead
  Cursor ahead = me;
  int issued = 0;
  int pg0 = -1, pg1 = -1;  // the pages of the unit to be copied next
  auto pages_of = [&](const Cursor& s) {
    const int col = (s.tile * TK) >> c.tshift;
    const int* row = bt.table + int64_t(s.b) * bt.width + col;
    pg0 = (col << c.tshift) < s.len ? __ldg(row) : -1;
    pg1 = T_ < TK && ((col + 1) << c.tshift) < s.len ? __ldg(row + 1) : -1;
  };
  pages_of(ahead);
  // a unit's keys (and scales) are requested as soon as the buffer's last ones
  // have been used, its values when those have: STAGES units on their way
  constexpr int PER = D / 16, STEP = 32 / PER, COPIES = TK / STEP;
  const int copy_row = lane / PER, piece = lane % PER;
  int64_t from0 = 0, from1 = 0;  // of the unit whose keys were requested last
  int rows = 0;
  bool ok0 = false, ok1 = false, live = false;
  // rows are contiguous in a page, so a lane's pieces are 512 bytes apart
  auto request = [&](const uint8_t* src, uint32_t dst, int pitch) {
    if (live) {
      if (T_ >= TK && ok0 && rows >= TK) {
        const uint8_t* p = src + from0;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int r = copy_row + i * STEP;
          cp16(dst + r * pitch + swz(D, r, piece) * 16, p + i * 512);
        }
      } else {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int r = copy_row + i * STEP;
          const bool second = T_ < TK && i >= COPIES / 2;
          cp16z(dst + r * pitch + swz(D, r, piece) * 16, src + (second ? from1 : from0) + i * 512,
                r < rows && (second ? ok1 : ok0));
        }
      }
    }
    cp_commit();
  };
  auto request_keys = [&]() {
    live = ahead.at < count;
    const uint32_t st = base + uint32_t(issued % S::STAGES) * S::STAGE;
    if (live) {
      const int tok0 = ahead.tile * TK, col = tok0 >> c.tshift;
      ok0 = pg0 >= 0 && pg0 < c.pages, ok1 = pg1 >= 0 && pg1 < c.pages;
      rows = ahead.len - tok0;
      if (lane < 2 && (lane == 0 || T_ < TK)) {
        const bool ok = lane ? ok1 : ok0, used = ((col + lane) << c.tshift) < ahead.len;
        const uint32_t sc = st + S::KBYTES + S::VBYTES + 8 * lane;
        if (ok) {
          const int64_t at = c.block(lane ? pg1 : pg0, ahead.h);
          cp4(sc, c.ks + at);
          cp4(sc + 4, c.vs + at);
        } else {
          // no page: its positions are masked
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sc), "f"(0.f), "f"(-1.f)
                       : "memory");
          if (used) record_error(status, WQ_ERR_ARG);
        }
      }
      from0 = ((c.block(ok0 ? pg0 : 0, ahead.h) << c.tshift) + (tok0 & (T_ - 1))) * D + lane * 16;
      from1 = T_ < TK ? (c.block(ok1 ? pg1 : 0, ahead.h) << c.tshift) * D + lane * 16 - 16 * D : from0;
      advance(ahead);
      if (ahead.at < count) pages_of(ahead);
    }
    request(c.kq, st, S::KP);
  };
  auto request_values = [&]() {
    request(c.vq, base + uint32_t(issued % S::STAGES) * S::STAGE + S::KBYTES, S::VP);
    ++issued;
  };
#pragma unroll
  for (int i = 0; i < S::STAGES; ++i) {
    request_keys();
    request_values();
  }
  if (lane == 0)
    write_cut(ar.cuts + id, cuts, runs, seg_begin, START, cut_tiles, cut_rb, cut_n, cut_q0, cut_h);

  uint32_t qa[KS][4];
  float acc[MT][4];
  float m = -CUDART_INF_F, l = 0.f, fq = 0.f, start = 0.f;
  int lim = 0;
  bool fresh = true, first_seg = true;
  bool nans = false;  // values that are no number where the segment's rows differ in what they see
  int seg_tile0 = me.tile;
  // the first unit with positions that not every row of the block sees
  int hides = 0;
  // the first unit that no row of the block sees any of.  Prompts with heads of 256 walk over
  // many, and would look for NaN codes in them: 2 x 1024 queries of 8 heads over 2 kv heads
  // behind 1024 positions 370 us, 423 without the test (int8, which has no such codes, 430,
  // and 410 without; other calls have 32 rows at most, and so a few such positions)
  int over = 0;

  for (int u = 0; me.at < count; ++u) {
    if (fresh) {
      // -------------------------------------------- a segment's queries
      fresh = false;
      seg_tile0 = me.tile;
      hides = max(0, me.len - me.n + (me.rb * RB) / ar.G + 1) / TK;
      if (D == 256 && FMT == WQ_W8_E4M3) {
        const int last = min(me.n - 1, (me.rb * RB + RB - 1) / ar.G);
        over = (max(0, min(me.len, me.len - me.n + last + 1)) + TK - 1) / TK;
      }
      // P lanes per row, 32 / P rows at a time; rows are loaded together (all
      // eight, or four of 256 elements) and staged four at a time
      constexpr int P = D / 8, RPP = 32 / P, ITER = RB / RPP, HALF = ITER / 2;
      constexpr int LOADS = ITER > 4 ? HALF : ITER;
      const int d = (lane % P) * 8;
      float x[LOADS][8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          if (half == 1 && LOADS == ITER) break;
          const int rr = me.rb * RB + (half * HALF + k) * RPP + lane / P;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
          if (rr < me.n * ar.G) {
            const int i = rr / ar.G;
            int pos = me.len - me.n + i;
            Rope rq = rp;
            if (pos < 0 || (rq.cos != nullptr && pos >= rq.max_pos)) {
              // (a row before the sequence's start sees no key)
              if (pos >= 0) record_error(status, WQ_ERR_ARG);
              rq.cos = nullptr;
            }
            const TQ* row = Q + int64_t(me.q0 + i) * ar.ldq +
                            int64_t(me.h * ar.G + (rr - i * ar.G)) * D;
            rotated8(row, d, pos, rq, x[k]);
          }
        }
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
          const int k = LOADS == ITER ? half * HALF + j : j;
          float a = 0.f, sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[k][e]));
#pragma unroll
          for (int o = P / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          // a power of two brings the row's largest element to [2^14, 2^15)
          int ex = (a > 0.f && a <= 3.4028234663852886e38f)
                       ? 141 - int(__float_as_uint(a) >> 23)
                       : 0;
          ex = ex > 100 ? 100 : ex;
          const float up = __uint_as_float(uint32_t(127 + ex) << 23);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[k][e] *= up;
            sum += x[k][e];
          }
#pragma unroll
          for (int o = P / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          // rounded to f16, and what that left: word e of both side by side
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(x[k][2 * e], x[k][2 * e + 1]);
            const float2 f = __half22float2(h);
            hi[e] = *reinterpret_cast<const uint32_t*>(&h);
            lo[e] = f16x2(x[k][2 * e] - f.x, x[k][2 * e + 1] - f.y);
          }
          __half* dst = qs + (j * RPP + lane / P) * S::QP;
          *reinterpret_cast<uint4*>(dst + 2 * d) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
          *reinterpret_cast<uint4*>(dst + 2 * d + 8) = make_uint4(hi[2], hi[3], lo[2], lo[3]);
          if (lane % P == 0)
            *reinterpret_cast<float2*>(dst + 2 * D) =
                make_float2(__uint_as_float(uint32_t(127 - ex) << 23), sum);
        }
        __syncwarp();
        if (g >> 2 == half) {
          const uint32_t row = qbase + uint32_t((g & 3) * S::QP) * 2;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int j = ks >> 2, w = ks & 3;
            const int pc = D == 64 ? t : 2 * t + (j & 1) + 8 * (j >> 1);
            const uint4 v = lds128(row + uint32_t(2 * (pc * 16 + w * 4)) * 2);
            qa[ks][0] = v.x;
            qa[ks][1] = v.z;
            qa[ks][2] = v.y;
            qa[ks][3] = v.w;
          }
          fq = lds32f(row + 4 * D) * ar.scale_log2 * Code<FMT>::KEY;
          start = -Code<FMT>::BIAS * lds32f(row + 4 * D + 4);
        }
        __syncwarp();
      }
      const int rr = me.rb * RB + g;
      lim = rr < me.n * ar.G ? min(me.len, me.len - me.n + rr / ar.G + 1) : 0;
      m = -CUDART_INF_F;
      l = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
    }
    cp_wait<2 * S::STAGES - 1>();
    __syncwarp();
    const uint32_t st = base + uint32_t(u % S::STAGES) * S::STAGE;
    const uint32_t vb = st + S::KBYTES, scb = vb + S::VBYTES;

    // (the unit's second page, where it has two, is that of the upper half)
    auto page_scales = [&](int k, float& f, float& lv, float& rv) {
      const float ks = lds32f(scb + 8 * k), vs = lds32f(scb + 8 * k + 4);
      const float v = fmaxf(vs, 1e-30f);
      f = fq * ks;
      lv = vs < 0.f ? -CUDART_INF_F : __log2f(vs < 1e-30f ? 1e-30f : vs);  // (NaN stays)
      rv = __fdividef(1.f, v);
    };
    const bool unseen = D == 256 && FMT == WQ_W8_E4M3 && me.tile >= over;
    float f0, lv0, rv0, f1, lv1, rv1;
    float sc[NT][4];
    if (!unseen) {
      page_scales(0, f0, lv0, rv0);
      f1 = f0, lv1 = lv0, rv1 = rv0;
      if (T_ < TK) page_scales(1, f1, lv1, rv1);

      // -------------------------------------------------- scores
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[nt][0] = sc[nt][1] = start;
        sc[nt][2] = sc[nt][3] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const int pc = D == 64 ? t : 2 * t + (j & 1) + 8 * (j >> 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = nt * 8 + g;
          const uint4 k4 = lds128(st + r * S::KP + swz(D, r, pc) * 16);
          const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t b0, b1;
            Code<FMT>::key(kw[w], b0, b1);
            const int ks = j * 4 + w;
            mma16816(sc[nt], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
          }
        }
      }
    }

    __syncwarp();
    request_keys();

    // -------------------------------------------------- softmax, base 2
    uint32_t pb[NT];
    if (!unseen) {
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool hi = NT == 4 && nt >= 2;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sc[nt][e] = fmaf(sc[nt][e] + sc[nt][2 + e], hi ? f1 : f0, hi ? lv1 : lv0);
      }
      if (__any_sync(0xffffffffu, (me.tile + 1) * TK > lim)) {
        const int left = lim - me.tile * TK - 2 * t;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (nt * 8 + e >= left) sc[nt][e] = -CUDART_INF_F;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(sc[nt][0], sc[nt][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, moves(mx, m))) {
        const float now = fmaxf(m, mx);
        const float al = now == m ? 1.f : exp2_approx(m - now);
        m = now;
        l *= al;
        const float a0 = __shfl_sync(0xffffffffu, al, t * 8);
        const float a1 = __shfl_sync(0xffffffffu, al, t * 8 + 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][0] *= a0;
          acc[mt][1] *= a1;
          acc[mt][2] *= a0;
          acc[mt][3] *= a1;
        }
      }
      {
        const float off = OFF - (m == -CUDART_INF_F ? 0.f : m);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float a = exp2_approx(sc[nt][0] + off), b = exp2_approx(sc[nt][1] + off);
          if (NT == 4 && nt >= 2)
            s1 += a + b;
          else
            s0 += a + b;
          pb[nt] = f16x2(a, b);
        }
        l += s0 * rv0 + s1 * rv1;
      }
    }

    // -------------------------------------------------- values
    cp_wait<2 * S::STAGES - 1>();
    __syncwarp();
    if (!unseen) {
      if (FMT == WQ_W8_E4M3 && me.tile >= hides) nans |= zero_nans<D>(vb);
#pragma unroll
      for (int ks = 0; ks < TK / 16; ++ks) {
        const int r = ks * 16 + 2 * t;
        constexpr int WORDS = D == 64 ? 2 : 4;
#pragma unroll
        for (int q = 0; q < (D == 64 ? 1 : D / 128); ++q) {
          uint32_t w[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // positions r, r + 1, r + 8, r + 9
            const int row = r + (k & 1) + 8 * (k >> 1);
            if (D == 64) {
              const uint2 x = lds64(vb + row * S::VP + g * 8);
              w[k][0] = x.x, w[k][1] = x.y;
            } else {
              const uint4 x = lds128(vb + row * S::VP + swz(D, row, g + 8 * q) * 16);
              w[k][0] = x.x, w[k][1] = x.y, w[k][2] = x.z, w[k][3] = x.w;
            }
          }
#pragma unroll
          for (int k = 0; k < 2 * WORDS; ++k) {
            uint32_t a0, a1, a2, a3;
            Code<FMT>::value(w[0][k >> 1], w[1][k >> 1], k & 1, a0, a1);
            Code<FMT>::value(w[2][k >> 1], w[3][k >> 1], k & 1, a2, a3);
            mma16816(acc[q * 8 + k], a0, a1, a2, a3, pb[2 * ks], pb[2 * ks + 1]);
          }
        }
      }
    }

    __syncwarp();
    request_values();

    // -------------------------------------------------- end of a segment
    const bool last = me.tile + 1 == me.tiles || me.at + 1 >= count;
    if (last) {
      const bool whole = seg_tile0 == 0 && me.tile + 1 == me.tiles;
      const int64_t part = int64_t(id) * 2 + (first_seg ? 0 : 1);
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (!whole && t == 0) {
        float* ml = ar.part_ml + (part * RB + g) * 2;
        __stcg(ml, m);
        __stcg(ml + 1, l);
      }
      if (FMT == WQ_W8_E4M3 && nans) {
        const int lim0 = __shfl_sync(0xffffffffu, lim, t * 8);
        const int lim1 = __shfl_sync(0xffffffffu, lim, t * 8 + 4);
        const int end = min(me.len, (me.tile + 1) * TK);
#pragma unroll 1
        for (int p = max(seg_tile0, hides) * TK; p < end; ++p) {
          const int page = __ldg(bt.table + int64_t(me.b) * bt.width + (p >> c.tshift));
          if (page < 0 || page >= c.pages) continue;
          const uint8_t* v =
              c.vq + ((c.block(page, me.h) << c.tshift) + (p & (T_ - 1))) * D;
          constexpr int RUN = D == 64 ? 8 : 16;  // consecutive elements of this lane
#pragma unroll
          for (int k = 0; k < D / 8; k += 4) {
            const uint32_t b = e4m3_nans(
                __ldg(reinterpret_cast<const uint32_t*>(v + (k / RUN) * 128 + g * RUN + k % RUN)));
            if (b == 0) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (b >> (8 * e) & 0x80u) {
                if (p < lim0) acc[(k + e) / 2][2 * (e & 1)] = CUDART_NAN_F;
                if (p < lim1) acc[(k + e) / 2][1 + 2 * (e & 1)] = CUDART_NAN_F;
              }
          }
        }
        nans = false;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = 2 * t + q;
        const float iv = __shfl_sync(0xffffffffu, inv, t * 8 + 4 * q);
        const int rr = me.rb * RB + r;
        constexpr int RUN = D == 64 ? 8 : 16;  // consecutive elements of this lane
        if (!whole) {
#pragma unroll
          for (int k = 0; k < D / 8; k += 4) {
            float* dst = ar.parts + (part * RB + r) * D + (k / RUN) * 128 + g * RUN + k % RUN;
            __stcg(reinterpret_cast<float4*>(dst),
                   make_float4(acc[k / 2][q], acc[k / 2][q + 2], acc[k / 2 + 1][q],
                               acc[k / 2 + 1][q + 2]));
          }
        } else if (rr < me.n * ar.G) {
          const int i = rr / ar.G;
          TQ* o = O + (int64_t(me.q0 + i) * ar.heads + me.h * ar.G + (rr - i * ar.G)) * D;
#pragma unroll
          for (int k = 0; k < D / 8; k += 8) {
            union {
              uint4 v;
              TQ e[8];
            } y;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float v = acc[(k + e) / 2][q + 2 * (e & 1)] * iv;
              if constexpr (std::is_same<TQ, __half>::value)
                y.e[e] = __float2half_rn(v);
              else
                y.e[e] = __float2bfloat16_rn(v);
            }
            *reinterpret_cast<uint4*>(o + (k / RUN) * 128 + g * RUN + k % RUN) = y.v;
          }
        }
      }
      fresh = true;
      first_seg = false;
    }
    advance(me);
  }
  cp_wait<0>();
}

// Joins the parts of cut segments: a block of 8 warps for each start of a run, one
// row of the segment per warp, or more warps to a row where it has many parts.
template <typename TQ, int D>
__global__ void __launch_bounds__(256, 5)
    attn_kv8_join_kernel(TQ* __restrict__ O, Args ar) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = 1 + int(blockIdx.x);
  const Cut cut = ar.cuts[w];
  JoinShare js;
  if (!join_share(w, cut, &js)) return;
  float l, o[D / 32];
  if (!join_row<D>(js, cut, RB, js.row, ar.parts, ar.part_ml, &l, o)) return;
  const int rr = cut.rows * RB + js.row;
  if (rr >= cut.n * ar.G) return;
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

}  // namespace kv8
}  // namespace wq

namespace wq_host {

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct Ws {
  size_t ml, cuts, bytes;
};
Ws attn_ws(int64_t D) {
  const size_t w2 = size_t(sm_count()) * wq::kv8::MAX_WARPS * 2, rb = size_t(wq::kv8::RB);
  Ws s;
  s.ml = up256(w2 * rb * size_t(D) * 4);
  s.cuts = s.ml + up256(w2 * rb * 8);
  s.bytes = s.cuts + w2 / 2 * sizeof(wq::kv8::Cut);
  return s;
}

template <typename TQ, int FMT, int D>
int launch_decode(const void* Q, int64_t ldq, int64_t heads, const Kv8& a, int max_pos, float scale,
                  void* out, uint8_t* ws, cudaStream_t s) {
  using namespace wq::kv8;
  auto kern = attn_kv8_kernel<TQ, FMT, D>;
  constexpr int WARPS = Shape<D>::WARPS;
  constexpr size_t smem = size_t(WARPS) * Shape<D>::WARP_BYTES;
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
  int tshift = 0;
  while ((int64_t(1) << tshift) < a.page) ++tshift;
  const int G = int(heads / a.kv_heads);
  const Cache c{static_cast<uint8_t*>(a.kq), a.ks, static_cast<uint8_t*>(a.vq), a.vs, a.pages,
                int(a.kv_heads), tshift};
  const Batch bt{a.table, a.cu, a.lens, int(a.B), int(a.width), int(a.rows), int(a.max_new)};
  const Rope rp{a.cos, a.sin, int(a.rot), max_pos, a.interleaved};
  const Ws w = attn_ws(D);
  const Args ar{ldq, int(heads), G, scale * 1.4426950408889634f, reinterpret_cast<float*>(ws),
                reinterpret_cast<float*>(ws + w.ml), reinterpret_cast<Cut*>(ws + w.cuts)};
  const int grid = sm_count();
  TQ* o = static_cast<TQ*>(out);
  kern<<<grid, WARPS * 32, smem, s>>>(static_cast<const TQ*>(Q), o, c, bt, rp, ar, status_ptr());
  WQ_LAUNCH_CHECK("attn_kv8_kernel");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid * WARPS - 1));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  WQ_CUDA_CHECK(cudaLaunchKernelEx(&cfg, attn_kv8_join_kernel<TQ, D>, o, ar));
  return WQ_OK;
}

template <typename TQ, int FMT>
int launch_by_shape(const void* Q, int64_t ldq, int64_t heads, const Kv8& a, int max_pos,
                    float scale, void* out, uint8_t* ws, cudaStream_t s) {
  if (a.D == 64) return launch_decode<TQ, FMT, 64>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
  if (a.D == 128) return launch_decode<TQ, FMT, 128>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
  return launch_decode<TQ, FMT, 256>(Q, ldq, heads, a, max_pos, scale, out, ws, s);
}

}  // namespace

size_t attn_kv8_workspace_bytes(int64_t heads, int64_t kv_heads, int64_t D, int64_t max_q) {
  if (attn_kv8_on_tc(heads, kv_heads, D, max_q))
    return attn_kv8_tc_workspace_bytes(heads, kv_heads, D, max_q);
  return attn_ws(D).bytes;
}

int launch_attn_kv8(const void* Q, int dtype, int64_t ldq, int64_t heads, const Kv8& a,
                    int max_pos, float scale, void* out, void* ws, cudaStream_t s) {
  if (attn_kv8_on_tc(heads, a.kv_heads, a.D, a.max_new))
    return launch_attn_kv8_tc(Q, dtype, ldq, heads, a, max_pos, scale, out, ws, s);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool i8 = a.fmt == WQ_W8_INT8;
  if (dtype == WQ_BF16)
    return i8 ? launch_by_shape<__nv_bfloat16, WQ_W8_INT8>(Q, ldq, heads, a, max_pos, scale, out, w, s)
              : launch_by_shape<__nv_bfloat16, WQ_W8_E4M3>(Q, ldq, heads, a, max_pos, scale, out, w, s);
  return i8 ? launch_by_shape<__half, WQ_W8_INT8>(Q, ldq, heads, a, max_pos, scale, out, w, s)
            : launch_by_shape<__half, WQ_W8_E4M3>(Q, ldq, heads, a, max_pos, scale, out, w, s);
}

}  // namespace wq_host
