// attn_kv8.cu -- causal attention over the paged 8-bit cache, few queries per
// sequence (decode, verification of drafts).
//
//   row (i, g) of kv head h: query i of the sequence, head h G + g, G = Hq / Hkv
//   s_j = scale (rope(q) . kq_j) ks(page of j),  j <= len - n + i
//   o   = sum_j softmax(s)_j vq_j vs(page of j)
//
// Bound by HBM: every code is read once per block of RB rows (8 or 16), 2 D
// bytes per position and head.  The codes go to f16 (exactly: int8 and E4M3
// are subsets) and through mma.sync m16n8k16; at one row block per code byte
// that needs about a tenth of the rate that the memory can feed, so the
// tensor memory's hand-offs would only add latency here.
//
// Work is cut into units of TK positions of one (sequence, head, row block),
// numbered with the position fastest, and every warp of the grid takes an
// equal run of them, whatever the sequences' lengths: no warp waits for
// another.  A run's whole segments are written out directly; cut ones go to
// the workspace and attn_kv8_join_kernel adds them in a fixed order.
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

constexpr int WARPS = 8;
constexpr float LAG = 8.f;  // how far the maximum may grow before the sums are rescaled
constexpr float OFF = 6.f;

template <int D_>
struct Shape {
  static constexpr int D = D_;
  static constexpr int TK = D == 256 ? 16 : 32;    // positions per unit
  static constexpr int STAGES = D == 64 ? 5 : 3;
  // rows of 128 bytes and more are kept as 16-byte pieces XORed with the row
  // (conflict-free fragment reads); 64-byte value rows are 80 bytes apart
  static constexpr int KP = D, VP = D == 64 ? 80 : D;
  static constexpr int KBYTES = TK * KP, VBYTES = TK * VP;
  static constexpr int STAGE = KBYTES + VBYTES + 32;  // + scales of up to two pages
  static constexpr int QP = D + 8;                    // halves per staged query row
  static constexpr int WARP_BYTES = STAGES * STAGE + 8 * QP * 2;
};

__device__ __forceinline__ int swz(int D, int row, int piece) {
  return D == 64 ? piece : piece ^ (row & 7);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Codes as f16 pairs.  int8: the byte with its top bit flipped is u = c + 128;
// 0x6400 | u is 1024 + u in f16, minus 1152 gives c.  E4M3: sign, then exponent
// and mantissa one bit lower, is c 2^-8 in f16 (subnormals too); the 2^8 is in
// the caller's scale.  Every byte gives a finite value, so that slots nobody
// wrote cannot reach a result through their zero weights.
template <int FMT>
struct Code {
  static constexpr float SCALE = FMT == WQ_W8_INT8 ? 1.f : 256.f;
  // the halves of t hold a code in both of their bytes
  static __device__ __forceinline__ uint32_t halves(uint32_t t) {
    if (FMT == WQ_W8_INT8) {
      const uint32_t u = (t & 0x00FF00FFu) ^ 0x64806480u;
      uint32_t r;
      asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
      return r;
    }
    return (t & 0x80008000u) | ((t >> 1) & 0x3F803F80u);
  }
  // codes 0, 1 (a) and 2, 3 (b) of a word
  static __device__ __forceinline__ void word(uint32_t w, uint32_t& a, uint32_t& b) {
    a = halves(__byte_perm(w, 0, 0x1100));
    b = halves(__byte_perm(w, 0, 0x3322));
  }
  // code e of two words
  static __device__ __forceinline__ uint32_t cross(uint32_t w0, uint32_t w1, int e) {
    return halves(__byte_perm(w0, w1, 0x4400 + 0x1111 * e));
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

// A sequence as this kernel sees it, and a position in the numbering of units.
struct Cursor {
  int b, h, rb, tile;           // sequence, kv head, row block, unit of positions
  int n, q0, len, tiles, nrb;   // of sequence b

  __device__ __forceinline__ void load(const Batch& bt, int tshift, int G, int RB, int TK,
                                       int* status) {
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
    return n > 0 ? int64_t(nrb) * heads * tiles : 0;
  }
};

struct Args {
  int64_t ldq;
  int heads, G;  // query heads, heads per kv head
  float scale_log2;
  float* parts;      // [2 W][RB][D]
  float* part_ml;    // [2 W][RB][2]
  int64_t* prefix;   // [B + 1] first unit of each sequence
};

template <typename TQ, int FMT, int D, int NB>
__global__ void __launch_bounds__(WARPS * 32, 1)
    attn_kv8_kernel(const TQ* __restrict__ Q, TQ* __restrict__ O, Cache c, Batch bt, Rope rp,
                    Args ar, int* status) {
  using S = Shape<D>;
  constexpr int RB = 8 * NB, TK = S::TK, NT = TK / 8, MT = D / 16;
  constexpr int KS = D / 16;  // steps of the product over D
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t warp_sum[WARPS], start_at[WARPS], run_at[WARPS];
  __shared__ int start_b[WARPS];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int T_ = 1 << c.tshift;

  // ------------------------------------------------ which units are this warp's
  Cursor me;
  int64_t U = 0, u0 = 0, u1 = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t run = 0;
    for (int b0 = 0; b0 < bt.B; b0 += WARPS * 32) {
      Cursor s;
      s.b = b0 + int(threadIdx.x);
      int64_t mine = 0;
      if (s.b < bt.B) {
        s.load(bt, c.tshift, ar.G, RB, TK, pass ? nullptr : status);
        mine = s.units(c.heads);
      }
      int64_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      int64_t before = run;
      for (int w = 0; w < warp; ++w) before += warp_sum[w];
      for (int w = 0; w < WARPS; ++w) run += warp_sum[w];
      const int64_t first = before + inc - mine;
      if (pass == 1) {
        // the sequence that holds a warp's first unit
        for (int w = 0; w < WARPS; ++w) {
          const int64_t u = run_at[w];
          if (mine > 0 && u >= first && u < first + mine) {
            start_b[w] = s.b;
            start_at[w] = u - first;
          }
        }
        if (blockIdx.x == 0 && s.b < bt.B) {
          ar.prefix[s.b] = first;
          if (s.b == bt.B - 1) ar.prefix[bt.B] = U;
        }
      }
      __syncthreads();
    }
    U = run;
    if (pass == 0 && threadIdx.x < WARPS) {
      const int64_t W = workers(U, int64_t(gridDim.x) * WARPS);
      const int64_t id = int64_t(threadIdx.x) * gridDim.x + blockIdx.x;
      run_at[threadIdx.x] = id < W ? run_start(id, U, W) : -1;
    }
    __syncthreads();
    if (U == 0 && pass == 0) {
      if (blockIdx.x == 0)
        for (int b = int(threadIdx.x); b <= bt.B; b += WARPS * 32) ar.prefix[b] = 0;
      return;
    }
  }
  const int64_t W = workers(U, int64_t(gridDim.x) * WARPS);
  const int64_t id = int64_t(warp) * gridDim.x + blockIdx.x;
  if (id >= W) return;
  u0 = run_start(id, U, W);
  u1 = run_start(id + 1, U, W);
  me.b = start_b[warp];
  me.load(bt, c.tshift, ar.G, RB, TK, nullptr);
  {
    const int64_t at = start_at[warp];
    me.tile = int(at % me.tiles);
    const int64_t seg = at / me.tiles;
    me.rb = int(seg % me.nrb);
    me.h = int(seg / me.nrb);
  }
  auto advance = [&](Cursor& s) {
    if (++s.tile < s.tiles) return;
    s.tile = 0;
    if (++s.rb < s.nrb) return;
    s.rb = 0;
    if (++s.h < c.heads) return;
    s.h = 0;
    do {
      ++s.b;
      if (s.b >= bt.B) return;
      s.load(bt, c.tshift, ar.G, RB, TK, nullptr);
    } while (s.n == 0);
  };

  uint8_t* wbase = smem + size_t(warp) * S::WARP_BYTES;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(wbase));
  __half* qs = reinterpret_cast<__half*>(wbase + S::STAGES * S::STAGE);
  const uint32_t qbase = base + S::STAGES * S::STAGE;

  // ------------------------------------------------ the copies, a few units ahead
  Cursor ahead = me;
  int64_t issued = u0;
  int pg0 = -1, pg1 = -1;  // the pages of the unit to be copied next
  auto pages_of = [&](const Cursor& s) {
    const int col = (s.tile * TK) >> c.tshift;
    const int* row = bt.table + int64_t(s.b) * bt.width + col;
    pg0 = (col << c.tshift) < s.len ? __ldg(row) : -1;
    pg1 = T_ < TK && ((col + 1) << c.tshift) < s.len ? __ldg(row + 1) : -1;
  };
  pages_of(ahead);
  auto issue = [&]() {
    if (issued < u1) {
      const uint32_t st = base + uint32_t((issued - u0) % S::STAGES) * S::STAGE;
      const int tok0 = ahead.tile * TK, col = tok0 >> c.tshift;
      const bool ok0 = pg0 >= 0 && pg0 < c.pages, ok1 = pg1 >= 0 && pg1 < c.pages;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool used = (k == 0 || T_ < TK) && ((col + k) << c.tshift) < ahead.len;
        if (lane == k && (used || k == 0)) {
          const uint32_t sc = st + S::KBYTES + S::VBYTES + 8 * k;
          if (k ? ok1 : ok0) {
            cp4(sc, c.ks + c.block(k ? pg1 : pg0, ahead.h));
            cp4(sc + 4, c.vs + c.block(k ? pg1 : pg0, ahead.h));
          } else {
            // no such page: its positions are masked
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sc), "f"(0.f), "f"(-1.f)
                         : "memory");
            if (used) record_error(status, WQ_ERR_ARG);
          }
        }
      }
      constexpr int PER = D / 16, STEP = 32 / PER > 0 ? 32 / PER : 1;
      const int piece = lane % PER;
#pragma unroll
      for (int r0 = 0; r0 < TK; r0 += STEP) {
        const int r = r0 + lane / PER, tok = tok0 + r;
        const bool second = (tok >> c.tshift) != col;
        if (tok < ahead.len && (second ? ok1 : ok0)) {
          const int64_t at = ((c.block(second ? pg1 : pg0, ahead.h) << c.tshift) + (tok & (T_ - 1))) * D +
                             piece * 16;
          cp16(st + r * S::KP + swz(D, r, piece) * 16, c.kq + at);
          cp16(st + S::KBYTES + r * S::VP + swz(D, r, piece) * 16, c.vq + at);
        }
      }
      ++issued;
      advance(ahead);
      if (issued < u1) pages_of(ahead);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) issue();

  uint32_t qa[KS][2 * NB];
  float acc[NB][MT][4];
  float m[NB], l[NB], fq[NB];
  int lim[NB];
  bool fresh = true, first_seg = true;
  int seg_tile0 = me.tile;

  for (int64_t u = u0; u < u1; ++u) {
    if (fresh) {
      // -------------------------------------------- a segment's queries
      fresh = false;
      seg_tile0 = me.tile;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        constexpr int P = D / 8, RPP = 32 / P;
        __syncwarp();
#pragma unroll 1
        for (int r0 = 0; r0 < 8; r0 += RPP) {
          const int r = r0 + lane / P, d = (lane % P) * 8;
          const int rr = me.rb * RB + nb * 8 + r;
          float x[8] = {};
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
            rotated8(row, d, pos, rq, x);
          }
          float a = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
#pragma unroll
          for (int o = P / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          // a power of two brings the row's largest element to [2^14, 2^15)
          int ex = (a > 0.f && a <= 3.4028234663852886e38f)
                       ? 141 - int(__float_as_uint(a) >> 23)
                       : 0;
          ex = ex > 100 ? 100 : ex;
          const float up = __uint_as_float(uint32_t(127 + ex) << 23);
          uint4 o;
          o.x = f16x2(x[0] * up, x[1] * up);
          o.y = f16x2(x[2] * up, x[3] * up);
          o.z = f16x2(x[4] * up, x[5] * up);
          o.w = f16x2(x[6] * up, x[7] * up);
          *reinterpret_cast<uint4*>(qs + r * S::QP + d) = o;
          if (lane % P == 0)
            *reinterpret_cast<float*>(qs + r * S::QP + D) =
                __uint_as_float(uint32_t(127 - ex) << 23);
        }
        __syncwarp();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int j = ks >> 2, w = ks & 3;
          const int pc = D == 64 ? t : 2 * t + (j & 1) + 8 * (j >> 1);
          const uint2 v = lds64(qbase + uint32_t(g * S::QP + pc * 16 + w * 4) * 2);
          qa[ks][nb] = v.x;
          qa[ks][NB + nb] = v.y;
        }
        fq[nb] = lds32f(qbase + uint32_t(g * S::QP + D) * 2) * ar.scale_log2 * Code<FMT>::SCALE;
        const int rr = me.rb * RB + nb * 8 + g;
        lim[nb] = rr < me.n * ar.G ? min(me.len, me.len - me.n + rr / ar.G + 1) : 0;
        m[nb] = -CUDART_INF_F;
        l[nb] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nb][mt][e] = 0.f;
      }
    }
    cp_wait<S::STAGES - 2>();
    __syncwarp();
    issue();
    const uint32_t st = base + uint32_t((u - u0) % S::STAGES) * S::STAGE;
    const uint32_t vb = st + S::KBYTES, scb = vb + S::VBYTES;

    // -------------------------------------------------- scores
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
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
          Code<FMT>::word(kw[w], b0, b1);
          const int ks = j * 4 + w;
          mma16816(sc[nt], qa[ks][0], NB == 2 ? qa[ks][NB - 1] : 0u, qa[ks][NB],
                   NB == 2 ? qa[ks][2 * NB - 1] : 0u, b0, b1);
        }
      }
    }

    // -------------------------------------------------- softmax, base 2
    float k0 = lds32f(scb), v0 = lds32f(scb + 4), k1 = k0, v1 = v0;
    if (T_ < TK) {
      k1 = lds32f(scb + 8);
      v1 = lds32f(scb + 12);
      if ((((me.tile * TK) >> c.tshift) + 1) << c.tshift >= me.len) k1 = 0.f, v1 = -1.f;
    }
    const float lv0 = v0 < 0.f ? -CUDART_INF_F : __log2f(fmaxf(v0, 1e-30f));
    const float lv1 = v1 < 0.f ? -CUDART_INF_F : __log2f(fmaxf(v1, 1e-30f));
    const float rv0 = __fdividef(1.f, fmaxf(v0, 1e-30f)), rv1 = __fdividef(1.f, fmaxf(v1, 1e-30f));
    float mx[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float f0 = fq[nb] * k0, f1 = fq[nb] * k1;
      mx[nb] = -CUDART_INF_F;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool hi = NT == 4 && nt >= 2;  // the unit's second page, where it has two
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = sc[nt][2 * nb + e];
          x = fmaf(x, hi ? f1 : f0, hi ? lv1 : lv0);
          if (me.tile * TK + nt * 8 + 2 * t + e >= lim[nb]) x = -CUDART_INF_F;
          mx[nb] = fmaxf(mx[nb], x);
        }
      }
      mx[nb] = fmaxf(mx[nb], __shfl_xor_sync(0xffffffffu, mx[nb], 1));
      mx[nb] = fmaxf(mx[nb], __shfl_xor_sync(0xffffffffu, mx[nb], 2));
    }
    bool grow = mx[0] > m[0] + LAG;
    if (NB == 2) grow |= mx[NB - 1] > m[NB - 1] + LAG;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float now = fmaxf(m[nb], mx[nb]);
        const float al = now == m[nb] ? 1.f : exp2_approx(m[nb] - now);
        m[nb] = now;
        l[nb] *= al;
        const float a0 = __shfl_sync(0xffffffffu, al, t * 8);
        const float a1 = __shfl_sync(0xffffffffu, al, t * 8 + 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[nb][mt][0] *= a0;
          acc[nb][mt][1] *= a1;
          acc[nb][mt][2] *= a0;
          acc[nb][mt][3] *= a1;
        }
      }
    }
    uint32_t pb[NB][NT];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float off = OFF - (m[nb] == -CUDART_INF_F ? 0.f : m[nb]);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float a = exp2_approx(sc[nt][2 * nb] + off);
        const float b = exp2_approx(sc[nt][2 * nb + 1] + off);
        if (NT == 4 && nt >= 2)
          s1 += a + b;
        else
          s0 += a + b;
        pb[nb][nt] = f16x2(a, b);
      }
      l[nb] += s0 * rv0 + s1 * rv1;
    }

    // -------------------------------------------------- values
#pragma unroll
    for (int ks = 0; ks < TK / 16; ++ks) {
      const int r = ks * 16 + 2 * t;
      if (D == 64) {
        const int pc = g >> 1, off = (g & 1) * 8;
        const uint2 x0 = lds64(vb + r * S::VP + pc * 16 + off);
        const uint2 x1 = lds64(vb + (r + 1) * S::VP + pc * 16 + off);
        const uint2 x8 = lds64(vb + (r + 8) * S::VP + pc * 16 + off);
        const uint2 x9 = lds64(vb + (r + 9) * S::VP + pc * 16 + off);
        const uint32_t w0[2] = {x0.x, x0.y}, w1[2] = {x1.x, x1.y};
        const uint32_t w8[2] = {x8.x, x8.y}, w9[2] = {x9.x, x9.y};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int w = mt >> 1 & 1, e = (mt & 1) * 2;
          const uint32_t a0 = Code<FMT>::cross(w0[w], w1[w], e);
          const uint32_t a1 = Code<FMT>::cross(w0[w], w1[w], e + 1);
          const uint32_t a2 = Code<FMT>::cross(w8[w], w9[w], e);
          const uint32_t a3 = Code<FMT>::cross(w8[w], w9[w], e + 1);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(acc[nb][mt], a0, a1, a2, a3, pb[nb][2 * ks], pb[nb][2 * ks + 1]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < D / 128; ++q) {
          const int pc = g + 8 * q;
          const uint4 x0 = lds128(vb + r * S::VP + swz(D, r, pc) * 16);
          const uint4 x1 = lds128(vb + (r + 1) * S::VP + swz(D, r + 1, pc) * 16);
          const uint4 x8 = lds128(vb + (r + 8) * S::VP + swz(D, r + 8, pc) * 16);
          const uint4 x9 = lds128(vb + (r + 9) * S::VP + swz(D, r + 9, pc) * 16);
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
          const uint32_t w8[4] = {x8.x, x8.y, x8.z, x8.w}, w9[4] = {x9.x, x9.y, x9.z, x9.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int w = k >> 1, e = (k & 1) * 2;
            const uint32_t a0 = Code<FMT>::cross(w0[w], w1[w], e);
            const uint32_t a1 = Code<FMT>::cross(w0[w], w1[w], e + 1);
            const uint32_t a2 = Code<FMT>::cross(w8[w], w9[w], e);
            const uint32_t a3 = Code<FMT>::cross(w8[w], w9[w], e + 1);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma16816(acc[nb][(q * 8 + k) % MT], a0, a1, a2, a3, pb[nb][2 * ks],
                       pb[nb][2 * ks + 1]);
          }
        }
      }
    }

    // -------------------------------------------------- end of a segment
    const bool last = me.tile + 1 == me.tiles || u + 1 == u1;
    if (last) {
      const bool whole = seg_tile0 == 0 && me.tile + 1 == me.tiles;
      const int64_t part = id * 2 + (first_seg ? 0 : 1);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 1);
        l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 2);
        if (!whole && t == 0) {
          float* ml = ar.part_ml + (part * RB + nb * 8 + g) * 2;
          __stcg(ml, m[nb]);
          __stcg(ml + 1, l[nb]);
        }
        const float inv = l[nb] == 0.f ? 0.f : Code<FMT>::SCALE / l[nb];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int r = nb * 8 + 2 * t + q;
          const float iv = __shfl_sync(0xffffffffu, inv, t * 8 + 4 * q);
          const int rr = me.rb * RB + r;
          constexpr int RUN = D == 64 ? 8 : 16;  // consecutive elements of this lane
          if (!whole) {
#pragma unroll
            for (int k = 0; k < D / 8; k += 4) {
              float* dst = ar.parts + (part * RB + r) * D + (k / RUN) * 128 + g * RUN + k % RUN;
              __stcg(reinterpret_cast<float4*>(dst),
                     make_float4(acc[nb][k / 2][q], acc[nb][k / 2][q + 2], acc[nb][k / 2 + 1][q],
                                 acc[nb][k / 2 + 1][q + 2]));
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
                const float v = acc[nb][(k + e) / 2][q + 2 * (e & 1)] * iv;
                if constexpr (sizeof(TQ) == 2 && std::is_same<TQ, __half>::value)
                  y.e[e] = __float2half_rn(v);
                else
                  y.e[e] = __float2bfloat16_rn(v);
              }
              *reinterpret_cast<uint4*>(o + (k / RUN) * 128 + g * RUN + k % RUN) = y.v;
            }
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

// Joins the parts of cut segments: one CTA per (sequence, head, row block),
// RB x 32 threads times GROUPS; group k takes parts k, k + GROUPS, ... of its
// row in order, and the groups are added in order.
template <typename TQ, int FMT, int D, int NB>
__global__ void __launch_bounds__(1024)
    attn_kv8_join_kernel(TQ* __restrict__ O, Cache c, Batch bt, Args ar, int64_t total_warps,
                         int most_rb) {
  constexpr int RB = 8 * NB, GROUPS = 32 / RB, PER = D / 32;  // elements per lane
  __shared__ float sm[GROUPS][RB], sl[GROUPS][RB];
  __shared__ float so[GROUPS][RB][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t id = blockIdx.x;
  const int rb = int(id % most_rb);
  id /= most_rb;
  const int h = int(id % c.heads), b = int(id / c.heads);
  Cursor s;
  s.b = b;
  s.load(bt, c.tshift, ar.G, RB, Shape<D>::TK, nullptr);
  if (s.n == 0 || rb >= s.nrb) return;
  const int64_t U = ar.prefix[bt.B], W = workers(U, total_warps);
  const int64_t f = ar.prefix[b] + (int64_t(h) * s.nrb + rb) * s.tiles;
  const int64_t wa = run_owner(f, U, W), wb = run_owner(f + s.tiles - 1, U, W);
  if (wa == wb) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = warp % RB, grp = warp / RB;
  float m = -CUDART_INF_F, l = 0.f, o[PER] = {};
  // a worker's first segment is its part 0, a later (cut) one its part 1
  for (int64_t w0 = wa + grp; w0 <= wb; w0 += GROUPS * 8) {
    float pm[8], pl[8], po[8][PER];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t w = w0 + k * GROUPS;
      pm[k] = -CUDART_INF_F, pl[k] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) po[k][e] = 0.f;
      if (w <= wb) {
        const int64_t row = (w * 2 + (run_start(w, U, W) >= f ? 0 : 1)) * RB + r;
        pm[k] = __ldcg(ar.part_ml + row * 2);
        pl[k] = __ldcg(ar.part_ml + row * 2 + 1);
#pragma unroll
        for (int e = 0; e < PER; ++e) po[k][e] = __ldcg(ar.parts + row * D + e * 32 + lane);
      }
    }
    float now = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) now = fmaxf(now, pm[k]);
    if (now == -CUDART_INF_F) now = 0.f;
    const float a = exp2_approx(m - now);
    m = now;
    l *= a;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= a;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = exp2_approx(pm[k] - now);
      l = fmaf(pl[k], x, l);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(po[k][e], x, o[e]);
    }
  }
  if (lane == 0) sm[grp][r] = m, sl[grp][r] = l;
#pragma unroll
  for (int e = 0; e < PER; ++e) so[grp][r][e * 32 + lane] = o[e];
  __syncthreads();
  if (grp != 0) return;
  float now = -CUDART_INF_F;
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) now = fmaxf(now, sm[k][r]);
  if (now == -CUDART_INF_F) now = 0.f;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) {
    const float x = exp2_approx(sm[k][r] - now);
    l = fmaf(sl[k][r], x, l);
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = fmaf(so[k][r][e * 32 + lane], x, o[e]);
  }
  const int rr = rb * RB + r;
  if (rr >= s.n * ar.G) return;
  const float inv = l == 0.f ? 0.f : Code<FMT>::SCALE / l;
  const int i = rr / ar.G;
  TQ* dst = O + (int64_t(s.q0 + i) * ar.heads + h * ar.G + (rr - i * ar.G)) * D;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if constexpr (std::is_same<TQ, __half>::value)
      dst[e * 32 + lane] = __float2half_rn(o[e] * inv);
    else
      dst[e * 32 + lane] = __float2bfloat16_rn(o[e] * inv);
  }
}

}  // namespace kv8
}  // namespace wq

namespace wq_host {

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Row blocks of 16 where there are more than 8 rows to a (sequence, head); a
// 256-wide head's sums fit the registers of 8 rows only.
int row_blocks(int64_t max_rows, int64_t D) { return max_rows > 8 && D <= 128 ? 2 : 1; }

struct Ws {
  size_t ml, prefix, bytes;
};
Ws attn_ws(int64_t B, int64_t max_rows, int64_t D) {
  const size_t w2 = size_t(sm_count()) * wq::kv8::WARPS * 2, rb = size_t(8 * row_blocks(max_rows, D));
  Ws s;
  s.ml = up256(w2 * rb * size_t(D) * 4);
  s.prefix = s.ml + up256(w2 * rb * 8);
  s.bytes = s.prefix + up256(size_t(B + 1) * 8);
  return s;
}

template <typename TQ, int FMT, int D, int NB>
int launch_decode(const void* Q, int64_t ldq, int64_t heads, const Kv8& a, int max_pos, float scale,
                  void* out, uint8_t* ws, cudaStream_t s) {
  using namespace wq::kv8;
  auto kern = attn_kv8_kernel<TQ, FMT, D, NB>;
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
  const Ws w = attn_ws(a.B, a.max_new * G, D);
  const Args ar{ldq, int(heads), G, scale * 1.4426950408889634f, reinterpret_cast<float*>(ws),
                reinterpret_cast<float*>(ws + w.ml), reinterpret_cast<int64_t*>(ws + w.prefix)};
  const int grid = sm_count();
  TQ* o = static_cast<TQ*>(out);
  kern<<<grid, WARPS * 32, smem, s>>>(static_cast<const TQ*>(Q), o, c, bt, rp, ar, status_ptr());
  WQ_LAUNCH_CHECK("attn_kv8_kernel");
  const int64_t most_rb = (a.max_new * G + 8 * NB - 1) / (8 * NB);
  const int64_t joins = a.B * a.kv_heads * most_rb;
  if (joins > 0x7fffffff) return WQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(joins));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  WQ_CUDA_CHECK(cudaLaunchKernelEx(&cfg, attn_kv8_join_kernel<TQ, FMT, D, NB>, o, c, bt, ar,
                                   int64_t(grid) * WARPS, int(most_rb)));
  return WQ_OK;
}

template <typename TQ, int FMT>
int launch_by_shape(const void* Q, int64_t ldq, int64_t heads, const Kv8& a, int max_pos,
                    float scale, void* out, uint8_t* ws, cudaStream_t s) {
  const int nb = row_blocks(a.max_new * (heads / a.kv_heads), a.D);
#define WQ_ATTN(D_, NB_) \
  return launch_decode<TQ, FMT, D_, NB_>(Q, ldq, heads, a, max_pos, scale, out, ws, s)
  if (a.D == 64) {
    if (nb == 1) WQ_ATTN(64, 1);
    WQ_ATTN(64, 2);
  }
  if (a.D == 128) {
    if (nb == 1) WQ_ATTN(128, 1);
    WQ_ATTN(128, 2);
  }
  WQ_ATTN(256, 1);
#undef WQ_ATTN
}

}  // namespace

size_t attn_kv8_workspace_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t D,
                                int64_t max_q) {
  return attn_ws(B, max_q * (heads / kv_heads), D).bytes;
}

int launch_attn_kv8(const void* Q, int dtype, int64_t ldq, int64_t heads, const Kv8& a,
                    int max_pos, float scale, void* out, void* ws, cudaStream_t s) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool i8 = a.fmt == WQ_W8_INT8;
  if (dtype == WQ_BF16)
    return i8 ? launch_by_shape<__nv_bfloat16, WQ_W8_INT8>(Q, ldq, heads, a, max_pos, scale, out, w, s)
              : launch_by_shape<__nv_bfloat16, WQ_W8_E4M3>(Q, ldq, heads, a, max_pos, scale, out, w, s);
  return i8 ? launch_by_shape<__half, WQ_W8_INT8>(Q, ldq, heads, a, max_pos, scale, out, w, s)
            : launch_by_shape<__half, WQ_W8_E4M3>(Q, ldq, heads, a, max_pos, scale, out, w, s);
}

}  // namespace wq_host
