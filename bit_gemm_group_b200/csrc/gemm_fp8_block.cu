// gemm_fp8_block.cu -- E4M3 x E4M3 product with a scale for each block of 128
// along K (per token for X, per 128 output channels for W):
//
//   Y[m, n] = bf16( sum_J sx[m, J] sw[n / 128, J] sum_{k in J} qx[m, k] qw[n, k] )
//
// The inner sums run on the fp8 tensor cores into tensor memory, one 128-wide
// K block at a time; warps read each block's sums back and add them, scaled,
// to fp32 registers while the tensor cores work on the next block.  Two
// kernels, by what bounds them:
//
//   gemm_fp8_block_kernel    (tensor cores) 128 tokens x 256 channels per
//     tile, tokens on the tensor-memory lanes: a thread owns one token and 128
//     channels of one weight block, so a K block's scale is one number per
//     thread.
//   gemm_fp8_block_split_kernel  (HBM or L2) 128 channels x NT tokens per
//     tile, channels on the lanes: every SM streams the same number of
//     (tile, K block) units whatever the shape; a tile cut between CTAs is
//     joined, in K order, by the CTA that arrives last.  1 x 28672 x 8192: 51
//     us, 4.6 TB/s with the quantizer's launch and the join (about 11 us that do
//     not depend on the weights: at 16 x 4096 x 11008 they are half of 19 us).
#include <mutex>

#include "kernels.h"
#include "tc.cuh"

namespace wq {
namespace fp8b {

constexpr int BK = 128;

// ---------------------------------------------------------------------------
// Large products
// ---------------------------------------------------------------------------
// 4 x 48 KB of operands on their way, two 128 x 256 sums in tensor memory.  At
// 4096 x 11008 x 4096 the copies and products alone take 117 us (3.2 PFLOP/s);
// with the sums read back for every K block the GPU is at its 1 kW cap (1.63
// GHz) and at 180 us: what is left is the hand-off of two buffers, not L2 (a
// CTA pair on 256 x 256 tiles, a third less traffic, measured the same), nor
// the additions (without them 175 us), nor more and smaller buffers (four of
// 128 channels: 220 us, operands are read twice).
constexpr int BM = 128, BN = 256;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 16;
constexpr int OUT_BYTES = 32 * 32 * 2;  // a warp's rows x 32 channels, on their way out
// warps 0 to 3 copy and issue, 4 to 19 add: 96 registers a thread at launch,
// split 32 to 112 (64 sums and a chunk of 32 on its way)
constexpr int THREADS_L = 32 * (4 + EPI_WARPS);
constexpr int REGS_ISSUE = 32, REGS_ADD = 112;
static_assert(4 * REGS_ISSUE + EPI_WARPS * REGS_ADD <= (4 + EPI_WARPS) * 96, "registers");
constexpr uint32_t IDESC_L = tc::idesc_e4m3_f32(BM, BN);

struct SmemL {
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t SMEM_L =
    1024 + size_t(STAGES) * STAGE_BYTES + size_t(EPI_WARPS) * OUT_BYTES + sizeof(SmemL);

// acc[0..1] += s * d[0..1] (two fp32 fused multiply-adds in one instruction)
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s2) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s2));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  return r;
}
__device__ __forceinline__ float one_of(uint64_t v, int i) {
  return __uint_as_float(uint32_t(i ? v >> 32 : v));
}
__device__ __forceinline__ uint32_t bf16x2_of(uint64_t v) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(THREADS_L, 1)
    gemm_fp8_block_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB, const float* __restrict__ sxT,
                          int64_t ldsx, const float* __restrict__ sw, __nv_bfloat16* __restrict__ Y,
                          int M, int N, int K, int* status, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t* outs = tiles + size_t(STAGES) * STAGE_BYTES;
  SmemL& sm = *reinterpret_cast<SmemL*>(outs + EPI_WARPS * OUT_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mtiles = (M + BM - 1) / BM, ntiles = (N + BN - 1) / BN;
  const int total = mtiles * ntiles;
  const int kblocks = (K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&sm.full[s], 1);
      tc::mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&sm.tfull[b], 1);
      tc::mbar_init(&sm.tempty[b], EPI_WARPS);
    }
    tc::mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmA);
    tc::tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tc::tmem_alloc(&sm.tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // (the limit starts again with every tile: a product may take longer than one wait)
  tc::Watchdog wd{tc::globaltimer_ns() + limit_ns, &sm.abort_flag, status};
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- producer
      // W does not depend on the quantizer of X, whose codes and scales are
      // complete after griddepcontrol.wait: the first weight tiles come before it
      uint32_t it = 0, pre = 0;
      for (int tile = blockIdx.x; tile < total && pre < uint32_t(STAGES); tile += gridDim.x)
        for (int kb = 0; kb < kblocks && pre < uint32_t(STAGES); ++kb, ++pre) {
          tc::mbar_arrive_expect_tx(&sm.full[pre], STAGE_BYTES);
          tc::tma_load_2d(tiles + size_t(pre) * STAGE_BYTES + A_BYTES, &tmB, &sm.full[pre], kb * BK,
                          tile / mtiles * BN);
        }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        wd.deadline_ns = tc::globaltimer_ns() + limit_ns;
        const int mt = tile % mtiles, nt = tile / mtiles;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          uint8_t* a = tiles + size_t(s) * STAGE_BYTES;
          if (it >= pre) {
            if (!(ok = tc::wait_bounded(&sm.empty[s], ((it / STAGES) & 1u) ^ 1u, wd))) break;
            tc::mbar_arrive_expect_tx(&sm.full[s], STAGE_BYTES);
            tc::tma_load_2d(a + A_BYTES, &tmB, &sm.full[s], kb * BK, nt * BN);
          }
          tc::tma_load_2d(a, &tmA, &sm.full[s], kb * BK, mt * BM);
        }
      }
      // the last load issued into each stage has landed before exit
      const uint64_t dl = tc::globaltimer_ns() + tc::kDrainNs;
      const uint32_t n = it < uint32_t(STAGES) ? it : uint32_t(STAGES);
      for (uint32_t j = 0; j < n; ++j) {
        const uint32_t i = it - 1 - j;
        tc::wait_until(&sm.full[i % STAGES], (i / STAGES) & 1u, dl);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer
      // (the whole warp walks the loop and one lane issues, so that operand
      // addresses stay in uniform registers)
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        wd.deadline_ns = tc::globaltimer_ns() + limit_ns;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t buf = it & 1u;
          if (!(ok = tc::wait_warp(&sm.full[s], (it / STAGES) & 1u, wd))) break;
          if (!(ok = tc::wait_warp(&sm.tempty[buf], ((it >> 1) & 1u) ^ 1u, wd))) break;
          tc::fence_after_sync();
          const uint32_t a = tc::smem_u32(tiles) + uint32_t(s) * STAGE_BYTES, b = a + A_BYTES;
          const uint64_t da = tc::sdesc_k_sw128(a), db = tc::sdesc_k_sw128(b);
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < BK / 32; ++k)
              tc::mma_f8_ss(tmem + buf * BN, da + uint64_t(k * 2), db + uint64_t(k * 2), IDESC_L,
                            k != 0);
            tc::mma_commit(&sm.empty[s]);
            tc::mma_commit(&sm.tfull[buf]);
          }
          __syncwarp();
        }
      }
      if (tc::elect_one()) {
        tc::mma_commit(&sm.drain);
        tc::wait_until(&sm.drain, 0, tc::globaltimer_ns() + tc::kDrainNs);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ADD));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp & 3;            // tensor-memory lane quarter
    const int part = (warp - 4) >> 2;  // channels [64 part, 64 part + 64) of the tile
    const uint32_t out = tc::smem_u32(outs + (warp - 4) * OUT_BYTES);
    uint32_t it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      wd.deadline_ns = tc::globaltimer_ns() + limit_ns;
      const int mt = tile % mtiles, nt = tile / mtiles;
      const int row0 = mt * BM + q * 32;
      const int n0 = nt * BN + part * 64;
      const float* sxp = sxT + (row0 + lane < M ? row0 + lane : M - 1);
      const float* swp = sw + int64_t(n0 < N ? n0 / 128 : 0) * kblocks;
      const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t(part) * 64;
      uint64_t acc[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = 0;
      // scales one K block ahead (multiplied only when they are used)
      float x1 = __ldg(sxp), w1 = __ldg(swp);
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const uint32_t buf = it & 1u;
        const float s = x1 * w1;
        const uint64_t s2 = pair(s, s);
        if (kb + 1 < kblocks) {
          sxp += ldsx;
          ++swp;
        }
        x1 = __ldg(sxp), w1 = __ldg(swp);
        if (!(ok = tc::wait_warp(&sm.tfull[buf], (it >> 1) & 1u, wd))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
          tc::tmem_ld_x32(taddr + buf * BN + c * 32, r);
          tc::tmem_wait_ld();
          if (c == 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_relaxed(&sm.tempty[buf]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(acc[c * 16 + j], r[2 * j], r[2 * j + 1], s2);
        }
      }
      if (!ok) break;
      // 32 channels at a time through shared memory, so that 64 bytes of a row
      // leave together
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint64_t* v = acc + h * 16 + 4 * g;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           out + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)),
                       "r"(bf16x2_of(v[0])), "r"(bf16x2_of(v[1])), "r"(bf16x2_of(v[2])),
                       "r"(bf16x2_of(v[3]))
                       : "memory");
        }
        __syncwarp();
        const int col = n0 + h * 32 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(out + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)));
          if (row0 + r < M && col < N) *reinterpret_cast<uint4*>(Y + int64_t(row0 + r) * N + col) = v;
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Few tokens
// ---------------------------------------------------------------------------
// NT tokens per tile (16, 32, 64 or 128); the epilogue has four warps (one
// thread per channel) up to 64 tokens and eight at 128 (64 tokens each).
template <int NT>
struct Split {
  static constexpr int COLS = NT > 64 ? 64 : NT;  // tokens per epilogue thread
  static constexpr int EWARPS = 4 * (NT / COLS);
  static constexpr int THREADS = 32 * (2 + EWARPS);
  static constexpr int W_BYTES = 128 * BK, X_BYTES = NT * BK, S_BYTES = NT * 4;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  // scales lie behind the swizzled tiles
  static constexpr int STAGES = (200 * 1024) / (STAGE + S_BYTES) > 12 ? 12 : (200 * 1024) / (STAGE + S_BYTES);
  static constexpr int BUFS = 4;
  static constexpr uint32_t TMEM = NT * BUFS < 32 ? 32 : NT * BUFS;
  struct Bars {
    uint64_t full[STAGES], empty[STAGES], tfull[BUFS], tempty[BUFS], drain;
    uint32_t tmem_base;
    int abort_flag;
  };
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * (STAGE + S_BYTES) + sizeof(Bars);
};

// CTA c's units are [c U / G, (c + 1) U / G) of U = tiles x kblocks, tile major.
__device__ __forceinline__ int64_t first_unit(int64_t c, int64_t U, int64_t G) { return c * U / G; }
// the CTA that owns unit u
__device__ __forceinline__ int owner(int64_t u, int64_t U, int64_t G) {
  int64_t c = ((u + 1) * G - 1) / U;  // largest c with c U / G <= u
  return int(c);
}

template <int NT>
__global__ void __launch_bounds__(Split<NT>::THREADS, 1)
    gemm_fp8_block_split_kernel(const __grid_constant__ CUtensorMap tmW,
                                const __grid_constant__ CUtensorMap tmX,
                                const float* __restrict__ sxT, int64_t ldsx,
                                const float* __restrict__ sw, __nv_bfloat16* __restrict__ Y, int M,
                                int N, int K, int* __restrict__ counters,
                                float* __restrict__ partials, int* status, uint64_t limit_ns) {
  using P = Split<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  float* sscale = reinterpret_cast<float*>(tiles + size_t(P::STAGES) * P::STAGE);
  auto& sm = *reinterpret_cast<typename P::Bars*>(reinterpret_cast<uint8_t*>(sscale) +
                                                  size_t(P::STAGES) * P::S_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks = (K + BK - 1) / BK;
  const int ntiles = (N + 127) / 128, mtiles = (M + NT - 1) / NT;
  const int64_t U = int64_t(ntiles) * mtiles * kblocks, G = gridDim.x;
  const int64_t u0 = first_unit(blockIdx.x, U, G), u1 = first_unit(blockIdx.x + 1, U, G);

  const int n_units = int(u1 - u0), pre = n_units < P::STAGES ? n_units : P::STAGES;
  const int kb0 = int(u0 % kblocks), tile0 = int(u0 / kblocks);
  if (threadIdx.x == 0) {
    for (int s = 0; s < P::STAGES; ++s) {
      tc::mbar_init(&sm.full[s], 1);
      tc::mbar_init(&sm.empty[s], P::EWARPS);
    }
    for (int b = 0; b < P::BUFS; ++b) {
      tc::mbar_init(&sm.tfull[b], 1);
      tc::mbar_init(&sm.tempty[b], P::EWARPS);
    }
    tc::mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    tc::fence_mbar_init();
    // W does not depend on the kernel before this one (the quantizer of X): a
    // ring's worth of weight tiles is requested before anything else is set up
    int kb = kb0, tile = tile0;
    for (int i = 0; i < pre; ++i) {
      tc::mbar_arrive_expect_tx(&sm.full[i], P::STAGE + P::S_BYTES);
      tc::tma_load_2d(tiles + size_t(i) * P::STAGE, &tmW, &sm.full[i], kb * BK, tile / mtiles * 128);
      if (++kb == kblocks) kb = 0, ++tile;
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(&sm.tmem_base, P::TMEM);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  const tc::Watchdog wd{tc::globaltimer_ns() + limit_ns, &sm.abort_flag, status};

  if (warp == 0) {
    if (lane == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      int kb = kb0, tile = tile0;
      int it = 0;
      for (; it < n_units; ++it) {
        const int s = it % P::STAGES;
        const int mt = tile % mtiles, nt = tile / mtiles;
        uint8_t* w = tiles + size_t(s) * P::STAGE;
        if (it >= pre) {
          if (!tc::wait_bounded(&sm.empty[s], ((it / P::STAGES) & 1u) ^ 1u, wd)) break;
          tc::mbar_arrive_expect_tx(&sm.full[s], P::STAGE + P::S_BYTES);
          tc::tma_load_2d(w, &tmW, &sm.full[s], kb * BK, nt * 128);
        }
        tc::tma_load_2d(w + P::W_BYTES, &tmX, &sm.full[s], kb * BK, mt * NT);
        tc::bulk_load(sscale + s * NT, sxT + kb * ldsx + int64_t(mt) * NT, P::S_BYTES, &sm.full[s]);
        if (++kb == kblocks) kb = 0, ++tile;
      }
      const uint64_t dl = tc::globaltimer_ns() + tc::kDrainNs;
      const int back = it < P::STAGES ? it : P::STAGES;
      for (int j = 0; j < back; ++j) {
        const int i = it - 1 - j;
        tc::wait_until(&sm.full[i % P::STAGES], (i / P::STAGES) & 1u, dl);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3_f32(128, NT);
      for (int it = 0; it < n_units; ++it) {
        const int s = it % P::STAGES;
        const uint32_t buf = uint32_t(it) % P::BUFS;
        if (!tc::wait_bounded(&sm.tempty[buf], ((it / P::BUFS) & 1u) ^ 1u, wd)) break;
        if (!tc::wait_bounded(&sm.full[s], (it / P::STAGES) & 1u, wd)) break;
        tc::fence_after_sync();
        const uint32_t w = tc::smem_u32(tiles + size_t(s) * P::STAGE), x = w + P::W_BYTES;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          tc::mma_f8_ss(tmem + buf * NT, tc::sdesc_k_sw128(w + k * 32),
                        tc::sdesc_k_sw128(x + k * 32), idesc, k != 0);
        tc::mma_commit(&sm.tfull[buf]);
      }
      tc::mma_commit(&sm.drain);
      tc::wait_until(&sm.drain, 0, tc::globaltimer_ns() + tc::kDrainNs);
    }
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp & 3;
    const int cg = (warp - 2) >> 2;           // token group of COLS
    const int ch = q * 32 + lane;             // channel within the tile
    int it = 0;
    int slot = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const int tile = int(u / kblocks);
      const int64_t t0 = int64_t(tile) * kblocks, t1 = t0 + kblocks;
      const int64_t e = u1 < t1 ? u1 : t1;
      const int mt = tile % mtiles, nt = tile / mtiles;
      const int n = nt * 128 + ch;
      // weight scales: lane i holds that of the segment's K block 32 b + i, and
      // the next 32 are on their way
      const float* swp = sw + int64_t(nt) * kblocks + (u - t0);
      const int blocks = int(e - u);
      float w_now = lane < blocks ? __ldg(swp + lane) : 0.f;
      float w_next = lane + 32 < blocks ? __ldg(swp + lane + 32) : 0.f;
      const bool whole = u == t0 && e == t1;
      uint64_t acc[P::COLS / 2];
#pragma unroll
      for (int j = 0; j < P::COLS / 2; ++j) acc[j] = 0;
      for (int i = 0; i < blocks; ++i, ++u, ++it) {
        const uint32_t buf = uint32_t(it) % P::BUFS;
        const int s = it % P::STAGES;
        const float wk = __shfl_sync(0xffffffffu, w_now, i & 31);
        if ((i & 31) == 31) {
          w_now = w_next;
          w_next = i + 33 + lane < blocks ? __ldg(swp + i + 33 + lane) : 0.f;
        }
        // both, so that the scales (written by the copy) are seen as well
        if (!(ok = tc::wait_warp(&sm.full[s], (it / P::STAGES) & 1u, wd))) break;
        if (!(ok = tc::wait_warp(&sm.tfull[buf], (it / P::BUFS) & 1u, wd))) break;
        tc::fence_after_sync();
        const uint32_t taddr =
            tmem + (uint32_t(q * 32) << 16) + buf * NT + uint32_t(cg) * P::COLS;
        const uint32_t sp = tc::smem_u32(sscale + s * NT + cg * P::COLS);
        const uint64_t w2 = pair(wk, wk);
        constexpr int CH = P::COLS > 32 ? 32 : P::COLS;  // tokens read back at a time
#pragma unroll
        for (int c = 0; c < P::COLS / CH; ++c) {
          uint32_t r[CH];
          if constexpr (CH == 32)
            tc::tmem_ld_x32(taddr + c * CH, r);
          else
            tc::tmem_ld_x16(taddr + c * CH, r);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < CH / 4; ++j) {
            uint64_t f[2];
            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                         : "=l"(f[0]), "=l"(f[1])
                         : "r"(sp + (c * CH + j * 4) * 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(f[k]) : "l"(w2));
              fma2(acc[(c * CH + j * 4) / 2 + k], r[j * 4 + 2 * k], r[j * 4 + 2 * k + 1], f[k]);
            }
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        // the stage is free when every epilogue warp has read its scales and
        // the tensor cores its tiles (they have: tfull).  A release: the copy that
        // overwrites the scales comes after the warp's reads of them.
        if (lane == 0) {
          tc::mbar_arrive_relaxed(&sm.tempty[buf]);
          tc::mbar_arrive(&sm.empty[s]);
        }
      }
      if (!ok) break;
      const int tok0 = mt * NT + cg * P::COLS;
      if (!whole) {
        // a cut tile: this warp's part (32 channels) goes to the workspace, and
        // the last of the tile's warps for these channels adds the parts in K
        // order.  The counter's release and acquire cover the warp's stores and
        // loads (ordered with its lane 0 by the warp's synchronisation, on either side).
        const int64_t part = int64_t(P::COLS) * 128 * (NT / P::COLS);
        float* dst = partials + (int64_t(blockIdx.x) * 2 + slot) * part + cg * P::COLS * 128 + ch;
        slot = 1;
#pragma unroll
        for (int j = 0; j < P::COLS; ++j)
          if (tok0 + j < M) __stcg(dst + j * 128, one_of(acc[j / 2], j & 1));
        __syncwarp();
        const int c0 = owner(t0, U, G), c1 = owner(t1 - 1, U, G);
        int before = 0;
        if (lane == 0)
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(counters + int64_t(tile) * P::EWARPS + (warp - 2))
                       : "memory");
        if (__shfl_sync(0xffffffffu, before, 0) != c1 - c0) continue;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < P::COLS / 2; ++j) acc[j] = 0;
        for (int c = c0; c <= c1; ++c) {
          // a CTA's first part is in slot 0; it is a second one when the CTA
          // began with the tail of an earlier tile
          const bool second = first_unit(c, U, G) < t0 && (first_unit(c, U, G) % kblocks) != 0;
          const float* src = partials + (int64_t(c) * 2 + second) * part + cg * P::COLS * 128 + ch;
#pragma unroll
          for (int j = 0; j < P::COLS / 2; ++j) {  // (all loads in flight)
            const uint64_t v = pair(__ldcg(src + 2 * j * 128), __ldcg(src + (2 * j + 1) * 128));
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc[j]) : "l"(v));
          }
        }
      }
      if (n < N) {
#pragma unroll
        for (int j = 0; j < P::COLS; ++j)
          if (tok0 + j < M) Y[int64_t(tok0 + j) * N + n] = __float2bfloat16_rn(one_of(acc[j / 2], j & 1));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, P::TMEM);
  }
}

}  // namespace fp8b
}  // namespace wq

namespace wq_host {

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Tokens per tile of the split kernel, or 0 for the large-product kernel.  A K
// block takes a CTA of the large kernel 0.43 us for 128 x 256 sums, one of the
// split kernel 0.5 us for 128 x 128 (a quarter less for 128 x 64), but those are
// shared out evenly over the SMs and their join takes about as long as 30 (22).
// Measured, large and split, with weights from HBM: 96 x 2048 x 4096 24.6 and
// 30.7 us, 96 x 2048 x 8192 38.9 and 32.8, 129 x 8192 x 8192 45 and 51, 129 x
// 4096 x 8192 41 and 37, 96 x 28672 x 11008 76 and 92, 384 x 16384 x 4096 47 and
// 72, 64 x 28672 x 4096 37 and 45, 64 x 8192 x 8192 41 and 33; within a tenth
// near the border.  Up to 32 tokens the split kernel is as fast or faster but for
// K near 2048 (17 x 28672 x 2048: 24.6 and 28.7).
int split_tokens(int64_t M, int64_t N, int64_t K) {
  const int64_t kb = (K + 127) / 128, mt = (M + 127) / 128, sms = sm_count();
  const int64_t waves = (mt * ((N + 255) / 256) + sms - 1) / sms;
  const int64_t units = mt * ((N + 127) / 128) * kb / sms;
  if (M > 32 && waves * kb <= (M > 64 ? units + 30 : units * 3 / 4 + 22)) return 0;
  return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
}

struct Plan {
  int nt;
  int64_t mp;                  // tokens, padded to a multiple of 128
  int tiles, n_counters;
  size_t sx, counters, partials, bytes;  // offsets in the workspace, and its size
};

Plan plan(int64_t M, int64_t N, int64_t K) {
  Plan p;
  const int64_t kb = (K + 127) / 128;
  p.nt = split_tokens(M, N, K);
  p.mp = (M + 127) / 128 * 128;
  p.sx = up256(size_t(M) * size_t(K));
  p.counters = p.sx + up256(size_t(kb * p.mp) * 4);
  p.tiles = p.nt ? int(((N + 127) / 128) * ((M + p.nt - 1) / p.nt)) : 0;
  p.n_counters = p.tiles * (p.nt > 64 ? 8 : 4);  // one for each adding warp
  // room for the split kernel whether it is taken or not, so that the size grows
  // with M and a workspace serves fewer tokens too
  const int64_t most = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  p.partials = p.counters + up256(size_t((N + 127) / 128) * size_t(p.mp / 128) * 8 * 4);
  p.bytes = p.partials + size_t(sm_count()) * 2 * size_t(most) * 128 * 4;
  return p;
}

template <typename Kern>
cudaError_t set_smem(Kern kern, size_t bytes, int which) {
  static std::mutex mu;
  static bool done[5][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && done[which][dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess && dev < 64) done[which][dev] = true;
  return e;
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(int grid, int threads, size_t smem, cudaStream_t s) {
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <int NT>
int launch_split(const CUtensorMap& tx, const void* Wq, const float* sx, const float* sw,
                 const Plan& p, int64_t M, int64_t N, int64_t K, void* Y, uint8_t* ws,
                 cudaStream_t s) {
  using namespace wq::fp8b;
  CUtensorMap tw;
  int st = make_tmap_2d(&tw, Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(N), uint64_t(K), 128,
                        BK, 128);
  if (st != WQ_OK) return st;
  constexpr int which = NT == 16 ? 1 : NT == 32 ? 2 : NT == 64 ? 3 : 4;
  WQ_CUDA_CHECK(set_smem(gemm_fp8_block_split_kernel<NT>, Split<NT>::SMEM, which));
  const int64_t units = int64_t(p.tiles) * ((K + 127) / 128);
  const int grid = int(units < sm_count() ? units : sm_count());
  Launch l(grid, Split<NT>::THREADS, Split<NT>::SMEM, s);
  WQ_CUDA_CHECK(cudaLaunchKernelEx(&l.cfg, gemm_fp8_block_split_kernel<NT>, tw, tx, sx, p.mp, sw,
                                   static_cast<__nv_bfloat16*>(Y), int(M), int(N), int(K),
                                   reinterpret_cast<int*>(ws + p.counters),
                                   reinterpret_cast<float*>(ws + p.partials), status_ptr(),
                                   wait_limit_ns()));
  return WQ_OK;
}

}  // namespace

size_t fp8_block_workspace_bytes(int64_t M, int64_t N, int64_t K) { return plan(M, N, K).bytes; }

int launch_gemm_fp8_block(const void* X, int64_t M, int64_t K, const void* Wq, const float* sw,
                          int64_t N, void* Y, void* ws, cudaStream_t s) {
  using namespace wq::fp8b;
  const Plan p = plan(M, N, K);
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* sx = reinterpret_cast<float*>(w + p.sx);
  int st = launch_quantize_fp8_block(X, WQ_BF16, M, K, 1, w, sx, p.mp, true,
                                     reinterpret_cast<int*>(w + p.counters), p.n_counters, s);
  if (st != WQ_OK) return st;
  CUtensorMap tx;
  st = make_tmap_2d(&tx, w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(M), uint64_t(K),
                    p.nt ? uint32_t(p.nt) : uint32_t(BM), BK, 128);
  if (st != WQ_OK) return st;
  switch (p.nt) {
    case 16: return launch_split<16>(tx, Wq, sx, sw, p, M, N, K, Y, w, s);
    case 32: return launch_split<32>(tx, Wq, sx, sw, p, M, N, K, Y, w, s);
    case 64: return launch_split<64>(tx, Wq, sx, sw, p, M, N, K, Y, w, s);
    case 128: return launch_split<128>(tx, Wq, sx, sw, p, M, N, K, Y, w, s);
  }
  CUtensorMap tw;
  st = make_tmap_2d(&tw, Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(N), uint64_t(K), BN, BK,
                    128);
  if (st != WQ_OK) return st;
  WQ_CUDA_CHECK(set_smem(gemm_fp8_block_kernel, SMEM_L, 0));
  const int64_t total = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  if (total > 0x7fffffff) return WQ_ERR_UNSUPPORTED;
  const int grid = int(total < sm_count() ? total : sm_count());
  Launch l(grid, THREADS_L, SMEM_L, s);
  WQ_CUDA_CHECK(cudaLaunchKernelEx(&l.cfg, gemm_fp8_block_kernel, tx, tw, sx, p.mp, sw,
                                   static_cast<__nv_bfloat16*>(Y), int(M), int(N), int(K),
                                   status_ptr(), wait_limit_ns()));
  return WQ_OK;
}

}  // namespace wq_host
