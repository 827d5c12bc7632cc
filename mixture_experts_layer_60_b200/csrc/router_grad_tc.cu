// The scored router's two gradient products on tcgen05 CTA pairs (bf16 u, E):
//   du[t] = du_base[t] + sum_i d_logit[t,i] E[i]
//   dE[i] = sum_t d_logit[t,i] u[t]
// d_logit is float32; it enters as bf16 planes hi + mid + lo (8 bits each,
// round to nearest), laid out [3][Tp][Np] by the gradient kernel, with zero
// rows from T to Tp (a multiple of 64) and zero columns from N_r to Np (a
// multiple of 8).  du is rounded to bf16, so hi and mid (an error of 2^-18 of
// each term) are enough; dE is float32 and takes all three.
//
// Every wait is bounded (1 s of %globaltimer) and reported through the device
// error word.
#include "launch.h"
#include "sm100.cuh"

namespace moe {

moe_status make_tmap_2d(CUtensorMap* tm, const void* base, CUtensorMapDataType dtype,
                        int elem_bytes, uint64_t inner, uint64_t outer, uint32_t box_inner,
                        uint32_t box_outer);

namespace {

using namespace sm100;

constexpr int BK = 64;                       // contraction per stage
constexpr int BN = 256;                      // columns of d per slab (128 per CTA of the pair)
constexpr int kBox = 64 * BK * 2;            // one [64][64] bf16 box: 8 KB
constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kPieces = 4;                   // 16-column pieces per epilogue warp and slab
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kPairs = 74;                   // CTA pairs of 148 SMs

// Barriers: full, empty per stage, tfull[2], tempty[2], mma_done, afull, aempty.
template <int STAGES, int STAGE_BYTES, int FIXED_BYTES>
struct Layout {
  static constexpr int OFF_FIXED = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_FIXED + FIXED_BYTES;
  static constexpr int N_BARS = 2 * STAGES + 7;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
};

__device__ __forceinline__ void raise_abort(volatile int* abort, int* err) {
  *abort = 1;
  atomicOr(err, ERR_GEMM_TIMEOUT);
}

// 32 bytes of global memory: one access where the row is 32-byte aligned,
// whole sectors either way.
__device__ __forceinline__ void ld32(const void* p, bool wide, uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
  }
}
__device__ __forceinline__ void st32(void* p, bool wide, const uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    static_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// ---------------------------------------------------------------- dE
// A pair owns 256 experts (128 rows of C per CTA) x a slab of 256 columns x
// one of S slices of the tokens.  Both operands are MN-major (the contraction
// runs over token rows): per stage of 64 tokens each CTA holds its 128 experts
// of the three planes (48 KB) and its half of the slab of u (16 KB); u is
// loaded once for the three planes.  36 accumulation steps (three stages) go
// into one TMEM buffer, then the epilogue warps add it into float32 registers
// (round to nearest): over thousands of tokens the tensor core's truncating
// accumulator alone would cost 1e-5.  Bound by the tensor pipe (three planes).
constexpr int E_STAGES = 3, E_CHUNK = 3;
constexpr int E_A = 3 * 2 * kBox, E_B = 2 * kBox;
using ELay = Layout<E_STAGES, E_A + E_B, 0>;

struct DeParams {
  int T, Tp, N_r, d;
  int nk;                    // Tp / 64
  int n_et, n_slab, S;
  float* C;                  // [S][N_r][d]
  bool wide;
  int* err;
};

__global__ void __launch_bounds__(kThreads, 1)
    router_de_kernel(const __grid_constant__ CUtensorMap tmD,
                     const __grid_constant__ CUtensorMap tmU, const DeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ELay::OFF_BAR);
  uint64_t* empty = full + E_STAGES;
  uint64_t* tfull = empty + E_STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + ELay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + ELay::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const bool is_leader = half == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < E_STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiWarps); }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmD);
    tma_prefetch_desc(&tmU);
  }
  if (warp == 1) {
    tmem2_alloc(tmem_slot, 512);
    tmem2_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = map_shared_to(smem_u32(&full[0]), 0);
  const uint32_t tempty0 = map_shared_to(smem_u32(&tempty[0]), 0);
  const int items = p.n_et * p.n_slab * p.S, step = (int)n_clusters_x();
  const int first = (int)cluster_id_x();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step) {
        const int slab = it % p.n_slab, sl = (it / p.n_slab) % p.S, et = it / p.n_slab / p.S;
        const int e0 = et * 256 + (int)half * 128, c0 = slab * BN + (int)half * 128;
        const int k1 = (int)((long long)(sl + 1) * p.nk / p.S);
        for (int kb = (int)((long long)sl * p.nk / p.S); kb < k1; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          if (is_leader) mbar_arrive_expect_tx(&full[stage], 2u * (E_A + E_B));
          const uint32_t fb = full0 + stage * 8;
          uint8_t* a = smem + stage * (E_A + E_B);
          uint8_t* b = a + E_A;
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(a + (pl * 2 + j) * kBox, &tmD, e0 + 64 * j, pl * p.Tp + kb * BK, fb);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_2d_pair(b + j * kBox, &tmU, c0 + 64 * j, kb * BK, fb);
          if (++stage == E_STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (is_leader)
        for (int s = 0; s < E_STAGES; ++s)
          mbar_wait_bounded(&full[s], ((s < stage) ? phase : phase ^ 1), nullptr, kWaitNs);
    }
  } else if (warp == 1) {
    if (is_leader && lane == 0) {
      const uint32_t idesc = idesc_bf16_f32_major(256, BN, true, true);
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step) {
        const int sl = (it / p.n_slab) % p.S;
        const int k0 = (int)((long long)sl * p.nk / p.S);
        const int k1 = (int)((long long)(sl + 1) * p.nk / p.S);
        for (int c0 = k0; c0 < k1 && ok; c0 += E_CHUNK) {
          if (!mbar_wait_bounded(&tempty[buf], tphase ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          tc_fence_after();
          const int c1 = min(k1, c0 + E_CHUNK);
          for (int kb = c0; kb < c1; ++kb) {
            if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitNs)) {
              raise_abort(abort_flag, p.err);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a0 = smem_u32(smem + stage * (E_A + E_B)), b0 = a0 + E_A;
#pragma unroll
            for (int pl = 2; pl >= 0; --pl)          // the small planes first
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                mma2_f16_ss(tmem_base + buf * BN,
                            smem_desc_mn_sw128(a0 + pl * 2 * kBox + k * 2048, kBox),
                            smem_desc_mn_sw128(b0 + k * 2048, kBox), idesc,
                            (kb > c0 || pl < 2 || k > 0) ? 1u : 0u);
            mma2_commit_mask(&empty[stage], 3);
            if (++stage == E_STAGES) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          mma2_commit_mask(&tfull[buf], 3);
          if (++buf == 2) { buf = 0; tphase ^= 1; }
        }
      }
      mma2_commit_local(mma_done);
      mbar_wait_bounded(mma_done, 0, nullptr, kWaitNs);
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    int buf = 0;
    uint32_t tphase = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += step) {
      const int slab = it % p.n_slab, sl = (it / p.n_slab) % p.S, et = it / p.n_slab / p.S;
      const int k0 = (int)((long long)sl * p.nk / p.S);
      const int k1 = (int)((long long)(sl + 1) * p.nk / p.S);
      float acc[kPieces][16];
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
      for (int c0 = k0; c0 < k1; c0 += E_CHUNK) {
        const bool got = mbar_wait_bounded(&tfull[buf], tphase, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(trow + buf * BN + part * 64 + i * 16, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[i][j] += __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + buf * 8);
        if (++buf == 2) { buf = 0; tphase ^= 1; }
      }
      if (!ok) break;
      const int e = et * 256 + (int)half * 128 + q * 32 + lane;
      if (e < p.N_r) {
        float* out = p.C + ((size_t)sl * p.N_r + e) * p.d;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int c = slab * BN + part * 64 + i * 16;
          if (c < p.d) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(acc[i][8 * v + j]);
              st32(out + c + 8 * v, p.wide, w);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_base, 512);
  }
}

// dE = sum of its S slices, in slice order.
__global__ void __launch_bounds__(256) router_de_join_kernel(const float4* __restrict__ P, int S,
                                                             long long n4,
                                                             float4* __restrict__ dE) {
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += step) {
    float4 a = P[i];
    for (int s = 1; s < S; ++s) {
      const float4 b = P[i + s * n4];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    dE[i] = a;
  }
}

// ---------------------------------------------------------------- du
// A pair owns 256 tokens (128 per CTA) and a run of 256-column slabs.  The
// token rows of both planes (K-major) stay in shared memory for the whole run
// where N_r <= 256 (RES: 128 KB), so a slab streams only its half of E
// (MN-major, 16 KB per 64 experts); otherwise each stage brings both planes'
// rows again.  Two TMEM buffers: the epilogue of a slab (base rows read ahead,
// added in float32, rounded once) runs under the next slab's products.  Bound
// by reading du_base and writing du.
constexpr int U_A = 2 * 128 * BK * 2, U_B = 2 * kBox;       // 32 KB, 16 KB
constexpr int U_RES_BLOCKS = 4;                             // 4 x 64 experts resident
template <bool RES>
struct ULay : Layout<4, RES ? U_B : U_A + U_B, RES ? U_RES_BLOCKS * U_A : 0> {
  static constexpr int STAGES = 4;
  static constexpr int STAGE_BYTES = RES ? U_B : U_A + U_B;
};

struct DuParams {
  int T, Tp, d;
  int nk;                    // ceil(Np / 64)
  int n_tt, n_slab, n_run;   // token tiles, slabs, runs of slabs per token tile
  const __nv_bfloat16* base; // or nullptr
  __nv_bfloat16* du;
  bool wide_in, wide_out;
  int* err;
};

template <bool RES>
__global__ void __launch_bounds__(kThreads, 1)
    router_du_kernel(const __grid_constant__ CUtensorMap tmD,
                     const __grid_constant__ CUtensorMap tmE, const DuParams p) {
  using L = ULay<RES>;
  constexpr int STAGES = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint64_t* afull = mma_done + 1;
  uint64_t* aempty = afull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const bool is_leader = half == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiWarps); }
    mbar_init(mma_done, 1);
    mbar_init(afull, 1);
    mbar_init(aempty, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmD);
    tma_prefetch_desc(&tmE);
  }
  if (warp == 1) {
    tmem2_alloc(tmem_slot, 512);
    tmem2_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = map_shared_to(smem_u32(&full[0]), 0);
  const uint32_t afull0 = map_shared_to(smem_u32(afull), 0);
  const uint32_t tempty0 = map_shared_to(smem_u32(&tempty[0]), 0);
  const int items = p.n_tt * p.n_run, step = (int)n_clusters_x();
  const int first = (int)cluster_id_x();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, seen = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step, ++seen) {
        const int tt = it / p.n_run, run = it % p.n_run;
        const int t0 = tt * 256 + (int)half * 128;
        if (RES) {
          if (!mbar_wait_bounded(aempty, (seen & 1) ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          if (is_leader) mbar_arrive_expect_tx(afull, 2u * (uint32_t)(p.nk * U_A));
          for (int kb = 0; kb < p.nk; ++kb)
            for (int pl = 0; pl < 2; ++pl)
              tma_load_2d_pair(smem + L::OFF_FIXED + kb * U_A + pl * (U_A / 2), &tmD, kb * BK,
                               pl * p.Tp + t0, afull0);
        }
        const int s1 = (int)((long long)(run + 1) * p.n_slab / p.n_run);
        for (int slab = (int)((long long)run * p.n_slab / p.n_run); slab < s1 && ok; ++slab) {
          const int c0 = slab * BN + (int)half * 128;
          for (int kb = 0; kb < p.nk; ++kb) {
            if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitNs)) {
              raise_abort(abort_flag, p.err);
              ok = false;
              break;
            }
            if (is_leader) mbar_arrive_expect_tx(&full[stage], 2u * L::STAGE_BYTES);
            const uint32_t fb = full0 + stage * 8;
            uint8_t* b = smem + stage * L::STAGE_BYTES;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(b + j * kBox, &tmE, c0 + 64 * j, kb * BK, fb);
            if (!RES)
              for (int pl = 0; pl < 2; ++pl)
                tma_load_2d_pair(b + U_B + pl * (U_A / 2), &tmD, kb * BK, pl * p.Tp + t0, fb);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
        }
      }
      // the leader waits until every armed copy has landed
      if (is_leader) {
        for (int s = 0; s < STAGES; ++s)
          mbar_wait_bounded(&full[s], ((s < stage) ? phase : phase ^ 1), nullptr, kWaitNs);
        if (RES && seen > 0) mbar_wait_bounded(afull, (seen - 1) & 1, nullptr, kWaitNs);
      }
    }
  } else if (warp == 1) {
    if (is_leader && lane == 0) {
      const uint32_t idesc = idesc_bf16_f32_major(256, BN, false, true);
      int stage = 0, buf = 0, seen = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step, ++seen) {
        const int run = it % p.n_run;
        if (RES && !mbar_wait_bounded(afull, seen & 1, abort_flag, kWaitNs)) {
          raise_abort(abort_flag, p.err);
          break;
        }
        const int s1 = (int)((long long)(run + 1) * p.n_slab / p.n_run);
        for (int slab = (int)((long long)run * p.n_slab / p.n_run); slab < s1 && ok; ++slab) {
          if (!mbar_wait_bounded(&tempty[buf], tphase ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = 0; kb < p.nk; ++kb) {
            if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitNs)) {
              raise_abort(abort_flag, p.err);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t b0 = smem_u32(smem + stage * L::STAGE_BYTES);
            const uint32_t a0 = RES ? smem_u32(smem + L::OFF_FIXED + kb * U_A) : b0 + U_B;
#pragma unroll
            for (int pl = 1; pl >= 0; --pl)
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                mma2_f16_ss(tmem_base + buf * BN, smem_desc_k_sw128(a0 + pl * (U_A / 2) + k * 32),
                            smem_desc_mn_sw128(b0 + k * 2048, kBox), idesc,
                            (kb > 0 || pl < 1 || k > 0) ? 1u : 0u);
            mma2_commit_mask(&empty[stage], 3);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          mma2_commit_mask(&tfull[buf], 3);
          if (++buf == 2) { buf = 0; tphase ^= 1; }
        }
        if (RES && ok) mma2_commit_mask(aempty, 3);   // the run's products have read the rows
      }
      mma2_commit_local(mma_done);
      mbar_wait_bounded(mma_done, 0, nullptr, kWaitNs);
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    int buf = 0;
    uint32_t tphase = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += step) {
      const int tt = it / p.n_run, run = it % p.n_run;
      const int t = tt * 256 + (int)half * 128 + q * 32 + lane;
      const int s1 = (int)((long long)(run + 1) * p.n_slab / p.n_run);
      for (int slab = (int)((long long)run * p.n_slab / p.n_run); slab < s1; ++slab) {
        const int c0 = slab * BN + part * 64;
        // d is a multiple of 64, so this warp's 64 columns are all inside or all outside
        const bool live = t < p.T && c0 < p.d;
        const size_t at = (size_t)t * p.d + c0;
        uint32_t bs[kPieces][8];
        if (live && p.base) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) ld32(p.base + at + i * 16, p.wide_in, bs[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) bs[i][j] = 0u;
        }
        const bool got = mbar_wait_bounded(&tfull[buf], tphase, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(trow + buf * BN + part * 64 + i * 16, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float lo = __uint_as_float(bs[i][j] << 16) + __uint_as_float(r[2 * j]);
            const float hi = __uint_as_float(bs[i][j] & 0xffff0000u) + __uint_as_float(r[2 * j + 1]);
            const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
            bs[i][j] = *reinterpret_cast<const uint32_t*>(&w);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + buf * 8);
        if (++buf == 2) { buf = 0; tphase ^= 1; }
        if (live) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) st32(p.du + at + i * 16, p.wide_out, bs[i]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_base, 512);
  }
}

template <typename Kern, typename Params>
moe_status launch_pairs(Kern kern, const CUtensorMap& a, const CUtensorMap& b, const Params& p,
                        long long items, int smem, bool* attr_done, const char* what,
                        cudaStream_t s) {
  const moe_status st = ensure_max_smem(reinterpret_cast<const void*>(kern), smem, attr_done, what);
  if (st != MOE_OK) return st;
  const int pairs = sm_count() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(items < pairs ? items : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, a, b, p), what);
}

bool al32(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

// Slices of the tokens for dE: as many as fill the GPU's pairs once, each of
// at least two stages.
int de_slices(int T, int d, int N_r) {
  const int items = (N_r + 255) / 256 * ((d + BN - 1) / BN), nk = (T + BK - 1) / BK;
  int S = kPairs / items;
  if (S > nk / 2) S = nk / 2;
  if (S > 16) S = 16;
  return S < 1 ? 1 : S;
}

}  // namespace

// Planes [3][Tp][Np], then the slices of dE where there is more than one.
RouterPlanes router_planes(int T, int N_r) {
  RouterPlanes r;
  r.Tp = (T + BK - 1) / BK * BK;
  r.Np = (N_r + 7) / 8 * 8;
  r.bytes = align_up((size_t)3 * r.Tp * r.Np * 2, 256);
  return r;
}

size_t router_grad_tc_ws_bytes(int T, int d, int N_r) {
  const int S = de_slices(T, d, N_r);
  return router_planes(T, N_r).bytes + (S > 1 ? align_up((size_t)S * N_r * d * 4, 256) : 0);
}

moe_status launch_router_grad_tc(const void* u, const void* E, int T, int d, int N_r,
                                 const void* du_base, void* du, float* dE, void* ws,
                                 cudaStream_t s) {
  const RouterPlanes pl = router_planes(T, N_r);
  int* err = device_error_word();
  if (!err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tmA, tmB;
  moe_status st;
  {
    DuParams p;
    p.T = T;
    p.Tp = pl.Tp;
    p.d = d;
    p.nk = (pl.Np + BK - 1) / BK;
    p.n_tt = (T + 255) / 256;
    p.n_slab = (d + BN - 1) / BN;
    // runs of slabs per token tile: enough to give every pair one
    p.n_run = kPairs / p.n_tt;
    if (p.n_run > p.n_slab) p.n_run = p.n_slab;
    if (p.n_run < 1) p.n_run = 1;
    p.base = static_cast<const __nv_bfloat16*>(du_base);
    p.du = static_cast<__nv_bfloat16*>(du);
    p.wide_in = al32(du_base);
    p.wide_out = al32(du);
    p.err = err;
    st = make_tmap_2d(&tmA, ws, bf, 2, pl.Np, (uint64_t)3 * pl.Tp, BK, 128);
    if (st != MOE_OK) return st;
    st = make_tmap_2d(&tmB, E, bf, 2, d, N_r, 64, BK);
    if (st != MOE_OK) return st;
    static bool done_r[kMaxSmemDevices] = {}, done_s[kMaxSmemDevices] = {};
    const long long items = (long long)p.n_tt * p.n_run;
    st = p.nk <= U_RES_BLOCKS
             ? launch_pairs(router_du_kernel<true>, tmA, tmB, p, items, ULay<true>::ALLOC, done_r,
                            "router_du launch", s)
             : launch_pairs(router_du_kernel<false>, tmA, tmB, p, items, ULay<false>::ALLOC,
                            done_s, "router_du launch", s);
    if (st != MOE_OK) return st;
  }
  DeParams p;
  p.T = T;
  p.Tp = pl.Tp;
  p.N_r = N_r;
  p.d = d;
  p.nk = pl.Tp / BK;
  p.n_et = (N_r + 255) / 256;
  p.n_slab = (d + BN - 1) / BN;
  p.S = de_slices(T, d, N_r);
  float* part = p.S > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pl.bytes) : dE;
  p.C = part;
  p.wide = al32(part);
  p.err = err;
  st = make_tmap_2d(&tmA, ws, bf, 2, pl.Np, (uint64_t)3 * pl.Tp, 64, BK);
  if (st != MOE_OK) return st;
  st = make_tmap_2d(&tmB, u, bf, 2, d, T, 64, BK);
  if (st != MOE_OK) return st;
  static bool done_e[kMaxSmemDevices] = {};
  st = launch_pairs(router_de_kernel, tmA, tmB, p, (long long)p.n_et * p.n_slab * p.S, ELay::ALLOC,
                    done_e, "router_de launch", s);
  if (st != MOE_OK || p.S == 1) return st;
  const long long n4 = (long long)N_r * d / 4;
  const long long blocks = (n4 + 255) / 256;
  router_de_join_kernel<<<(unsigned)(blocks < 8 * sm_count() ? blocks : 8 * sm_count()), 256, 0,
                          s>>>(reinterpret_cast<const float4*>(part), p.S, n4,
                               reinterpret_cast<float4*>(dE));
  return cuda_check(cudaGetLastError(), "router_de_join launch");
}

}  // namespace moe
