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

// Barriers: full, empty per stage, tfull[2], tempty[2], mma_done, afull, aempty,
// one for each epilogue warp's patch.
template <int STAGES, int STAGE_BYTES, int FIXED_BYTES>
struct Layout {
  static constexpr int OFF_FIXED = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_FIXED + FIXED_BYTES;
  static constexpr int N_BARS = 2 * STAGES + 7 + kEpiWarps;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
};

__device__ __forceinline__ void raise_abort(volatile int* abort, int* err) {
  *abort = 1;
  atomicOr(err, ERR_GEMM_TIMEOUT);
}

// ---------------------------------------------------------------- dE
// A tile is 256 experts (128 rows of C per CTA of a pair) x a slab of 256
// columns; its work is one unit for each 64 tokens.  The units of all tiles,
// in order, are dealt to the pairs in equal runs, so every pair is busy to the
// end whatever the number of tiles; a run's part of a tile is a segment, kept
// as a float32 [256][256] block numbered pair + tile (either number grows
// along the units, so the blocks are distinct), and router_de_join_kernel adds
// a tile's segments in order.  Both operands are MN-major (the contraction
// runs over token rows): per stage of 64 tokens each CTA holds its 128 experts
// of the three planes (48 KB) and its half of the slab of u (16 KB); u is
// loaded once for the three planes.  36 accumulation steps (three stages) go
// into one TMEM buffer, then the epilogue warps add it into float32 registers
// (round to nearest): over thousands of tokens the tensor core's truncating
// accumulator alone would cost 1e-5.  Bound by the tensor pipe (three planes):
// T 8192, d 7168, 256 experts 64 us with the pipe 72 % busy.
constexpr int E_STAGES = 3, E_CHUNK = 3;
constexpr int E_A = 3 * 2 * kBox, E_B = 2 * kBox;
using ELay = Layout<E_STAGES, E_A + E_B, 0>;

struct DeParams {
  int T, Tp, N_r, d;
  int nk;                    // Tp / 64
  int n_et, n_slab, n_pairs;
  float* C;                  // segments [n_pairs + tiles][256][256]
  int* err;
};

// Column col (a multiple of 4) of a segment's row: [row / 32][col / 8][32][8], so
// that the 32 bytes which a lane (one row) writes at a time lie side by side
// over the warp.
__device__ __forceinline__ size_t seg_at(int seg, int row, int col) {
  return (size_t)seg * 256 * BN + (row >> 5) * (32 * BN) + (col >> 3) * 256 + (row & 31) * 8 +
         (col & 7);
}

// First unit of pair c of P over U units.
__host__ __device__ __forceinline__ int first_unit(int c, int P, int U) {
  return (int)((long long)c * U / P);
}

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
  pdl_wait();                  // d_logit's planes; the setup above overlaps their kernel
  pdl_trigger();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = map_shared_to(smem_u32(&full[0]), 0);
  const uint32_t tempty0 = map_shared_to(smem_u32(&tempty[0]), 0);
  const int pair = (int)cluster_id_x(), units = p.n_et * p.n_slab * p.nk;
  const int u0 = first_unit(pair, p.n_pairs, units), u1 = first_unit(pair + 1, p.n_pairs, units);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int un = u0; un < u1 && ok;) {
        const int tile = un / p.nk, slab = tile % p.n_slab, et = tile / p.n_slab;
        const int e0 = et * 256 + (int)half * 128, c0 = slab * BN + (int)half * 128;
        const int end = min(u1, (tile + 1) * p.nk);
        for (; un < end; ++un) {
          const int kb = un - tile * p.nk;
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
      for (int un = u0; un < u1 && ok;) {
        const int k1 = min(u1, (un / p.nk + 1) * p.nk);      // the segment's end
        for (int c0 = un; c0 < k1 && ok; c0 += E_CHUNK) {
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
        un = k1;
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
    for (int un = u0; un < u1 && ok;) {
      const int tile = un / p.nk, k0 = un, k1 = min(u1, (tile + 1) * p.nk);
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
      // experts past N_r are zero rows: not kept
      const int row = (int)half * 128 + q * 32 + lane;
      if (tile / p.n_slab * 256 + row < p.N_r) {
        float* out = p.C + seg_at(pair + tile, row, part * 64);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          st_global_v8(out + i * 512, &acc[i][0]);
          st_global_v8(out + i * 512 + 256, &acc[i][8]);
        }
      }
      un = k1;
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

// Adds a tile's segments in order: a block per tile and kJoinRows of its rows;
// a warp takes all of the rows by 16 columns, so that it reads runs of 256 bytes.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(256) router_de_join_kernel(const float* __restrict__ C, int P,
                                                             int nk, int n_slab, int units,
                                                             int N_r, int d,
                                                             float* __restrict__ dE) {
  __shared__ int s_c0, s_c1;
  pdl_wait();
  const int tile = blockIdx.x, slab = tile % n_slab, e0 = tile / n_slab * 256;
  if (threadIdx.x == 0) {
    // the pairs whose runs meet the tile's units
    int c0 = (int)((long long)tile * nk * P / units);
    while (c0 > 0 && first_unit(c0, P, units) > tile * nk) --c0;
    while (first_unit(c0 + 1, P, units) <= tile * nk) ++c0;
    int c1 = c0 + 1;
    while (c1 < P && first_unit(c1, P, units) < (tile + 1) * nk) ++c1;
    s_c0 = c0;
    s_c1 = c1;
  }
  __syncthreads();
  const int c0 = s_c0, c1 = s_c1, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinRows + ((lane >> 1) & 7);
  if (e0 + row >= N_r) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int col = (threadIdx.x >> 5) * 16 + k * 128 + (lane >> 4) * 8 + (lane & 1) * 4;
    if (slab * BN + col >= d) continue;
    const float* src = C + seg_at(c0 + tile, row, col);
    float4 a = *reinterpret_cast<const float4*>(src);
#pragma unroll 4
    for (int c = c0 + 1; c < c1; ++c) {
      src += 256 * BN;
      const float4 b = *reinterpret_cast<const float4*>(src);
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    *reinterpret_cast<float4*>(dE + (size_t)(e0 + row) * d + slab * BN + col) = a;
  }
}

// ---------------------------------------------------------------- du
// A pair owns 256 tokens (128 per CTA) and a run of 256-column slabs.  The
// token rows of both planes (K-major) stay in shared memory for the whole run
// where N_r <= 256 (RES: 128 KB), so a slab streams only its half of E
// (MN-major, 8 KB per 32 experts); otherwise each stage brings both planes'
// rows again (64 experts).  Two TMEM buffers: the epilogue of a slab runs under the next
// slab's products.  Each epilogue warp owns a [32 tokens][64 columns] patch
// (128-byte swizzle): TMA brings the base values, the warp adds its float32
// sums, rounds once and writes them back in place, TMA takes them out; the
// next slab's patch is fetched while its sums are being made.  At T 8192, d
// 7168, N_r 256 this takes 71 us (61 without a base): what holds it back is the
// pair's round trip for a stage of E (commit, both producers, L2, the leader's
// barrier: some 3600 cycles against the 2048 tensor cycles in the ring).
// Measured instead: a ring twice as large leaves room for patches of 2 KB
// only, 52 us without a base but 80 with one; row accesses straight from the
// lanes touch 32 lines an instruction, 82 us.
constexpr int U_A = 2 * 128 * BK * 2;                       // both planes' rows of 64 experts
constexpr int U_RES_BLOCKS = 4;                             // 4 x 64 experts resident
template <bool RES>
struct ULay : Layout<RES ? 4 : 3, RES ? kBox : U_A + 2 * kBox,
                     (RES ? U_RES_BLOCKS * U_A : 0) + kEpiWarps * 4096> {
  static constexpr int STAGES = RES ? 4 : 3;
  static constexpr int KB = RES ? 32 : 64;                  // experts per stage
  static constexpr int B_BOX = KB * 128;                    // [KB][64 columns]
  static constexpr int STAGE_BYTES = RES ? kBox : U_A + 2 * kBox;
  static constexpr int OFF_PATCH = ULay::OFF_FIXED + (RES ? U_RES_BLOCKS * U_A : 0);
};

struct DuParams {
  int T, Tp, d;
  int nk, n_stage;           // blocks of 64 experts; stages of L::KB experts
  int n_tt, n_slab, n_run;   // token tiles, slabs, runs of slabs per token tile
  bool base;                 // tmBase is read
  int* err;
};

template <bool RES>
__global__ void __launch_bounds__(kThreads, 1)
    router_du_kernel(const __grid_constant__ CUtensorMap tmD,
                     const __grid_constant__ CUtensorMap tmE,
                     const __grid_constant__ CUtensorMap tmBase,
                     const __grid_constant__ CUtensorMap tmOut, const DuParams p) {
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
  uint64_t* pbar = aempty + 1;
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
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&pbar[w], 1);
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
  pdl_wait();                  // d_logit's planes; the setup above overlaps their kernel
  pdl_trigger();
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
          for (int kb = 0; kb < p.n_stage; ++kb) {
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
              tma_load_2d_pair(b + j * L::B_BOX, &tmE, c0 + 64 * j, kb * L::KB, fb);
            if (!RES)
              for (int pl = 0; pl < 2; ++pl)
                tma_load_2d_pair(b + 2 * L::B_BOX + pl * (U_A / 2), &tmD, kb * L::KB,
                                 pl * p.Tp + t0, fb);
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
          for (int kb = 0; kb < p.n_stage; ++kb) {
            if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitNs)) {
              raise_abort(abort_flag, p.err);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t b0 = smem_u32(smem + stage * L::STAGE_BYTES);
            // RES: the second stage of a 64-expert block starts 64 bytes into its rows
            const uint32_t a0 = RES ? smem_u32(smem + L::OFF_FIXED + (kb >> 1) * U_A) + (kb & 1) * 64
                                    : b0 + 2 * L::B_BOX;
#pragma unroll
            for (int pl = 1; pl >= 0; --pl)
#pragma unroll
              for (int k = 0; k < L::KB / 16; ++k)
                mma2_f16_ss(tmem_base + buf * BN, smem_desc_k_sw128(a0 + pl * (U_A / 2) + k * 32),
                            smem_desc_mn_sw128(b0 + k * 2048, L::B_BOX), idesc,
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
    uint4* patch = reinterpret_cast<uint4*>(smem + L::OFF_PATCH + (warp - 2) * 4096);   // [32][8]
    uint64_t* pb = &pbar[warp - 2];
    int buf = 0;
    uint32_t tphase = 0, pphase = 0;
    bool ok = true, armed = false;
    const auto row_of = [&](int it) { return it / p.n_run * 256 + (int)half * 128 + q * 32; };
    const auto slab0 = [&](int it) { return (int)((long long)(it % p.n_run) * p.n_slab / p.n_run); };
    const auto slab1 = [&](int it) { return (int)((long long)(it % p.n_run + 1) * p.n_slab / p.n_run); };
    // d is a multiple of 64: a patch's columns are all inside or all outside
    const auto live = [&](int it, int c) { return row_of(it) < p.T && c < p.d; };
    // fetches a slab's base values (the store out of the patch has to have read it)
    const auto fetch = [&](int it, int slab) {
      const int c = slab * BN + part * 64;
      if (!p.base || !live(it, c)) return;
      if (lane == 0) {
        tma_store_wait_read_all();
        mbar_arrive_expect_tx(pb, 4096);
        tma_load_2d(patch, &tmBase, c, row_of(it), pb);
      }
      armed = true;
    };
    if (first < items) fetch(first, slab0(first));
    for (int it = first; it < items && ok; it += step) {
      const int s1 = slab1(it);
      for (int slab = slab0(it); slab < s1; ++slab) {
        const bool got = mbar_wait_bounded(&tfull[buf], tphase, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld_32x32b_x32(trow + buf * BN + part * 64, r[0]);
        tmem_ld_32x32b_x32(trow + buf * BN + part * 64 + 32, r[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + buf * 8);
        if (++buf == 2) { buf = 0; tphase ^= 1; }
        const int c = slab * BN + part * 64;
        if (live(it, c)) {
          if (p.base) {
            const bool in = mbar_wait_bounded(pb, pphase, abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, in)) {
              if (lane == 0) raise_abort(abort_flag, p.err);
              ok = false;
              break;
            }
            pphase ^= 1;
            armed = false;
          } else {
            if (lane == 0) tma_store_wait_read_all();
            __syncwarp();
          }
          // row `lane`: 16-byte slot i sits at i ^ (row & 7)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4* at = patch + lane * 8 + (i ^ (lane & 7));
            float f[8];
            Vec<__nv_bfloat16>::load(p.base ? *at : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += __uint_as_float(r[i >> 2][8 * (i & 3) + j]);
            *at = Vec<__nv_bfloat16>::store(f);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, patch, c, row_of(it));
            tma_store_commit();
          }
        }
        if (slab + 1 < s1) fetch(it, slab + 1);
        else if (it + step < items) fetch(it + step, slab0(it + step));
      }
    }
    // no copy may still use shared memory when the CTA leaves
    if (armed) mbar_wait_bounded(pb, pphase, nullptr, kWaitNs);
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_base, 512);
  }
}

template <typename... Params, typename... Args>
moe_status launch_pairs(void (*kern)(Params...), long long pairs, int smem, bool* attr_done,
                        const char* what, cudaStream_t s, const Args&... args) {
  const moe_status st = ensure_max_smem(reinterpret_cast<const void*>(kern), smem, attr_done, what);
  if (st != MOE_OK) return st;
  return launch_after(kern, dim3(2 * (unsigned)pairs), dim3(kThreads), smem, s, 2, what, args...);
}

// Pairs that share dE's units: all of the GPU's, but none with fewer than two.
int de_pairs(int T, int d, int N_r) {
  const long long units = (long long)((N_r + 255) / 256) * ((d + BN - 1) / BN) *
                          ((T + BK - 1) / BK);
  const long long most = units < 2 ? 1 : units / 2;
  return (int)(most < kPairs ? most : kPairs);
}

}  // namespace

// Planes [3][Tp][Np], then the segments of dE.
RouterPlanes router_planes(int T, int N_r) {
  RouterPlanes r;
  r.Tp = (T + BK - 1) / BK * BK;
  r.Np = (N_r + 7) / 8 * 8;
  r.bytes = align_up((size_t)3 * r.Tp * r.Np * 2, 256);
  return r;
}

size_t router_grad_tc_ws_bytes(int T, int d, int N_r) {
  const size_t tiles = (size_t)((N_r + 255) / 256) * ((d + BN - 1) / BN);
  return router_planes(T, N_r).bytes + (de_pairs(T, d, N_r) + tiles) * 256 * BN * 4;
}

moe_status launch_router_grad_tc(const void* u, const void* E, int T, int d, int N_r,
                                 const void* du_base, void* du, float* dE, void* ws,
                                 cudaStream_t s) {
  const RouterPlanes pl = router_planes(T, N_r);
  int* err = device_error_word();
  if (!err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tmA, tmB, tmBase, tmOut;
  moe_status st;
  {
    DuParams p;
    p.T = T;
    p.Tp = pl.Tp;
    p.d = d;
    p.nk = (pl.Np + BK - 1) / BK;
    const bool res = p.nk <= U_RES_BLOCKS;
    const int kb = res ? ULay<true>::KB : ULay<false>::KB;
    p.n_stage = (pl.Np + kb - 1) / kb;
    p.n_tt = (T + 255) / 256;
    p.n_slab = (d + BN - 1) / BN;
    // runs of slabs per token tile: enough to give every pair one
    p.n_run = kPairs / p.n_tt;
    if (p.n_run > p.n_slab) p.n_run = p.n_slab;
    if (p.n_run < 1) p.n_run = 1;
    p.base = du_base != nullptr;
    p.err = err;
    st = make_tmap_2d(&tmA, ws, bf, 2, pl.Np, (uint64_t)3 * pl.Tp, BK, 128);
    if (st == MOE_OK) st = make_tmap_2d(&tmB, E, bf, 2, d, N_r, 64, kb);
    if (st == MOE_OK) st = make_tmap_2d(&tmOut, du, bf, 2, d, T, 64, 32);
    if (st == MOE_OK) st = make_tmap_2d(&tmBase, du_base ? du_base : du, bf, 2, d, T, 64, 32);
    if (st != MOE_OK) return st;
    static bool done_r[kMaxSmemDevices] = {}, done_s[kMaxSmemDevices] = {};
    const long long items = (long long)p.n_tt * p.n_run;
    const long long pairs = items < kPairs ? items : kPairs;
    st = res ? launch_pairs(router_du_kernel<true>, pairs, ULay<true>::ALLOC, done_r,
                            "router_du launch", s, tmA, tmB, tmBase, tmOut, p)
             : launch_pairs(router_du_kernel<false>, pairs, ULay<false>::ALLOC, done_s,
                            "router_du launch", s, tmA, tmB, tmBase, tmOut, p);
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
  p.n_pairs = de_pairs(T, d, N_r);
  p.C = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pl.bytes);
  p.err = err;
  st = make_tmap_2d(&tmA, ws, bf, 2, pl.Np, (uint64_t)3 * pl.Tp, 64, BK);
  if (st == MOE_OK) st = make_tmap_2d(&tmB, u, bf, 2, d, T, 64, BK);
  if (st != MOE_OK) return st;
  static bool done_e[kMaxSmemDevices] = {};
  st = launch_pairs(router_de_kernel, p.n_pairs, ELay::ALLOC, done_e, "router_de launch", s, tmA,
                    tmB, p);
  if (st != MOE_OK) return st;
  const int rows = N_r < 256 ? N_r : 256;
  const dim3 grid(p.n_et * p.n_slab, (rows + kJoinRows - 1) / kJoinRows);
  return launch_after(router_de_join_kernel, grid, dim3(256), 0, s, 1, "router_de_join launch", p.C,
                      p.n_pairs, p.nk, p.n_slab, p.n_et * p.n_slab * p.nk, N_r, d, dE);
}

}  // namespace moe
