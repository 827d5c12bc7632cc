// Grouped weight-gradient GEMM on tcgen05 CTA pairs: for every expert g with
// token rows [off_g, off_g+1),
//   C_g[m, n] = sum over those rows r of A[r, m] * B[r, n]     (bf16 in and out)
// Both operands are MN-major (the contraction runs over rows).
//
// Tile: 256 x 256 of C per pair (128 rows of C per CTA, each CTA staging its
// 128 columns of A and half the columns of B), 64 token rows per stage, five
// stages of 32 KB per CTA; two TMEM accumulators of 256 columns, so the
// epilogue of one tile runs under the products of the next.  A pair streams
// two thirds of the bytes per product of one CTA's 128 x 256 tile.
//
// A group's last rows need not fill a stage.  The rows past its end belong to
// the next group or to none, and may hold anything (0 x NaN is NaN), so they
// are cleared in shared memory, up to the next 16 rows, before their products
// run, and only those 16-row steps are issued.  The rows of such a part stage
// go to a buffer of their own, which a warp of each CTA fills and clears while
// the tile's whole stages run; the leader multiplies it last.  Cleared inside
// the ring of stages instead, the extra latency showed in every tile: 8 groups
// of 500 rows, gradient 4096 x 7168: 309 us, with the buffer 223.
//
// Measured at that gradient's 4096 rows: 8 equal groups 216 us (1.1 PFLOP/s),
// ragged groups (1059, 1, 1104, 235, 586, 1109, 0 and 2 rows) 252: those of a
// few rows are bound by writing C.  Longer groups add 185 us per 4096 rows
// (1.3 PFLOP/s); what equal groups spend beyond it is the 470 MB of C, which
// take 125 us at the rate of a plain fill (3.7 TB/s) and are written under the
// products only in part.  Tiles in group order; spread over all groups, so
// that short ones write while long ones multiply, they cost 260 and 232 us:
// the operands of all the groups then compete for L2.
//
// Roles: warp 0 TMA producer, warp 1 TMEM allocation and (leader) MMA issuer,
// warps 2-17 epilogue (a [32][32] patch each, written out by TMA), warp 18 the
// part stages.  Every wait is bounded (1 s) and reported through the device
// error word.
#include "launch.h"
#include "sm100.cuh"

namespace moe {

moe_status make_tmap_2d(CUtensorMap* tm, const void* base, CUtensorMapDataType dtype,
                        int elem_bytes, uint64_t inner, uint64_t outer, uint32_t box_inner,
                        uint32_t box_outer);
moe_status make_tmap_2d_swz(CUtensorMap* tm, const void* base, CUtensorMapDataType dtype,
                            int elem_bytes, uint64_t inner, uint64_t outer, uint32_t box_inner,
                            uint32_t box_outer, CUtensorMapSwizzle swz);

namespace {

using namespace sm100;

constexpr int BT = 256;                        // rows and columns of C per pair
constexpr int BK = 64;                         // token rows per stage
constexpr int STAGES = 5;
constexpr int kBox = 64 * BK * 2;              // [64 tokens][64 columns]: 8 KB
constexpr int STAGE_BYTES = 4 * kBox;          // A: two boxes, B: two boxes
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (2 + kEpiWarps + 1);
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int OFF_TAIL = STAGES * STAGE_BYTES;
constexpr int OFF_PATCH = OFF_TAIL + STAGE_BYTES;
constexpr int OFF_BAR = OFF_PATCH + kEpiWarps * 2048;
constexpr int N_BARS = 2 * STAGES + 8;   // full, empty, tfull[2], tempty[2], done, tail, cleared, tail_free
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int SMEM_ALLOC = OFF_MISC + 16 + 1024;

struct WgPairParams {
  const int32_t* offsets;   // [G+1] or nullptr
  int G, rows, M, N;
  __nv_bfloat16* C;         // [G, M, N]
  int* err;
};

__device__ __forceinline__ void raise_abort(volatile int* abort, int* err) {
  *abort = 1;
  atomicOr(err, ERR_GEMM_TIMEOUT);
}

__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmC, const WgPairParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint64_t* tail = mma_done + 1;               // this CTA's copies of a group's last rows
  uint64_t* cleared = tail + 1;                // leader: both CTAs have cleared the rows past them
  uint64_t* tail_free = cleared + 1;           // their products are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const bool is_leader = half == 0;
  const int n_n = p.N / BT, per_group = p.M / BT * n_n, total = p.G * per_group;
  const int first = (int)cluster_id_x(), step = (int)n_clusters_x();

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tail, 1);
    mbar_init(cleared, 2);
    mbar_init(tail_free, 1);
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiWarps); }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem2_alloc(tmem_slot, 512);
    tmem2_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  pdl_wait();                  // the operands; the setup above overlaps the kernel before
  pdl_trigger();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = map_shared_to(smem_u32(&full[0]), 0);
  const uint32_t tempty0 = map_shared_to(smem_u32(&tempty[0]), 0);
  const uint32_t cleared0 = map_shared_to(smem_u32(cleared), 0);
  // Rows [r0, r0 + cnt) of the tile's group, inside [0, rows).
  const auto group_rows = [&](int t, int& r0, int& cnt) {
    int r1;
    clamp_group_rows(p.offsets, t / per_group, p.rows, p.err, r0, r1);
    cnt = r1 - r0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const int loc = t % per_group;
        const int m0 = loc / n_n * BT + (int)half * 128, n0 = loc % n_n * BT + (int)half * 128;
        int r0, cnt;
        group_rows(t, r0, cnt);
        for (int k = 0; k + BK <= cnt; k += BK) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          uint8_t* dst = smem + stage * STAGE_BYTES;
          if (is_leader) mbar_arrive_expect_tx(&full[stage], 2u * STAGE_BYTES);
          const uint32_t fb = full0 + stage * 8;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tma_load_2d_pair(dst + j * kBox, &tmA, m0 + 64 * j, r0 + k, fb);
            tma_load_2d_pair(dst + (2 + j) * kBox, &tmB, n0 + 64 * j, r0 + k, fb);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      // every armed stage's copies have landed
      if (is_leader)
        for (int s = 0; s < STAGES; ++s)
          mbar_wait_bounded(&full[s], ((s < stage) ? phase : phase ^ 1), nullptr, kWaitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (pair leader)
    if (is_leader && lane == 0) {
      const uint32_t idesc = idesc_bf16_f32_major(BT, BT, true, true);
      int stage = 0, used = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        int r0, cnt;
        group_rows(t, r0, cnt);
        if (cnt <= 0) continue;
        const int ab = used & 1;
        if (!mbar_wait_bounded(&tempty[ab], ((used >> 1) & 1) ^ 1, abort_flag, kWaitNs)) {
          raise_abort(abort_flag, p.err);
          break;
        }
        ++used;
        tc_fence_after();
        const auto products = [&](const uint8_t* src, int k) {
          const uint32_t a0 = smem_u32(src), b0 = a0 + 2 * kBox;
          const int nks = (min(BK, cnt - k) + 15) / 16;
          for (int i = 0; i < nks; ++i)
            mma2_f16_ss(tmem_base + ab * BT, smem_desc_mn_sw128(a0 + i * 2048, kBox),
                        smem_desc_mn_sw128(b0 + i * 2048, kBox), idesc, (k | i) != 0 ? 1u : 0u);
        };
        int k = 0;
        for (; k + BK <= cnt; k += BK) {
          if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          products(smem + stage * STAGE_BYTES, k);
          mma2_commit_mask(&empty[stage], 3);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (ok && k < cnt) {
          ok = mbar_wait_cluster_bounded(cleared, tphase, abort_flag, kWaitNs);
          tphase ^= 1;
          if (ok) {
            tc_fence_after();
            products(smem + OFF_TAIL, k);
            mma2_commit_mask(tail_free, 3);
          }
        }
        if (!ok) raise_abort(abort_flag, p.err);
        if (!ok) break;
        mma2_commit_mask(&tfull[ab], 3);
      }
      mma2_commit_local(mma_done);
      mbar_wait_bounded(mma_done, 0, nullptr, kWaitNs);
    }
  } else if (warp == 2 + kEpiWarps) {
    // ------------------------------------------------------------ part stages (both CTAs)
    uint32_t phase = 0;
    for (int t = first; t < total; t += step) {
      int r0, cnt;
      group_rows(t, r0, cnt);
      const int valid = cnt % BK;
      if (!valid) continue;
      uint8_t* dst = smem + OFF_TAIL;
      bool got = mbar_wait_bounded(tail_free, phase ^ 1, abort_flag, kWaitNs);
      if (__all_sync(0xffffffffu, got)) {
        if (lane == 0) {
          const int loc = t % per_group;
          const int m0 = loc / n_n * BT + (int)half * 128, n0 = loc % n_n * BT + (int)half * 128;
          const int row = r0 + cnt - valid;
          mbar_arrive_expect_tx(tail, STAGE_BYTES);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tma_load_2d(dst + j * kBox, &tmA, m0 + 64 * j, row, tail);
            tma_load_2d(dst + (2 + j) * kBox, &tmB, n0 + 64 * j, row, tail);
          }
        }
        __syncwarp();
        // copies in flight end before the CTA does, so this wait heeds no abort
        got = mbar_wait_bounded(tail, phase, nullptr, kWaitNs);
      }
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) raise_abort(abort_flag, p.err);
        break;
      }
      phase ^= 1;
      // rows valid .. up to the next 16 of the four boxes (a row is 128 bytes
      // whatever its swizzle)
      const int bytes = ((valid + 15) / 16 * 16 - valid) * 128;
#pragma unroll
      for (int bx = 0; bx < 4; ++bx)
        for (int i = lane * 16; i < bytes; i += 512)
          *reinterpret_cast<uint4*>(dst + bx * kBox + valid * 128 + i) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(cleared0);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, cq = (warp - 2) >> 2;
    uint4* patch = reinterpret_cast<uint4*>(smem + OFF_PATCH + (warp - 2) * 2048);   // [32][4]
    int used = 0;
    for (int t = first; t < total; t += step) {
      const int loc = t % per_group;
      const int row = t / per_group * p.M + loc / n_n * BT + (int)half * 128 + q * 32;
      const int col = loc % n_n * BT + cq * 64;
      int r0, cnt;
      group_rows(t, r0, cnt);
      uint32_t r[2][32] = {};                                // a group of no rows: zero
      if (cnt > 0) {
        const int ab = used & 1;
        const bool got = mbar_wait_bounded(&tfull[ab], (used >> 1) & 1, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          break;
        }
        ++used;
        tc_fence_after();
        const uint32_t tl = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + ab * BT + cq * 64;
        tmem_ld_32x32b_x32(tl, r[0]);
        tmem_ld_32x32b_x32(tl + 32, r[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + ab * 8);   // sums read
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (lane == 0) tma_store_wait_read_all();              // the last box has been read
        __syncwarp();
        // 16-byte slot i of row r sits at i ^ ((r >> 1) & 3) (64-byte swizzle)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r[c][8 * i + k]);
          patch[lane * 4 + (i ^ ((lane >> 1) & 3))] = Vec<__nv_bfloat16>::store(f);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmC, patch, col + 32 * c, row);
          tma_store_commit();
        }
      }
    }
    if (lane == 0) tma_store_wait_all();                     // stores done before the CTA leaves
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // no CTA leaves while the other may use its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_base, 512);
  }
}

}  // namespace

moe_status launch_wgrad_pair(const void* A, int M, const void* B, int N, const int32_t* offsets,
                         int n_groups, int rows, void* C, cudaStream_t s) {
  const int G = offsets ? n_groups : 1;
  if (M % BT || N % BT)
    return fail(MOE_ERR_UNSUPPORTED, "wgrad_pair: M=%d and N=%d must be multiples of %d", M, N, BT);
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tmA, tmB, tmC;
  moe_status st = make_tmap_2d(&tmA, A, bf, 2, M, rows, 64, BK);
  if (st == MOE_OK) st = make_tmap_2d(&tmB, B, bf, 2, N, rows, 64, BK);
  if (st == MOE_OK)
    st = make_tmap_2d_swz(&tmC, C, bf, 2, N, (uint64_t)G * M, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != MOE_OK) return st;
  static bool attr_done[kMaxSmemDevices] = {};
  st = ensure_max_smem(reinterpret_cast<const void*>(wgrad_pair_kernel), SMEM_ALLOC, attr_done,
                       "wgrad_pair smem attribute");
  if (st != MOE_OK) return st;
  WgPairParams p;
  p.offsets = offsets;
  p.G = G;
  p.rows = rows;
  p.M = M;
  p.N = N;
  p.C = static_cast<__nv_bfloat16*>(C);
  p.err = device_error_word();
  if (!p.err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const long long tiles = (long long)G * (M / BT) * (N / BT);
  const int sms = sm_count() / 2, pairs = tiles < sms ? (int)tiles : sms;
  return launch_after(wgrad_pair_kernel, dim3(2 * (unsigned)pairs),
                      dim3(kThreads), SMEM_ALLOC, s, 2, "wgrad_pair launch", tmA, tmB, tmC, p);
}

}  // namespace moe
