// Scored router (moe_route_scored): softmax or sigmoid scores of u E^T, biased
// and group-limited top-K, gates, load.
//
// Logits come as S partial sums over slices of d, [S][T][ld]:
//   float32 inputs: float64 on the tensor cores' float64 pipe (router_logits64_kernel);
//   few bf16 tokens: float64, a block per expert (router_logits_few_kernel);
//   else bf16 on tcgen05 CTA pairs, float32 (router_logits_tc_kernel).
// A block or a warp per token joins the slices and routes (router_select.cuh).
// From float64 logits the keys are the definition's; from float32 ones a
// decision too close for them is made again from float64 logits of the experts
// that can take part in it: by the token's block, or, where warps route, by a
// block for each token that they listed (router_token_kernel).
//
// Every wait is bounded (1 s of %globaltimer) and reported through the device
// error word.
#include "launch.h"
#include "router_select.cuh"
#include "sm100.cuh"

namespace moe {

moe_status make_tmap_2d(CUtensorMap* tm, const void* base, CUtensorMapDataType dtype,
                        int elem_bytes, uint64_t inner, uint64_t outer, uint32_t box_inner,
                        uint32_t box_outer);

namespace {

using namespace sm100;

// ---------------------------------------------------------------- tensor-core logits
// A CTA pair (cta_group::2) owns 256 tokens x Nt <= 256 experts x one slice of
// d: each CTA stages its 128 token rows (the MMA's M side) and half of the
// experts, so the pair streams each centroid byte once.  The token side is
// read once from memory.  T 8192, d 7168, 256 experts: 54 us, u at 2.2 TB/s.
// Some 9 us of it are there at any size (TMEM and barriers 1, first loads 1.5
// to 2.5, last products and drain 1.5, stores 3, exit 1).
//
// The tensor core adds into its accumulator with truncation, and what a step
// loses follows the largest of its products and running sums, not the logit.
// The sum is therefore cut every kChunk blocks (8 accumulation steps): two TMEM
// buffers take turns, and the epilogue warps add each finished chunk into float32
// registers (round to nearest) while the next one runs.  A buffer's round trip
// through the pair's barriers stalls the products of short chunks (chunks of 2, 4,
// 6 and 8 blocks take 54, 41, 39 and 38 us), but the error bound, and with it the
// tokens that are decided again, grows with the chunk: the whole call takes 117 us
// with 2 and 120 with 4.
//
// |u| |E| bounds every product and running sum, and with it the logits' error
// (logit_error in router_select.cuh).  Two warps sum the tokens' squares from each
// stage in shared memory once its products are done (5 us); then it is free.  The
// experts' are summed by the epilogue warps from global memory before the first
// products are done.
constexpr int BK = 64;                 // bf16 K elements per 128-byte swizzle row
constexpr int TM = 128;                // token rows per CTA (TMEM lanes)
constexpr int kMaxN = 256;
constexpr int kChunk = 2;
constexpr int STAGES = 6;              // of a block each
constexpr int kEpiWarps = 16;          // four per TMEM lane quarter, 16-column pieces in turn
constexpr int kSqWarps = 2;            // square sums
constexpr int kTcThreads = 64 + 32 * (kEpiWarps + kSqWarps);
constexpr int kPieces = kMaxN / 16 / (kEpiWarps / 4);
constexpr int kMaxE2 = 1024 / kEpiWarps;   // blocks that sum experts' squares
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int A_BOX = TM * BK * 2, B_BOX = (kMaxN / 2) * BK * 2;
constexpr int OFF_B = STAGES * A_BOX;
constexpr int OFF_BAR = OFF_B + STAGES * B_BOX;
constexpr int N_BARS = 3 * STAGES + 5;   // full, used, empty, tfull[2], tempty[2], mma_done
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int OFF_EMAX = OFF_MISC + 16;          // an epilogue warp's largest square sum each
constexpr int SMEM_BYTES = OFF_EMAX + kEpiWarps * 4;
static_assert(OFF_BAR % 8 == 0, "barriers");
constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;

// Partial logits of the tensor-core path: groups of 32 tokens, [ld / 8][32][8]
// each, so that the 32 bytes which a lane (one token) writes at a time lie side
// by side over the warp: in rows of ld every store touches 32 lines, 1.5 us
// more whatever T.
__host__ __device__ __forceinline__ int token_groups(int T) { return T / 32 + (T % 32 != 0); }
__host__ __device__ __forceinline__ size_t slice_stride(int T, int ld) {
  return (size_t)token_groups(T) * 32 * ld;
}
__device__ __forceinline__ size_t tc_row(int t, int ld) {
  return (size_t)(t >> 5) * 32 * ld + (t & 31) * 8;
}
__device__ __forceinline__ int tc_col(int e) { return (e >> 3) * 256 + (e & 7); }

struct LogitParams {
  int T, N_r, nk, S;
  int n_tt, n_et, Nt;       // token tiles of 256, expert tiles of Nt
  int ld;                   // n_et * Nt
  float* P;                 // S slices of groups of 32 tokens (tc_row)
  const __nv_bfloat16* E;
  int d;
  float* u2;                // square sums of the tokens' slices: [S][whole groups of 32 tokens]
  float* e2;                // [n_e2]: the largest square sum of a block's experts
  int n_e2;
  int32_t* counts;          // zeroed here, as is the listing's length
  int32_t* n_listed;        // two lengths
  int* err;
};

__device__ __forceinline__ void raise_abort(volatile int* abort, int* err) {
  *abort = 1;
  atomicOr(err, ERR_GEMM_TIMEOUT);
}

// Adds the squares of eight bf16 values to s and their bits to any.  Four squares
// are added in bf16 (at most three roundings of 2^-8: s is a bound's scale).
__device__ __forceinline__ void add_squares(const uint4& v, float& s, uint32_t& any) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
  __nv_bfloat162 a = __hmul2(h[0], h[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) a = __hfma2(h[i], h[i], a);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&a);
  s += __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u);
  any |= v.x | v.y | v.z | v.w;
}
// A square sum as a bound: 0 for zeros alone, and never 0 by underflow.
__device__ __forceinline__ float square_bound(float s, uint32_t any) {
  return (any & 0x7fff7fffu) == 0u ? 0.f : s < 1e-30f ? 1e-30f : s;
}

__global__ void __launch_bounds__(kTcThreads, 1)
    router_logits_tc_kernel(const __grid_constant__ CUtensorMap tmU,
                            const __grid_constant__ CUtensorMap tmE, const LogitParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + OFF_B;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* used = full + STAGES;       // the stage's products are done
  uint64_t* empty = used + STAGES;      // and its tokens have been squared
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  float* emax = reinterpret_cast<float*>(smem + OFF_EMAX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();           // which 128 tokens, which half of the experts
  const bool is_leader = half == 0;
  const int Nt = p.Nt;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&used[s], 1);
      mbar_init(&empty[s], kSqWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);          // the epilogue warps of both CTAs
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmU);
    tma_prefetch_desc(&tmE);
  }
  if (warp == 1) {
    tmem2_alloc(tmem_slot, 512);
    tmem2_relinquish();
  }
  pdl_trigger();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.N_r; i += blockDim.x) p.counts[i] = 0;
    if (threadIdx.x < 2) p.n_listed[threadIdx.x] = 0;
  }
  tc_fence_before();
  cluster_sync_all();          // barriers initialised in both CTAs, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full_leader0 = map_shared_to(smem_u32(&full[0]), 0);
  const uint32_t tempty_leader0 = map_shared_to(smem_u32(&tempty[0]), 0);
  const int items = p.n_tt * p.n_et * p.S, step = (int)n_clusters_x();
  const int first = (int)cluster_id_x();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t bytes = 2u * (uint32_t)(A_BOX + (Nt / 2) * BK * 2);    // per block of 64
      for (int it = first; it < items && ok; it += step) {
        const int et = it % p.n_et, sl = (it / p.n_et) % p.S, tt = it / p.n_et / p.S;
        const int row0 = tt * 2 * TM + (int)half * TM, e0 = et * Nt + (int)half * (Nt / 2);
        const int kb1 = (sl + 1) * p.nk / p.S;
        for (int kb = sl * p.nk / p.S; kb < kb1; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          if (is_leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t fb = full_leader0 + stage * 8;
          tma_load_2d_pair(sA + stage * A_BOX, &tmU, kb * BK, row0, fb);
          tma_load_2d_pair(sB + stage * B_BOX, &tmE, kb * BK, e0, fb);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      // the leader waits until every armed stage's copies have landed
      if (is_leader)
        for (int s = 0; s < STAGES; ++s)
          mbar_wait_bounded(&full[s], ((s < stage) ? phase : phase ^ 1), nullptr, kWaitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (pair leader)
    if (is_leader && lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(2 * TM, Nt);
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step) {
        const int sl = (it / p.n_et) % p.S;
        const int kb0 = sl * p.nk / p.S, kb1 = (sl + 1) * p.nk / p.S;
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool first_of = (kb - kb0) % kChunk == 0;
          const bool last_of = (kb - kb0 + 1) % kChunk == 0 || kb + 1 == kb1;
          if ((first_of && !mbar_wait_bounded(&tempty[buf], tphase ^ 1, abort_flag, kWaitNs)) ||
              !mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitNs)) {
            raise_abort(abort_flag, p.err);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * A_BOX), b0 = smem_u32(sB + stage * B_BOX);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma2_f16_ss(tmem_base + buf * kMaxN, smem_desc_k_sw128(a0 + k * 32),
                        smem_desc_k_sw128(b0 + k * 32), idesc, (!first_of || k > 0) ? 1u : 0u);
          mma2_commit_mask(&used[stage], 3);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
          if (last_of) {
            mma2_commit_mask(&tfull[buf], 3);
            if (++buf == 2) { buf = 0; tphase ^= 1; }
          }
        }
      }
      mma2_commit_local(mma_done);
      mbar_wait_bounded(mma_done, 0, nullptr, kWaitNs);
    }
  } else if (warp >= 2 + kEpiWarps) {
    // ------------------------------------------------------------ square sums (both CTAs)
    // A lane takes 16 bytes of every fourth of its warp's 64 token rows (a row is
    // 128 bytes a block, in any order).
    const int w = warp - 2 - kEpiWarps;
    constexpr int kRows = TM / kSqWarps / 4;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += step) {
      const int et = it % p.n_et, sl = (it / p.n_et) % p.S, tt = it / p.n_et / p.S;
      const int kb1 = (sl + 1) * p.nk / p.S;
      float sq[kRows];
      uint32_t any[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) { sq[r] = 0.f; any[r] = 0u; }
      for (int kb = sl * p.nk / p.S; kb < kb1; ++kb) {
        const bool got = mbar_wait_bounded(&used[stage], phase, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          ok = false;
          break;
        }
        if (et == 0) {
          const uint4* rows =
              reinterpret_cast<const uint4*>(sA + stage * A_BOX) + w * (kRows * 32) + lane;
#pragma unroll
          for (int r = 0; r < kRows; ++r) add_squares(rows[r * 32], sq[r], any[r]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
      if (!ok) break;
      if (et == 0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) {              // the row's eight lanes
            sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
            any[r] |= __shfl_xor_sync(0xffffffffu, any[r], o);
          }
          const int row = tt * 2 * TM + (int)half * TM + (w * kRows + r) * 4 + (lane >> 3);
          if ((lane & 7) == 0 && row < p.T)
            p.u2[(size_t)sl * token_groups(p.T) * 32 + row] = square_bound(sq[r], any[r]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int w = warp - 2, q = warp & 3, part = w >> 2;
    const int n_pieces = Nt / 16;
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // the experts' square sums, a warp per expert
    float e_top = 0.f;
    for (int e = blockIdx.x * kEpiWarps + w; e < p.N_r; e += gridDim.x * kEpiWarps) {
      const uint4* row = reinterpret_cast<const uint4*>(p.E + (size_t)e * p.d);
      const int nv = p.d / 8;
      float sq = 0.f;
      uint32_t any = 0u;
#pragma unroll 8
      for (int v = lane; v < nv; v += 32) add_squares(__ldg(row + v), sq, any);
      const float b = square_bound(sel_warp_sum(sq), __reduce_or_sync(0xffffffffu, any));
      e_top = fmaxf(e_top, b == b ? b : 1e-30f);         // NaN: its logits are NaN either way
    }
    if (lane == 0) emax[w] = e_top;
    int buf = 0;
    uint32_t tphase = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += step) {
      const int et = it % p.n_et, sl = (it / p.n_et) % p.S, tt = it / p.n_et / p.S;
      const int kb0 = sl * p.nk / p.S, kb1 = (sl + 1) * p.nk / p.S;
      float acc[kPieces][16];
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
      for (int c0 = kb0; c0 < kb1; c0 += kChunk) {
        const bool got = mbar_wait_bounded(&tfull[buf], tphase, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) raise_abort(abort_flag, p.err);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int piece = part + i * (kEpiWarps / 4);
          if (piece < n_pieces) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(trow + buf * kMaxN + piece * 16, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][j] += __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader0 + buf * 8);
        if (++buf == 2) { buf = 0; tphase ^= 1; }
      }
      if (!ok) break;
      const int t = tt * 2 * TM + (int)half * TM + q * 32 + lane;
      if (t < p.T) {
        float* out = p.P + sl * slice_stride(p.T, p.ld) + tc_row(t, p.ld) + tc_col(et * Nt);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int piece = part + i * (kEpiWarps / 4);
          if (piece < n_pieces) {
            st_global_v8(out + piece * 512, &acc[i][0]);
            st_global_v8(out + piece * 512 + 256, &acc[i][8]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && blockIdx.x < p.n_e2) {
    float e_top = 0.f;
    for (int w = 0; w < kEpiWarps; ++w) e_top = fmaxf(e_top, emax[w]);
    p.e2[blockIdx.x] = e_top;
  }
  cluster_sync_all();          // no CTA leaves while the other may still use its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_base, 512);
  }
}

// CTA pairs of the logits kernel that run at once.
int resident_pairs() {
  static int cached[kMaxSmemDevices] = {};
  static bool attr_done[kMaxSmemDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxSmemDevices) return 0;
  const void* kern = reinterpret_cast<const void*>(router_logits_tc_kernel);
  if (ensure_max_smem(kern, SMEM_ALLOC, attr_done, "router_logits smem attribute") != MOE_OK)
    return 0;
  if (cached[dev]) return cached[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sm_count() / 2));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  cached[dev] = n;
  return n;
}

// Tiling of the tensor-core logits: expert tiles of equal width, as many
// slices of d as fill the GPU once (fewer tokens: more slices; a slice keeps
// at least four blocks of 64).  148 SMs are 74 pairs; the workspace is sized
// for that many.
constexpr int kPairs = 74, kMaxSlices = 16;
struct LogitTiling {
  int n_tt, n_et, Nt, S, ld;
};
LogitTiling logit_tiling(int T, int d, int N) {
  LogitTiling L;
  L.n_tt = (T + 2 * TM - 1) / (2 * TM);
  L.n_et = (N + kMaxN - 1) / kMaxN;
  L.Nt = ((N + L.n_et - 1) / L.n_et + 31) / 32 * 32;
  L.ld = L.n_et * L.Nt;
  int S = kPairs / (L.n_tt * L.n_et);
  if (S > d / BK / 4) S = d / BK / 4;
  if (S > kMaxSlices) S = kMaxSlices;
  L.S = S < 1 ? 1 : S;
  return L;
}

// ---------------------------------------------------------------- few tokens
// A block per expert, TT tokens at once: float64 sums of the products, which
// are exact in float32 (two 8-bit significands) unless they fall below 2^-126.
// Latency-bound: all of a thread's row pieces are in flight together.
template <int TT>
__global__ void __launch_bounds__(128) router_logits_few_kernel(
    const __nv_bfloat16* __restrict__ u, const __nv_bfloat16* __restrict__ E, int T, int d, int N,
    double* __restrict__ P, int32_t* __restrict__ counts) {
  __shared__ double part[4][TT];
  const int e = blockIdx.x, tid = threadIdx.x, nv = d / 8;
  pdl_trigger();
  if (e == 0)
    for (int i = tid; i < N; i += 128) counts[i] = 0;
  const uint4* er = reinterpret_cast<const uint4*>(E + (size_t)e * d);
  double a[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) a[t] = 0.0;
  constexpr int U = 8;
  for (int v0 = tid; v0 < nv; v0 += 128 * U) {
    uint4 w[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int v = v0 + 128 * q;
      w[q] = v < nv ? __ldg(er + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t >= T) break;
      const uint4* ur = reinterpret_cast<const uint4*>(u + (size_t)t * d);
      uint4 x[U];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int v = v0 + 128 * q;
        x[q] = v < nv ? __ldg(ur + v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        float fx[8], fw[8];
        Vec<__nv_bfloat16>::load(x[q], fx);
        Vec<__nv_bfloat16>::load(w[q], fw);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[t] += (double)(fx[i] * fw[i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    a[t] = sel_warp_sum(a[t]);
    if ((tid & 31) == 0) part[tid >> 5][t] = a[t];
  }
  __syncthreads();
  if (tid < TT && tid < T)
    P[(size_t)tid * N + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}
constexpr int kFewTokens = 8;

// ---------------------------------------------------------------- float64 logits
// P[s][t][i] = sum over slice s of d of u[t,k] E[i,k] of float32 inputs, on the
// float64 tensor pipe (m8n8k4).  A 32-token x 64-expert tile per block of four
// warps (16 x 32 each, eight products per four columns for six operand loads;
// one output per thread from shared memory was bound by those loads, 53 us at
// T 1037, d 2048, N_r 61), 32 columns of both operands staged as float64 while
// the next 32 are on their way.  Bound by the float64 rate.
constexpr int kT64 = 32, kE64 = 64, kK64 = 32, kLd64 = kK64 + 4;

__device__ __forceinline__ void mma_f64(double& c0, double& c1, double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
               : "+d"(c0), "+d"(c1)
               : "d"(a), "d"(b));
}

__global__ void __launch_bounds__(128) router_logits64_kernel(
    const float* __restrict__ u, const float* __restrict__ E, int T, int d, int N, int S, int ld,
    double* __restrict__ P, int32_t* __restrict__ counts) {
  __shared__ double su[kT64][kLd64], se[kE64][kLd64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kT64, e0 = blockIdx.y * kE64, sl = blockIdx.z;
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && sl == 0)
    for (int i = tid; i < N; i += 128) counts[i] = 0;
  const int nc = d / kK64;                                // d % 64 == 0
  const int c0 = (int)((long long)sl * nc / S), c1 = (int)((long long)(sl + 1) * nc / S);
  // 96 rows of eight float4s: six a thread
  constexpr int kLoads = (kT64 + kE64) * kK64 / 4 / 128;
  float4 nx[kLoads];
  const auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (i * 128 + tid) >> 3, k4 = (tid & 7) * 4 + c * kK64;
      const bool is_u = r < kT64;
      const int row = is_u ? t0 + r : e0 + r - kT64;
      nx[i] = row < (is_u ? T : N)
                  ? *reinterpret_cast<const float4*>((is_u ? u : E) + (size_t)row * d + k4)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  double acc[2][4][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j][0] = acc[i][j][1] = 0.0;
  const int wt = (warp & 1) * 16 + (lane >> 2), we = (warp >> 1) * 32 + (lane >> 2), kk = lane & 3;
  if (c0 < c1) fetch(c0);
  for (int c = c0; c < c1; ++c) {
    __syncthreads();                                      // the last columns have been used
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (i * 128 + tid) >> 3, k4 = (tid & 7) * 4;
      double* dst = r < kT64 ? &su[r][k4] : &se[r - kT64][k4];
      dst[0] = nx[i].x; dst[1] = nx[i].y; dst[2] = nx[i].z; dst[3] = nx[i].w;
    }
    __syncthreads();
    if (c + 1 < c1) fetch(c + 1);
#pragma unroll
    for (int k = 0; k < kK64; k += 4) {
      double a[2], b[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = su[wt + 8 * i][k + kk];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = se[we + 8 * j][k + kk];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f64(acc[i][j][0], acc[i][j][1], a[i], b[j]);
    }
  }
  double* out = P + (size_t)sl * T * ld;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = t0 + wt + 8 * i, e = e0 + (warp >> 1) * 32 + 8 * j + 2 * kk + h;
        if (t < T && e < N) out[(size_t)t * ld + e] = acc[i][j][h];
      }
}

// ---------------------------------------------------------------- selection
// A warp per token; the block's load histogram in shared memory, then added to
// counts (whole numbers: the order of the additions does not matter).

// The tokens listed for the exact pass: how many, their ids, and 32 words of
// experts that the open decisions wait for (word l, bit j: expert j*32 + l);
// and those of them whose every logit has to be exact: how many, ids, finished shares and
// float64 logits [T][N_r].  u2, e2: the square sums that router_logits_tc_kernel
// left (LogitParams), n_e2 of the latter.
struct Recheck {
  int32_t* n;             // [2]
  int32_t* tok;
  uint32_t* mask;
  int32_t* full_tok;
  int32_t* full_done;
  double* full_x;
  float* u2;
  float* e2;
  int n_e2;
};

// The largest square sum of an expert, by a warp.
__device__ __forceinline__ float largest_e2(const Recheck& rc) {
  constexpr int kMost = (kMaxE2 + 31) / 32;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = i * 32 + (threadIdx.x & 31);
    v = fmaxf(v, at < rc.n_e2 ? rc.e2[at] : 0.f);
  }
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));   // no sign, no NaN
}
// Bound on the error of token t's logits, by a warp (S <= kMaxSlices < 32 slices).
__device__ __forceinline__ float token_error(const Recheck& rc, int S, int T, int t, float e2) {
  const int lane = threadIdx.x & 31;
  const float v = lane < S ? rc.u2[(size_t)lane * token_groups(T) * 32 + t] : 0.f;
  return logit_error(sel_warp_sum(v), e2);
}

// x[j]: the slices' sums, joined in slice order.
template <int V>
__device__ __forceinline__ void join_slices(const float* __restrict__ row, int S, size_t stride,
                                            int N, float (&x)[V]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = j * 32 + lane < N ? row[tc_col(j * 32 + lane)] : 0.f;
  for (int s = 1; s < S; ++s) {
    row += stride;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] += j * 32 + lane < N ? row[tc_col(j * 32 + lane)] : 0.f;
  }
}

template <int V>
__global__ void __launch_bounds__(128, V <= 8 ? 7 : V <= 16 ? 4 : 2) router_select_kernel(
    const float* __restrict__ P, int S, int ld, const float* __restrict__ bias, int T,
    SelectRule r, int32_t* __restrict__ idx, float* __restrict__ gate,
    int32_t* __restrict__ counts, float* __restrict__ logits, Recheck rc) {
  extern __shared__ int hist[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wpb = blockDim.x >> 5;
  const int N = r.N_r;
  float* wk = reinterpret_cast<float*>(hist + N) + (size_t)warp * N;
  for (int i = threadIdx.x; i < N; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const float e2 = largest_e2(rc);
  float b_lo = 0.f, b_hi = 0.f;
  if (bias) {
    b_lo = INFINITY;
    b_hi = -INFINITY;
    for (int i = lane; i < N; i += 32) {
      b_lo = fminf(b_lo, bias[i]);
      b_hi = fmaxf(b_hi, bias[i]);
    }
    b_lo = -sel_warp_max(-b_lo);
    b_hi = sel_warp_max(b_hi);
  }
  for (int t = blockIdx.x * wpb + warp; t < T; t += gridDim.x * wpb) {
    float x[V], sc[V], key[V];
    const float logit_err = token_error(rc, S, T, t, e2);
    const bool wide = logit_err > kWideError;            // every logit from float64
    join_slices<V>(P + tc_row(t, ld), S, slice_stride(T, ld), N, x);
    if (logits) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * 32 + lane < N) logits[(size_t)t * N + j * 32 + lane] = x[j];
    }
    int32_t* ti = idx + (size_t)t * r.K;
    TokenScale ts = select_keys<V>(x, bias, r, logit_err, sc, key);
    ts.b_lo = b_lo;
    ts.b_hi = b_hi;
    const Selection sel = select_core<V>(key, ts, bias, r, wk, ti);
    if (sel.open || wide) {
      int slot = 0;
      if (lane == 0) {
        slot = atomicAdd(rc.n, 1);
        rc.tok[slot] = t;
      }
      slot = __shfl_sync(0xffffffffu, slot, 0);
      uint32_t mask = sel.mask;
      const float most = ts.range_error(sel.lo - key_error(ts.top, sel.lo),
                                        sel.hi + key_error(ts.top, sel.hi));
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * 32 + lane < N &&
            (wide || takes_part(key[j], key_error(most, key[j]), sel.lo, sel.hi)))
          mask |= 1u << j;
      rc.mask[(size_t)slot * 32 + lane] = mask;
      continue;                                     // its gates and load come with the exact pass
    }
    select_gates<V, float>(x, sel.e, ts.m, ts.z, r, ti, gate + (size_t)t * r.K);
    for (int k = lane; k < r.K; k += 32) atomicAdd(&hist[r.K <= 32 ? sel.e : ti[k]], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += blockDim.x)
    if (hist[i]) atomicAdd(&counts[i], hist[i]);
}

// A block per token, a thread per expert (router_select.cuh): every token, or
// the listed ones (rc.tok, the first pass left their decisions open).
//   EXACT   P holds float64 slices
//   else    float32 slices; the experts that open decisions wait for get
//           float64 logits, kDots at a time, their products spread over the
//           block (exact in float32 unless below 2^-126).  Usually two or
//           three experts and one turn.
// Latency-bound (at T 8192 some 700 tokens are listed), so a thread has two
// vectors of every row in flight at once (one where a block has more threads
// than 256); four of them, or more registers than let three blocks share an
// SM, were slower at T 256 and at T 1024.
constexpr int kDots = 4;
template <bool EXACT, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 3 : 1) router_token_kernel(
    const __nv_bfloat16* __restrict__ u, const __nv_bfloat16* __restrict__ E,
    const void* __restrict__ P, int S, int ld, const float* __restrict__ bias, int T, int d,
    SelectRule r, int32_t* __restrict__ idx, float* __restrict__ gate,
    int32_t* __restrict__ counts, float* __restrict__ logits, Recheck rc, bool all_tokens) {
  constexpr int kAhead = MAXT <= 256 ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ double part[MAXT / 32][kDots];
  __shared__ int n_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = r.N_r, nv = d / 8;
  const BlockRoute b = block_route_smem(smem_raw, N, r.K);
  pdl_wait();
  pdl_trigger();
  const int n = all_tokens ? T : rc.n[0];
  const float e2 = EXACT ? 0.f : largest_e2(rc);
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int t = all_tokens ? i : rc.tok[i];
    double a = 0.0;
    const float logit_err = EXACT ? 0.f : token_error(rc, S, T, t, e2);
    const bool wide = logit_err > kWideError;            // every logit from float64
    if (tid < N) {
      if (EXACT) {
        const size_t at = (size_t)t * ld + tid, stride = (size_t)T * ld;
        for (int s = 0; s < S; ++s) a += static_cast<const double*>(P)[at + s * stride];
      } else {
        // as the first pass joined them
        const size_t at = tc_row(t, ld) + tc_col(tid), stride = slice_stride(T, ld);
        float f = static_cast<const float*>(P)[at];
        for (int s = 1; s < S; ++s) f += static_cast<const float*>(P)[at + s * stride];
        a = (double)f;
      }
      if (logits) logits[(size_t)t * N + tid] = (float)a;
    }
    if (tid < N) {
      b.x[tid] = a;
      b.exact_f[tid] = EXACT || logit_err == 0.f;
    }
    const auto fetch = [&](int nl) {
      if (EXACT) return;                            // nothing is wanted
      const uint4* ur = reinterpret_cast<const uint4*>(u + (size_t)t * d);
      for (int c0 = 0; c0 < nl; c0 += kDots) {
        const int nc = min(kDots, nl - c0);
        const uint4* er[kDots];
        double acc[kDots];
#pragma unroll
        for (int c = 0; c < kDots; ++c) {
          er[c] = reinterpret_cast<const uint4*>(E + (size_t)b.list[c0 + min(c, nc - 1)] * d);
          acc[c] = 0.0;
        }
        for (int v0 = tid; v0 < nv; v0 += kAhead * blockDim.x) {
          uint4 x[kAhead], y[kAhead][kDots];
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            const int v = v0 + a * blockDim.x;
            x[a] = v < nv ? __ldg(ur + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < kDots; ++c)
              y[a][c] = v < nv && c < nc ? __ldg(er[c] + v) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            float fx[8], fy[8];
            Vec<__nv_bfloat16>::load(x[a], fx);
#pragma unroll
            for (int c = 0; c < kDots; ++c) {
              if (c < nc) {
                Vec<__nv_bfloat16>::load(y[a][c], fy);
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[c] += (double)(fx[k] * fy[k]);
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < kDots; ++c) {
          if (c < nc) {
            const double v = sel_warp_sum(acc[c]);
            if (lane == 0) part[warp][c] = v;
          }
        }
        __syncthreads();
        if (tid < nc) {
          double v = 0.0;
          for (int w = 0; w < (int)(blockDim.x >> 5); ++w) v += part[w][tid];
          b.x[b.list[c0 + tid]] = v;
        }
        __syncthreads();
      }
    };
    if (!EXACT && logit_err != 0.f && (wide || !all_tokens)) {
      // the experts that the first pass found wanting
      if (tid == 0) n_want = 0;
      __syncthreads();
      const bool want = tid < N && (wide || ((rc.mask[(size_t)i * 32 + lane] >> warp) & 1u));
      if (want) b.list[atomicAdd(&n_want, 1)] = (uint16_t)tid;
      __syncthreads();
      fetch(n_want);
      if (want) b.exact_f[tid] = 1;
    }
    const bool done = block_route(b, r, bias, logit_err, fetch, idx + (size_t)t * r.K,
                                  gate + (size_t)t * r.K, counts);
    if (!done && tid == 0) {
      const int slot = atomicAdd(&rc.n[1], 1);
      rc.full_tok[slot] = t;
      rc.full_done[slot] = 0;
    }
    __syncthreads();
  }
}

// The tokens whose every logit has to be exact (softmax scores a rounding
// apart: one token of some 30000).  A share is one expert for each warp of a
// block, so a lone token's N_r dot products spread over the GPU (by one block
// they took 200 us); the block that finishes a token's last share routes it.
template <int MAXT>
__global__ void __launch_bounds__(MAXT) router_full_kernel(
    const __nv_bfloat16* __restrict__ u, const __nv_bfloat16* __restrict__ E,
    const float* __restrict__ bias, int d, SelectRule r, int32_t* __restrict__ idx,
    float* __restrict__ gate, int32_t* __restrict__ counts, Recheck rc) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = r.N_r, nv = d / 8;
  const int per = blockDim.x >> 5, shares = (N + per - 1) / per;
  const BlockRoute b = block_route_smem(smem_raw, N, r.K);
  pdl_wait();
  const long long work = (long long)rc.n[1] * shares;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int i = (int)(w / shares), e = (int)(w - (long long)i * shares) * per + warp;
    const int t = rc.full_tok[i];
    if (e < N) {
      const uint4* ur = reinterpret_cast<const uint4*>(u + (size_t)t * d);
      const uint4* er = reinterpret_cast<const uint4*>(E + (size_t)e * d);
      double a = 0.0, c = 0.0;
      constexpr int U = 4;
      for (int v0 = lane; v0 < nv; v0 += 32 * U) {
        uint4 x[U], y[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const int v = v0 + 32 * q;
          x[q] = v < nv ? __ldg(ur + v) : make_uint4(0, 0, 0, 0);
          y[q] = v < nv ? __ldg(er + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
          float fx[8], fy[8];
          Vec<__nv_bfloat16>::load(x[q], fx);
          Vec<__nv_bfloat16>::load(y[q], fy);
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            a += (double)(fx[k] * fy[k]);
            c += (double)(fx[k + 1] * fy[k + 1]);
          }
        }
      }
      a = sel_warp_sum(a + c);
      if (lane == 0) {
        rc.full_x[(size_t)i * N + e] = a;
        __threadfence();
      }
    }
    __syncthreads();
    if (tid == 0) last = atomicAdd(&rc.full_done[i], 1) == shares - 1;
    __syncthreads();
    if (last) {
      __threadfence();
      if (tid < N) {
        b.x[tid] = __ldcg(rc.full_x + (size_t)i * N + tid);
        b.exact_f[tid] = 1;
      }
      block_route(b, r, bias, 0.f, [](int) {}, idx + (size_t)t * r.K, gate + (size_t)t * r.K,
                  counts);
    }
    __syncthreads();
  }
}

// Slices of d for the float64 logits: enough blocks for two per SM, at most
// kMaxSlices64, each slice at least 128 columns.
constexpr int kMaxSlices64 = 16;
int slices64(int T, int d, int N) {
  const long long tiles = (long long)((T + kT64 - 1) / kT64) * ((N + kE64 - 1) / kE64);
  long long S = (2LL * 148 + tiles - 1) / tiles;
  if (S > d / 128) S = d / 128;
  if (S > kMaxSlices64) S = kMaxSlices64;
  return S < 1 ? 1 : (int)S;
}

int dispatch_v(int N) {
  const int V = (N + 31) / 32;
  return V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : V <= 16 ? 16 : 32;
}

// Rows of partial logits over every token count up to T: slices times tokens
// (whole groups of 32) is at most the larger of T and what fills the pairs once
// (so a workspace for more tokens serves fewer).
size_t slice_rows(int T, int n_et) {
  const size_t t32 = (size_t)token_groups(T) * 32;
  const size_t fill = (size_t)kPairs * 2 * TM / n_et, most = kMaxSlices * t32;
  const size_t rows = most < fill ? most : fill;
  return rows > t32 ? rows : t32;
}
size_t slice_rows64(int T, int N) {
  const size_t et = (N + kE64 - 1) / kE64, most = (size_t)kMaxSlices64 * T;
  const size_t fill = (size_t)T + (2 * 148 * kT64 + et - 1) / et + kT64;
  return most < fill ? most : fill;
}

// Workspace of the tensor-core path: partial logits, then the listing.
size_t tc_ws_bytes(int T, int d, int N, Recheck* rc, uint8_t* base) {
  const LogitTiling L = logit_tiling(T, d, N);
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
  take(slice_rows(T, L.n_et) * L.ld * 4);
  const size_t u2 = take(slice_rows(T, L.n_et) * 4), e2 = take(kMaxE2 * 4);
  const size_t n = take(8), tok = take((size_t)T * 4), mask = take((size_t)T * 128), ftok = take((size_t)T * 4),
               fdone = take((size_t)T * 4), fx = take((size_t)T * N * 8);
  if (rc) {
    rc->u2 = reinterpret_cast<float*>(base + u2);
    rc->e2 = reinterpret_cast<float*>(base + e2);
    rc->n = reinterpret_cast<int32_t*>(base + n);
    rc->tok = reinterpret_cast<int32_t*>(base + tok);
    rc->mask = reinterpret_cast<uint32_t*>(base + mask);
    rc->full_tok = reinterpret_cast<int32_t*>(base + ftok);
    rc->full_done = reinterpret_cast<int32_t*>(base + fdone);
    rc->full_x = reinterpret_cast<double*>(base + fx);
  }
  return o;
}

moe_status launch_logits_tc(const void* u, const void* E, int T, int d, int N, float* P,
                            int32_t* counts, Recheck* rc, cudaStream_t s) {
  const LogitTiling L = logit_tiling(T, d, N);
  CUtensorMap tmU, tmE;
  moe_status st = make_tmap_2d(&tmU, u, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, T, BK, TM);
  if (st != MOE_OK) return st;
  st = make_tmap_2d(&tmE, E, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, N, BK, L.Nt / 2);
  if (st != MOE_OK) return st;
  LogitParams p;
  p.T = T;
  p.N_r = N;
  p.nk = d / BK;
  p.S = L.S;
  p.n_tt = L.n_tt;
  p.n_et = L.n_et;
  p.Nt = L.Nt;
  p.ld = L.ld;
  p.P = P;
  p.counts = counts;
  p.n_listed = rc->n;
  p.E = static_cast<const __nv_bfloat16*>(E);
  p.d = d;
  p.u2 = rc->u2;
  p.e2 = rc->e2;
  p.err = device_error_word();
  if (!p.err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const int resident = resident_pairs(), pairs = resident < kPairs ? resident : kPairs;
  if (pairs <= 0) return fail(MOE_ERR_CUDA, "router_logits: no resident CTA pair");
  const long long items = (long long)L.n_tt * L.n_et * L.S;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(items < pairs ? items : pairs));
  // every block of the grid, or as many as have an expert
  const int with_experts = (N + kEpiWarps - 1) / kEpiWarps;
  p.n_e2 = rc->n_e2 = with_experts < (int)cfg.gridDim.x ? with_experts : (int)cfg.gridDim.x;
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, router_logits_tc_kernel, tmU, tmE, p),
                    "router_logits launch");
}

}  // namespace

size_t route_scored_ws_bytes(int T, int d, int N_r) {
  // the larger of the float64 and the tensor-core path's needs: the dtype is
  // not among the arguments
  const size_t a = align_up(slice_rows64(T, N_r) * N_r * sizeof(double), 256);
  const size_t b = tc_ws_bytes(T, d, N_r, nullptr, nullptr);
  return a > b ? a : b;
}

// Whether blocks route every token: a block per token keeps a lone token's latency
// low, a warp per token costs a third of the instructions, and a block holds as
// many threads as there are experts.  Blocks and warps, grouped sigmoid, us:
//   d 7168, 256 experts: T 256 33 and 44, T 1024 51 and 53, T 2048 73 and 57
//   d 2048,  64 experts: T 256 23 and 29, T 1024 31 and 30, T 2048 39 and 35
//   d 4096, 1024 experts: T 64 46 and 72, T 256 68 and 77, T 512 103 and 72
constexpr int kBlockTokens = 1024, kBlockExperts = 256;
bool blocks_route(int T, int N_r) {
  return (long long)T * (N_r > kBlockExperts ? N_r : kBlockExperts) <=
         (long long)kBlockTokens * kBlockExperts;
}

namespace {
template <bool EXACT>
moe_status launch_router_token(const void* u, const void* E, const void* P, int S, int ld,
                               const float* b, int T, int d, const SelectRule& r, int32_t* idx,
                               float* gate, int32_t* counts, float* logits, const Recheck& rc,
                               bool all_tokens, int blocks, cudaStream_t s) {
  int threads = (r.N_r + 31) / 32 * 32;
  if (threads < 128) threads = 128;
  const size_t smem = block_route_bytes(r.N_r, r.K);
  const auto ub = static_cast<const __nv_bfloat16*>(u);
  const auto eb = static_cast<const __nv_bfloat16*>(E);
  const auto kern = threads <= 256 ? router_token_kernel<EXACT, 256> : router_token_kernel<EXACT, 1024>;
  return launch_after(kern, dim3(blocks), dim3(threads), smem, s, 1, "router_token launch", ub, eb, P,
                      S, ld, b, T, d, r, idx, gate, counts, logits, rc, all_tokens);
}

moe_status launch_router_full(const void* u, const void* E, const float* b, int d,
                              const SelectRule& r, int32_t* idx, float* gate, int32_t* counts,
                              const Recheck& rc, cudaStream_t s) {
  int threads = (r.N_r + 31) / 32 * 32;
  if (threads < 256) threads = 256;
  const auto kern = threads <= 256 ? router_full_kernel<256> : router_full_kernel<1024>;
  return launch_after(kern, dim3(sm_count()), dim3(threads), block_route_bytes(r.N_r, r.K), s, 1,
                      "router_full launch", static_cast<const __nv_bfloat16*>(u),
                      static_cast<const __nv_bfloat16*>(E), b, d, r, idx, gate, counts, rc);
}
}  // namespace

moe_status launch_route_scored(const void* u, const void* E, moe_dtype dt, const float* b, int T,
                               int d, int N_r, int K, int score, int n_groups, int topk_groups,
                               int group_top, int renorm, float gate_scale, int32_t* idx,
                               float* gate, int32_t* counts, float* logits, void* ws,
                               cudaStream_t s) {
  using bf = __nv_bfloat16;
  const SelectRule r{N_r, K, score, n_groups, topk_groups, group_top, renorm, gate_scale};
  moe_status st;
  if (dt == MOE_BF16 && T > kFewTokens) {
    float* P = static_cast<float*>(ws);
    Recheck rc{};
    tc_ws_bytes(T, d, N_r, &rc, static_cast<uint8_t*>(ws));
    const LogitTiling L = logit_tiling(T, d, N_r);
    st = launch_logits_tc(u, E, T, d, N_r, P, counts, &rc, s);
    if (st != MOE_OK) return st;
    // a sigmoid needs no other logit: only softmax tokens can ask for all of them
    const bool full = score == MOE_SCORE_SOFTMAX;
    if (blocks_route(T, N_r)) {
      st = launch_router_token<false>(u, E, P, L.S, L.ld, b, T, d, r, idx, gate, counts, logits, rc,
                                      true, T, s);
      return st == MOE_OK && full ? launch_router_full(u, E, b, d, r, idx, gate, counts, rc, s) : st;
    }
    const int wpb = 4, blocks = (T + wpb - 1) / wpb < 16 * sm_count() ? (T + wpb - 1) / wpb
                                                                      : 16 * sm_count();
    const size_t smem = (size_t)N_r * sizeof(int) * (1 + wpb);
#define MOE_SELECT(v)                                                                        \
  case v:                                                                                    \
    st = launch_after(router_select_kernel<v>, dim3(blocks), dim3(wpb * 32), smem, s, 1,     \
                      "router_select launch", P, L.S, L.ld, b, T, r, idx, gate, counts,      \
                      logits, rc);                                                           \
    break;
    switch (dispatch_v(N_r)) {
      MOE_SELECT(1) MOE_SELECT(2) MOE_SELECT(4) MOE_SELECT(8) MOE_SELECT(16) MOE_SELECT(32)
    }
#undef MOE_SELECT
    if (st != MOE_OK) return st;
    st = launch_router_token<false>(u, E, P, L.S, L.ld, b, T, d, r, idx, gate, counts, nullptr, rc,
                                    false, 3 * sm_count(), s);
    return st == MOE_OK && full ? launch_router_full(u, E, b, d, r, idx, gate, counts, rc, s) : st;
  }
  double* P = static_cast<double*>(ws);
  int S = 1;
  if (dt == MOE_F32) {
    S = slices64(T, d, N_r);
    const dim3 grid((T + kT64 - 1) / kT64, (N_r + kE64 - 1) / kE64, S);
    router_logits64_kernel<<<grid, 128, 0, s>>>(static_cast<const float*>(u),
                                                static_cast<const float*>(E), T, d, N_r, S, N_r, P,
                                                counts);
  } else {
    const bf* ub = static_cast<const bf*>(u);
    const bf* eb = static_cast<const bf*>(E);
    if (T <= 1) router_logits_few_kernel<1><<<N_r, 128, 0, s>>>(ub, eb, T, d, N_r, P, counts);
    else if (T <= 2) router_logits_few_kernel<2><<<N_r, 128, 0, s>>>(ub, eb, T, d, N_r, P, counts);
    else if (T <= 4) router_logits_few_kernel<4><<<N_r, 128, 0, s>>>(ub, eb, T, d, N_r, P, counts);
    else router_logits_few_kernel<8><<<N_r, 128, 0, s>>>(ub, eb, T, d, N_r, P, counts);
  }
  st = cuda_check(cudaGetLastError(), "router float64 logits launch");
  if (st != MOE_OK) return st;
  const int blocks = T < 16 * sm_count() ? T : 16 * sm_count();
  return launch_router_token<true>(u, E, P, S, N_r, b, T, d, r, idx, gate, counts, logits, Recheck{},
                                   true, blocks, s);
}

}  // namespace moe
