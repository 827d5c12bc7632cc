// Sequence-wise balance loss of the scored router and the gradients of the
// scored router (moe_balance_loss, moe_route_scored_backward).
//
//   s' = s / sum_j s_j;  over a sequence of n tokens
//   f_i = N_r / (K n) * #{(t, k): idx = i},   P_i = 1/n sum_t s'_{t,i}
//   loss = alpha sum_i f_i P_i;   coef_i = dloss / ds'_{t,i} = alpha f_i / n
//
// With c_k the selected scores, g~_k = c_k / sum c, G = sum_k g_k dg_k and
// q_i = d_loss * coef_i, Q = sum_j s'_j q_j, the logit gradient is
//   softmax: p_i (q_i - Q - R) + sum over slots k of i of
//            p_i scale dg_k  (raw, R = sum_k c_k scale dg_k)
//            g~_k (scale dg_k - G)  (renormalised, R = 0)
//   sigmoid: s_i (1 - s_i) (q_i - Q) / sum_j s_j + sum over slots k of i of
//            s_i (1 - s_i) scale dg_k  (raw)
//            g~_k (1 - s_i) (scale dg_k - G)  (renormalised)
#include <math.h>

#include "launch.h"

namespace moe {

namespace {

__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float wmax(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v || w != w ? w : v;
  }
  return v;
}

// s = Sigmoid(x) and om = 1 - s, both to full relative precision.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& om) {
  const float e = expf(x < 0.f ? x : -x), inv = 1.f / (1.f + e);
  s = x < 0.f ? e * inv : inv;
  om = x < 0.f ? inv : e * inv;
}

// Row [r0, r1) of sequence q, made safe: inside [0, T], not negative.
__device__ __forceinline__ void seq_range(const int32_t* off, int q, int T, int* err, int& r0,
                                          int& r1) {
  clamp_group_rows(off, q, T, err, r0, r1);
}

// The last sequence whose first token is <= t (-1: t lies before the first).
__device__ __forceinline__ int seq_at(const int32_t* off, int n_seq, int t) {
  if (!off) return 0;
  int lo = -1, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

constexpr int kChunk = 32;       // tokens per block of the balance sums
constexpr int kBalWarps = 8;

// Partial sums of one (chunk of tokens, sequence) pair, row chunk + sequence:
// along the pairs either number grows, so the rows are distinct.  Warp w takes
// the pair's tokens w, w + 8, ...; the warps' sums are added in warp order.
template <int V>
__global__ void __launch_bounds__(32 * kBalWarps) balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ off, int n_seq, int T, int N, int K, int softmax,
    float* __restrict__ psum, int32_t* __restrict__ pcnt) {
  extern __shared__ float sm[];                 // [kBalWarps][N] sums, then [N] counts
  int* cnt = reinterpret_cast<int*>(sm + kBalWarps * N);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * kChunk, t1 = min(T, t0 + kChunk);
  int q = seq_at(off, n_seq, t0);
  if (q < 0) q = 0;
  for (; q < n_seq; ++q) {
    int r0, r1;
    seq_range(off, q, T, nullptr, r0, r1);
    if (r0 >= t1) break;
    r0 = max(r0, t0);
    r1 = min(r1, t1);
    if (r0 >= r1) continue;
    for (int i = threadIdx.x; i < N; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int t = r0 + warp; t < r1; t += kBalWarps) {
      float s[V], m = -INFINITY, z = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = j * 32 + lane;
        s[j] = e < N ? logits[(size_t)t * N + e] : -INFINITY;
        m = fmaxf(m, s[j]);
      }
      if (softmax) m = wmax(m);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * 32 + lane < N) {
          float om;
          if (softmax) s[j] = expf(s[j] - m);
          else sigmoid_pair(s[j], s[j], om);
          z += s[j];
        } else {
          s[j] = 0.f;
        }
      }
      const float inv = 1.f / wsum(z);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(s[j], inv, acc[j]);
      for (int k = lane; k < K; k += 32) {
        const int e = idx[(size_t)t * K + k];
        if (e >= 0 && e < N) atomicAdd(&cnt[e], 1);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) sm[warp * N + j * 32 + lane] = acc[j];
    __syncthreads();
    const size_t row = (size_t)(blockIdx.x + q) * N;
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) a += sm[w * N + i];
      psum[row + i] = a;
      pcnt[row + i] = cnt[i];
    }
    __syncthreads();
  }
}

// One block per sequence: coef and loss from the partial rows in chunk order,
// the sums over chunks in float64.
__global__ void __launch_bounds__(256) balance_final_kernel(
    const float* __restrict__ psum, const int32_t* __restrict__ pcnt,
    const int32_t* __restrict__ off, int T, int N, int K, float alpha, float* __restrict__ loss,
    float* __restrict__ coef, int* err) {
  __shared__ double red[8];
  const int q = blockIdx.x;
  int r0, r1;
  seq_range(off, q, T, threadIdx.x == 0 ? err : nullptr, r0, r1);
  const int n = r1 - r0;
  double part = 0.0;
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    double p = 0.0;
    int c = 0;
    if (n > 0)
      for (int k = r0 / kChunk; k <= (r1 - 1) / kChunk; ++k) {
        p += (double)psum[(size_t)(k + q) * N + i];
        c += pcnt[(size_t)(k + q) * N + i];
      }
    // alpha f_i / n with f_i = N_r c / (K n): rounded once
    const double cf = n > 0 ? (double)alpha * N * c / ((double)K * n * n) : 0.0;
    coef[(size_t)q * N + i] = (float)cf;
    part += cf * p;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < 8; ++w) a += red[w];
    loss[q] = (float)a;
  }
}

// ---------------------------------------------------------------- logit gradient
// A warp per token.  planes: d_logit as bf16 planes too (router_grad_tc.cu).
constexpr int kGradWarps = 4;

template <int V>
__global__ void __launch_bounds__(32 * kGradWarps) router_logit_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const float* __restrict__ d_gate, const int32_t* __restrict__ off, int n_seq,
    const float* __restrict__ coef, const float* __restrict__ d_loss, int T, int N, int K,
    int softmax, int renorm, float scale, float* __restrict__ d_logit,
    __nv_bfloat16* __restrict__ planes, int Tp, int Np) {
  extern __shared__ float sm[];
  // the planes' rows past the last token
  if (planes) {
    const long long pad = (long long)(Tp - T) * Np;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < 3 * pad;
         i += (long long)gridDim.x * blockDim.x)
      planes[((i / pad) * Tp + T) * (long long)Np + i % pad] = __float2bfloat16_rn(0.f);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = sm + (size_t)warp * N;          // the token's scores, then its slots' terms
  for (int t = blockIdx.x * kGradWarps + warp; t < T; t += gridDim.x * kGradWarps) {
    float x[V], s[V], om[V], q[V], m = -INFINITY, z = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      x[j] = e < N ? logits[(size_t)t * N + e] : -INFINITY;
      m = fmaxf(m, x[j]);
      q[j] = 0.f;
    }
    if (softmax) m = wmax(m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j * 32 + lane < N) {
        if (softmax) { s[j] = expf(x[j] - m); om[j] = 1.f; }
        else sigmoid_pair(x[j], s[j], om[j]);
        z += s[j];
      } else {
        s[j] = 0.f;
        om[j] = 0.f;
      }
    }
    const float inv = 1.f / wsum(z);
    if (softmax) {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] *= inv;
    }
    // balance term
    float Q = 0.f;
    if (coef) {
      const int sq = seq_at(off, n_seq, t);
      int r0 = 0, r1 = 0;
      if (sq >= 0) seq_range(off, sq, T, nullptr, r0, r1);
      if (t >= r0 && t < r1) {
        const float dl = d_loss ? d_loss[sq] : 1.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = j * 32 + lane;
          if (e < N) q[j] = dl * coef[(size_t)sq * N + e];
          Q = fmaf(s[j], q[j], Q);
        }
        Q = wsum(Q);
        if (!softmax) Q *= inv;
      }
    }
    // the slots
    float R = 0.f;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) row[j * 32 + lane] = x[j];
    __syncwarp();
    float xm = -INFINITY, den = 1.f, G = 0.f;
    bool ratio = false;
    float sxm = 1.f, dum;
    const auto slot = [&](int k, int& e, float& dg) {      // expert (-1: left out) and d_gate
      e = idx[(size_t)t * K + k];
      if (e < 0 || e >= N) e = -1;
      dg = e >= 0 ? scale * d_gate[(size_t)t * K + k] : 0.f;
    };
    const auto weight = [&](float xk) {                    // the score over the largest one
      if (!ratio) return expf(xk - xm);
      float a, b;
      sigmoid_pair(xk, a, b);
      return a / sxm;
    };
    if (d_gate && renorm) {
      for (int k = lane; k < K; k += 32) {
        int e;
        float dg;
        slot(k, e, dg);
        if (e >= 0) { const float v = row[e]; xm = v > xm || v != v ? v : xm; }
      }
      xm = wmax(xm);
      ratio = !softmax && !(xm < -30.f);
      if (ratio) sigmoid_pair(xm, sxm, dum);
      float w = 0.f, wd = 0.f;
      for (int k = lane; k < K; k += 32) {
        int e;
        float dg;
        slot(k, e, dg);
        if (e >= 0) {
          const float v = weight(row[e]);
          w += v;
          wd = fmaf(v, dg, wd);
        }
      }
      den = wsum(w);
      G = wsum(wd) / den;
    }
    float mine_v = 0.f;
    int mine_e = -1;
    // terms of the slots, then added to the row in slot order (an expert may
    // come twice)
    float add[V];
#pragma unroll
    for (int j = 0; j < V; ++j) add[j] = 0.f;
    if (d_gate) {
      for (int k0 = 0; k0 < K; k0 += 32) {
        mine_e = -1;
        mine_v = 0.f;
        if (k0 + lane < K) {
          float dg;
          slot(k0 + lane, mine_e, dg);
          if (mine_e >= 0) {
            const float xk = row[mine_e];
            float a, b;
            if (softmax) { a = expf(xk - m) * inv; b = 1.f; }
            else sigmoid_pair(xk, a, b);
            if (renorm) mine_v = weight(xk) / den * b * (dg - G);
            else { mine_v = a * b * dg; R += softmax ? a * dg : 0.f; }
          }
        }
        const int kn = min(32, K - k0);
        for (int k = 0; k < kn; ++k) {
          const int e = __shfl_sync(0xffffffffu, mine_e, k);
          const float v = __shfl_sync(0xffffffffu, mine_v, k);
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (e == j * 32 + lane) add[j] += v;
        }
      }
      R = wsum(R);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      if (e < N) {
        const float dense = softmax ? s[j] * (q[j] - Q - R) : s[j] * om[j] * (q[j] - Q) * inv;
        add[j] += dense;
        if (d_logit) d_logit[(size_t)t * N + e] = add[j];
      } else {
        add[j] = 0.f;
      }
      if (planes && e < Np) {
        // hi + mid + lo: 24 bits in three roundings; an infinity stays in hi
        const __nv_bfloat16 hi = __float2bfloat16_rn(add[j]);
        const float fh = __bfloat162float(hi);
        const float r1 = fabsf(fh) < INFINITY ? add[j] - fh : 0.f;
        const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
        const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
        const size_t at = (size_t)t * Np + e, plane = (size_t)Tp * Np;
        planes[at] = hi;
        planes[at + plane] = mid;
        planes[at + 2 * plane] = lo;
      }
    }
  }
}

// ---------------------------------------------------------------- CUDA-core products (float32 u, E)
// C[m, n] = base[m, n] + sum_k A(m, k) B[k, n], A(m, k) = A[m*lda + k] (or
// A[k*lda + m] with TA) float32, B row-major.  64 x 64 tile per block, 4 x 4
// outputs a thread, 16 steps of k staged at a time; every 256 steps the
// running sums join a second set, so that a long sum keeps its low bits.
template <bool TA>
__global__ void __launch_bounds__(256) router_product_kernel(
    const float* __restrict__ A, int lda, const float* __restrict__ B, int ldb,
    const float* base, float* C, int M, int N, int Kd) {
  __shared__ float sa[16][64 + 4], sb[16][64 + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  float acc[4][4] = {}, tot[4][4] = {};
  for (int k0 = 0; k0 < Kd; k0 += 16) {
    for (int i = tid; i < 16 * 64; i += 256) {
      int k, m;
      if (TA) { k = i >> 6; m = i & 63; } else { k = i & 15; m = i >> 4; }
      const bool ok = k0 + k < Kd && m0 + m < M;
      sa[k][m] = ok ? (TA ? A[(size_t)(k0 + k) * lda + m0 + m] : A[(size_t)(m0 + m) * lda + k0 + k])
                    : 0.f;
      const int kb = i >> 6, n = i & 63;
      sb[kb][n] = k0 + kb < Kd && n0 + n < N ? B[(size_t)(k0 + kb) * ldb + n0 + n] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[i] = sa[k][ty * 4 + i]; b[i] = sb[k][tx * 4 + i]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
    if ((k0 & 255) == 240 || k0 + 16 >= Kd) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) { tot[i][j] += acc[i][j]; acc[i][j] = 0.f; }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) {
        const size_t at = (size_t)m * N + n;
        C[at] = tot[i][j] + (base ? base[at] : 0.f);
      }
    }
}

int dispatch_v(int N) {
  const int V = (N + 31) / 32;
  return V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : V <= 16 ? 16 : 32;
}

}  // namespace

// Partial rows: one for every (chunk, sequence) pair.
size_t balance_ws_bytes(int T, int N_r, int n_seq) {
  const size_t rows = (size_t)(T + kChunk - 1) / kChunk + n_seq;
  return 2 * align_up(rows * N_r * 4, 256);
}

moe_status launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                               int n_seq, int T, int N_r, int K, int score, float alpha,
                               float* loss, float* coef, void* ws, cudaStream_t s) {
  float* psum = static_cast<float*>(ws);
  int32_t* pcnt = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) +
                                             balance_ws_bytes(T, N_r, n_seq) / 2);
  int* err = device_error_word();
  if (!err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const int softmax = score == MOE_SCORE_SOFTMAX;
  const size_t smem = (size_t)(kBalWarps + 1) * N_r * 4;
  const int blocks = (T + kChunk - 1) / kChunk;
#define MOE_BAL(v)                                                                            \
  case v:                                                                                     \
    balance_partial_kernel<v><<<blocks, 32 * kBalWarps, smem, s>>>(                           \
        logits, idx, off, n_seq, T, N_r, K, softmax, psum, pcnt);                             \
    break;
  if (blocks > 0) {
    switch (dispatch_v(N_r)) {
      MOE_BAL(1) MOE_BAL(2) MOE_BAL(4) MOE_BAL(8) MOE_BAL(16) MOE_BAL(32)
    }
    const moe_status st = cuda_check(cudaGetLastError(), "balance_partial launch");
    if (st != MOE_OK) return st;
  }
#undef MOE_BAL
  balance_final_kernel<<<n_seq, 256, 0, s>>>(psum, pcnt, off, T, N_r, K, alpha, loss, coef, err);
  return cuda_check(cudaGetLastError(), "balance_final launch");
}

size_t route_scored_bwd_ws_bytes(moe_dtype dt, int T, int d, int N_r) {
  // bf16: d_logit as bf16 planes and dE's slices; float32: d_logit itself
  return dt == MOE_BF16 ? router_grad_tc_ws_bytes(T, d, N_r) : align_up((size_t)T * N_r * 4, 256);
}

moe_status launch_route_scored_backward(const void* u, const void* E, moe_dtype dt,
                                        const float* logits, const int32_t* idx,
                                        const float* d_gate, const int32_t* off, int n_seq,
                                        const float* coef, const float* d_loss, int T, int d,
                                        int N_r, int K, int score, int renorm, float scale,
                                        const void* du_base, float* d_logit, void* du, float* dE,
                                        void* ws, cudaStream_t s) {
  const bool tc = dt == MOE_BF16;
  float* dl = d_logit || tc ? d_logit : static_cast<float*>(ws);
  const RouterPlanes pl = router_planes(T, N_r);
  __nv_bfloat16* planes = tc ? static_cast<__nv_bfloat16*>(ws) : nullptr;
  int blocks = (T + kGradWarps - 1) / kGradWarps;
  const size_t smem = (size_t)kGradWarps * N_r * 4;
  const int softmax = score == MOE_SCORE_SOFTMAX;
#define MOE_GRAD(v)                                                                           \
  case v:                                                                                     \
    router_logit_grad_kernel<v><<<blocks, 32 * kGradWarps, smem, s>>>(                        \
        logits, idx, d_gate, off, n_seq, coef, d_loss, T, N_r, K, softmax, renorm, scale, dl,  \
        planes, pl.Tp, pl.Np);                                                                \
    break;
  switch (dispatch_v(N_r)) {
    MOE_GRAD(1) MOE_GRAD(2) MOE_GRAD(4) MOE_GRAD(8) MOE_GRAD(16) MOE_GRAD(32)
  }
#undef MOE_GRAD
  moe_status st = cuda_check(cudaGetLastError(), "router_logit_grad launch");
  if (st != MOE_OK) return st;
  if (tc) return launch_router_grad_tc(u, E, T, d, N_r, du_base, du, dE, ws, s);
  const dim3 gu((d + 63) / 64, (T + 63) / 64), ge((d + 63) / 64, (N_r + 63) / 64);
  router_product_kernel<false><<<gu, 256, 0, s>>>(dl, N_r, static_cast<const float*>(E), d,
                                                  static_cast<const float*>(du_base),
                                                  static_cast<float*>(du), T, d, N_r);
  router_product_kernel<true><<<ge, 256, 0, s>>>(dl, N_r, static_cast<const float*>(u), d, nullptr,
                                                 dE, N_r, d, T);
  return cuda_check(cudaGetLastError(), "router_product launch");
}

}  // namespace moe
