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
// Renormalised gates sum to a constant, so only differences of dg_k matter: dg_k
// and G are taken relative to the dg of the token's first slot, and upstream
// values that are equal (or a single slot's) leave exactly the balance term.
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
  const float e = expf(x < 0.f ? x : -x), inv = __fdividef(1.f, 1.f + e);
  s = x < 0.f ? e * inv : inv;
  om = x < 0.f ? inv : e * inv;
}

// A token whose sigmoids sum to less than this has every logit below -69: its s'
// are formed from e^(x - xm), xm its largest logit, which is s(x) / s(xm) to a
// part in e^69 and never underflows as a whole (1 / z would be infinite below
// 2^-128).
constexpr float kSmallSum = 1e-30f;

// Row [r0, r1) of sequence q, made safe: inside [0, T], not negative.
__device__ __forceinline__ void seq_range(const int32_t* off, int q, int T, int* err, int& r0,
                                          int& r1) {
  clamp_group_rows(off, q, T, err, r0, r1);
}

// Logits x of a token (a lane's V of them; -inf: none) to e^(x - xm); their sum.
template <int V>
__device__ __forceinline__ float relative_scores(float (&x)[V]) {
  float m = -INFINITY, z = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) m = fmaxf(m, x[j]);
  m = wmax(m);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x[j] = expf(x[j] - m);
    z += x[j];
  }
  return wsum(z);
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

// Tokens per block of the balance sums (T 8192, 256 experts and T 50000, 61: 14
// and 19 us; 128 tokens, fewer and longer blocks, 16 and 20).
constexpr int kChunk = 64;

// Partial sums of one (chunk of tokens, sequence) pair, row chunk + sequence:
// along the pairs either number grows, so the rows are distinct.  Each of W
// warps takes U tokens at a time (their loads and reductions overlap: a token
// alone is a chain of latencies), warps and tokens in a fixed order.  Reads
// each logit once.
template <int V, int W>
__global__ void __launch_bounds__(32 * W) balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ off, int n_seq, int T, int N, int K, int softmax,
    float2* __restrict__ part) {
  constexpr int U = V <= 2 ? 4 : V <= 8 ? 2 : 1;
  extern __shared__ float sm[];                 // [W][N] sums, then [N] counts
  int* cnt = reinterpret_cast<int*>(sm + W * N);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  const int t0 = blockIdx.x * kChunk, t1 = min(T, t0 + kChunk);
  // the sequence of the chunk's first token: offsets counted side by side (a
  // search is a chain of dependent loads), unless there are very many
  int q;
  if (off && n_seq <= 4096) {
    int c = 0;
    for (int i0 = 0; i0 < n_seq; i0 += 32 * W) {
      const int i = i0 + threadIdx.x;
      c += __syncthreads_count(i < n_seq && off[i] <= t0);
    }
    q = c - 1;
  } else {
    q = seq_at(off, n_seq, t0);
  }
  if (q < 0) q = 0;
  for (; q < n_seq; ++q) {
    int r0, r1;
    seq_range(off, q, T, nullptr, r0, r1);
    if (r0 >= t1) break;
    const bool last = r1 >= t1;                 // the next sequence starts in a later chunk
    r0 = max(r0, t0);
    r1 = min(r1, t1);
    if (r0 >= r1) continue;
    for (int i = threadIdx.x; i < N; i += blockDim.x) cnt[i] = 0;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    __syncthreads();
    for (int tb = r0 + warp * U; tb < r1; tb += W * U) {
      float s[U][V], z[U], m[U];
#pragma unroll
      for (int c = 0; c < U; ++c) {
        m[c] = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = j * 32 + lane;
          s[c][j] = tb + c < r1 && e < N ? logits[(size_t)(tb + c) * N + e] : -INFINITY;
          m[c] = fmaxf(m[c], s[c][j]);
        }
      }
      // the tokens' slots: whole numbers, in any order
      const int nk = min(U, r1 - tb) * K;
      for (int k = lane; k < nk; k += 32) {
        const int e = idx[(size_t)tb * K + k];
        if (e >= 0 && e < N) atomicAdd(&cnt[e], 1);
      }
      if (softmax) {
#pragma unroll
        for (int c = 0; c < U; ++c) m[c] = wmax(m[c]);
      }
#pragma unroll
      for (int c = 0; c < U; ++c) {
        z[c] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (tb + c < r1 && j * 32 + lane < N) {
            float om;
            if (softmax) s[c][j] = expf(s[c][j] - m[c]);
            else sigmoid_pair(s[c][j], s[c][j], om);
            z[c] += s[c][j];
          } else {
            s[c][j] = 0.f;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < U; ++c) z[c] = wsum(z[c]);
      if (!softmax) {
#pragma unroll
        for (int c = 0; c < U; ++c) {
          if (tb + c >= r1 || !(z[c] < kSmallSum)) continue;
          const float* row = logits + (size_t)(tb + c) * N;
#pragma unroll
          for (int j = 0; j < V; ++j) s[c][j] = j * 32 + lane < N ? row[j * 32 + lane] : -INFINITY;
          z[c] = relative_scores(s[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const float inv = tb + c < r1 ? 1.f / z[c] : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(s[c][j], inv, acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) sm[warp * N + j * 32 + lane] = acc[j];
    __syncthreads();
    float2* row = part + (size_t)(blockIdx.x + q) * N;
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) a += sm[w * N + i];
      row[i] = make_float2(a, __int_as_float(cnt[i]));
    }
    if (last) break;
    __syncthreads();
  }
}

// One block per sequence: coef and loss from the partial rows.  The block's
// threads are groups of `cols` columns (a power of two); group g sums rows
// g, g + groups, ... in float64, and the groups' sums join in group order.
constexpr int kFinalThreads = 1024;
__global__ void __launch_bounds__(kFinalThreads) balance_final_kernel(
    const float2* __restrict__ part, const int32_t* __restrict__ off, int T, int N, int K,
    int cols, float alpha, float* __restrict__ loss, float* __restrict__ coef, int* err) {
  __shared__ double red[32];
  __shared__ double sp[kFinalThreads];
  __shared__ int sc[kFinalThreads];
  const int q = blockIdx.x, g = threadIdx.x / cols, i = threadIdx.x % cols;
  const int groups = kFinalThreads / cols;
  pdl_wait();
  int r0, r1;
  seq_range(off, q, T, threadIdx.x == 0 ? err : nullptr, r0, r1);
  const int n = r1 - r0;
  double p = 0.0;
  int c = 0;
  if (n > 0 && i < N) {
    const float2* row = part + (size_t)q * N + i;
    const int k1 = (r1 - 1) / kChunk;
#pragma unroll 4
    for (int k = r0 / kChunk + g; k <= k1; k += groups) {
      const float2 v = row[(size_t)k * N];
      p += (double)v.x;
      c += __float_as_int(v.y);
    }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  double term = 0.0;
  if (g == 0 && i < N) {
    for (int k = 1; k < groups; ++k) {
      p += sp[k * cols + i];
      c += sc[k * cols + i];
    }
    // alpha f_i / n with f_i = N_r c / (K n): rounded once
    const double cf = n > 0 ? (double)alpha * N * c / ((double)K * n * n) : 0.0;
    coef[(size_t)q * N + i] = (float)cf;
    term = cf * p;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int w = 0; w < kFinalThreads / 32; ++w) a += red[w];
    loss[q] = (float)a;
  }
}

// ---------------------------------------------------------------- logit gradient
// A warp per token, bound by the logits, planes and d_logit it moves and by
// some 600 instructions a token.  planes: d_logit as bf16 planes too
// (router_grad_tc.cu).  PAIR: a lane holds two neighbouring experts of every
// 64 (8-byte loads and stores, rounded two at a time) where N_r is even and
// the rows are 8-byte aligned; else one of every 32.
constexpr int kGradWarps = 4;

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int V, bool PAIR>
__global__ void __launch_bounds__(32 * kGradWarps) router_logit_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const float* __restrict__ d_gate, const int32_t* __restrict__ off, int n_seq,
    const float* __restrict__ coef, const float* __restrict__ d_loss, int T, int N, int K,
    int softmax, int renorm, float scale, float* __restrict__ d_logit,
    __nv_bfloat16* __restrict__ planes, int Tp, int Np) {
  extern __shared__ float sm[];
  pdl_trigger();
  // the planes' rows past the last token
  if (planes) {
    const long long pad = (long long)(Tp - T) * Np;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < 3 * pad;
         i += (long long)gridDim.x * blockDim.x)
      planes[((i / pad) * Tp + T) * (long long)Np + i % pad] = __float2bfloat16_rn(0.f);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = sm + (size_t)warp * N;          // the slots' terms by expert
  const auto expert = [&](int j) { return PAIR ? (j >> 1) * 64 + 2 * lane + (j & 1) : j * 32 + lane; };
  for (int t = blockIdx.x * kGradWarps + warp; t < T; t += gridDim.x * kGradWarps) {
    const float* lrow = logits + (size_t)t * N;
    // the slot of this lane (K <= 32: one; else the loops below come back)
    float s[V], om[V], m = -INFINITY, z = 0.f;
    if (PAIR) {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const int e = expert(j);
        const float2 v = e < N ? *reinterpret_cast<const float2*>(lrow + e)
                               : make_float2(-INFINITY, -INFINITY);
        s[j] = v.x;
        s[j + 1 < V ? j + 1 : j] = v.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = expert(j) < N ? lrow[expert(j)] : -INFINITY;
    }
    if (d_gate)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (expert(j) < N) row[expert(j)] = 0.f;
    if (softmax) {
#pragma unroll
      for (int j = 0; j < V; ++j) m = fmaxf(m, s[j]);
      m = wmax(m);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (expert(j) < N) {
        if (softmax) { s[j] = expf(s[j] - m); om[j] = 1.f; }
        else sigmoid_pair(s[j], s[j], om[j]);
        z += s[j];
      } else {
        s[j] = 0.f;
        om[j] = 0.f;
      }
    }
    z = wsum(z);
    if (!softmax && z < kSmallSum) {
      // s (1 - s) / sum s is e^(x - xm) / sum e^(x - xm) here, and 1 - s is 1
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = expert(j);
        s[j] = e < N ? lrow[e] : -INFINITY;
        om[j] = 1.f;
      }
      z = relative_scores(s);
    }
    const float inv = 1.f / z;
    if (softmax) {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] *= inv;
    }
    // balance term
    float q[V], Q = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = 0.f;
    if (coef) {
      const int sq = seq_at(off, n_seq, t);
      int r0 = 0, r1 = 0;
      if (sq >= 0) seq_range(off, sq, T, nullptr, r0, r1);
      if (t >= r0 && t < r1) {
        const float dl = d_loss ? d_loss[sq] : 1.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (expert(j) < N) q[j] = dl * coef[(size_t)sq * N + expert(j)];
          Q = fmaf(s[j], q[j], Q);
        }
        Q = wsum(Q);
        if (!softmax) Q *= inv;
      }
    }
    // the slots' terms, by expert
    float R = 0.f;
    if (d_gate) {
      const auto slot = [&](int k, int& e, float& dg, float& x) {   // e < 0: left out
        e = k < K ? idx[(size_t)t * K + k] : -1;
        if (e >= N) e = -1;
        dg = e >= 0 ? scale * d_gate[(size_t)t * K + k] : 0.f;
        x = e >= 0 ? lrow[e] : -INFINITY;
      };
      int e = -1;
      float dg = 0.f, x = -INFINITY, xm = -INFINITY, sxm = 1.f, den = 1.f, G = 0.f, dum;
      float dg0 = 0.f;                                     // dg of the first slot that counts
      bool ratio = false, first = true;
      const auto weight = [&](float v) {                   // the score over the largest one
        if (!ratio) return expf(v - xm);
        float a, b;
        sigmoid_pair(v, a, b);
        return __fdividef(a, sxm);
      };
      if (renorm) {
        for (int k0 = 0; k0 < K; k0 += 32) {
          slot(k0 + lane, e, dg, x);
          if (e >= 0) xm = x > xm || x != x ? x : xm;
          const unsigned counts = __ballot_sync(0xffffffffu, e >= 0);
          if (first && counts) {
            dg0 = __shfl_sync(0xffffffffu, dg, __ffs(counts) - 1);
            first = false;
          }
        }
        xm = wmax(xm);
        ratio = !softmax && !(xm < -30.f);
        if (ratio) sigmoid_pair(xm, sxm, dum);
        float w = 0.f, wd = 0.f;
        for (int k0 = 0; k0 < K; k0 += 32) {
          if (K > 32) slot(k0 + lane, e, dg, x);
          if (e >= 0) {
            const float v = weight(x);
            w += v;
            wd = fmaf(v, dg - dg0, wd);
          }
        }
        den = wsum(w);
        G = wsum(wd) / den;
      }
      for (int k0 = 0; k0 < K; k0 += 32) {
        if (K > 32 || !renorm) slot(k0 + lane, e, dg, x);
        float v = 0.f;
        if (e >= 0) {
          float a, b;
          if (softmax) { a = expf(x - m) * inv; b = 1.f; }
          else sigmoid_pair(x, a, b);
          if (renorm) v = weight(x) / den * b * (dg - dg0 - G);
          else { v = a * b * dg; R += softmax ? v : 0.f; }
        }
        __syncwarp();
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (__all_sync(0xffffffffu, e < 0 || (same & (same - 1u)) == 0u)) {
          if (e >= 0) row[e] += v;
        } else {
          // an expert more than once: its slots one after the other
          for (int k = 0; k < 32; ++k) {
            if (lane == k && e >= 0) row[e] += v;
            __syncwarp();
          }
        }
      }
      R = wsum(R);
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert(j);
      float v = softmax ? s[j] * (q[j] - Q - R) : s[j] * om[j] * (q[j] - Q) * inv;
      if (d_gate && e < N) v += row[e];
      s[j] = e < N ? v : 0.f;
    }
    __syncwarp();                                  // the row is rewritten for the next token
    if (PAIR) {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        constexpr int last = V - 1;
        const int e = expert(j), j1 = j + 1 <= last ? j + 1 : j;
        if (d_logit && e < N)
          *reinterpret_cast<float2*>(d_logit + (size_t)t * N + e) = make_float2(s[j], s[j1]);
        if (planes && e < Np) {
          // hi + mid + lo: 24 bits in three roundings; an infinity stays in hi
          const uint32_t hi = bf16x2(s[j], s[j1]);
          const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xffff0000u);
          const float a0 = fabsf(h0) < INFINITY ? s[j] - h0 : 0.f;
          const float a1 = fabsf(h1) < INFINITY ? s[j1] - h1 : 0.f;
          const uint32_t mid = bf16x2(a0, a1);
          const uint32_t lo = bf16x2(a0 - __uint_as_float(mid << 16),
                                     a1 - __uint_as_float(mid & 0xffff0000u));
          uint32_t* at = reinterpret_cast<uint32_t*>(planes + (size_t)t * Np + e);
          const size_t plane = (size_t)Tp * Np / 2;
          at[0] = hi;
          at[plane] = mid;
          at[2 * plane] = lo;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = expert(j);
        if (d_logit && e < N) d_logit[(size_t)t * N + e] = s[j];
        if (planes && e < Np) {
          const __nv_bfloat16 hi = __float2bfloat16_rn(s[j]);
          const float fh = __bfloat162float(hi);
          const float r1 = fabsf(fh) < INFINITY ? s[j] - fh : 0.f;
          const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
          const size_t at = (size_t)t * Np + e, plane = (size_t)Tp * Np;
          planes[at] = hi;
          planes[at + plane] = mid;
          planes[at + 2 * plane] = __float2bfloat16_rn(r1 - __bfloat162float(mid));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- CUDA-core products (float32 u, E)
// C[m, n] = base[m, n] + sum_k A(m, k) B[k, n], A(m, k) = A[m*lda + k] (or
// A[k*lda + m] with TA) float32, B row-major; k in slices of blockIdx.y, each
// with a C of its own.  64 x 64 tile per block, 4 x 4 outputs a thread, 16
// steps of k staged at a time, the next ones on their way meanwhile; every 256
// steps the running sums join a second set, so that a long sum keeps its low
// bits.
template <bool TA>
__global__ void __launch_bounds__(256) router_product_kernel(
    const float* __restrict__ A, int lda, const float* __restrict__ B, int ldb,
    const float* base, float* C, int M, int N, int Kd) {
  __shared__ float sa[16][64 + 4], sb[16][64 + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n_n = (N + 63) / 64;               // tiles in one grid dimension: M may be many tokens
  const int m0 = (int)(blockIdx.x / n_n) * 64, n0 = (int)(blockIdx.x % n_n) * 64;
  const int kb = (int)((long long)Kd * blockIdx.y / gridDim.y);
  const int ke = (int)((long long)Kd * (blockIdx.y + 1) / gridDim.y);
  float ra[4], rb[4];
  const auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = j * 256 + tid;
      const int ka = k0 + (TA ? i >> 6 : i & 15), m = m0 + (TA ? i & 63 : i >> 4);
      const int k = k0 + (i >> 6), n = n0 + (i & 63);
      ra[j] = ka < ke && m < M ? (TA ? A[(size_t)ka * lda + m] : A[(size_t)m * lda + ka]) : 0.f;
      rb[j] = k < ke && n < N ? B[(size_t)k * ldb + n] : 0.f;
    }
  };
  float acc[4][4] = {}, tot[4][4] = {};
  fetch(kb);
  for (int k0 = kb; k0 < ke; k0 += 16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = j * 256 + tid;
      sa[TA ? i >> 6 : i & 15][TA ? i & 63 : i >> 4] = ra[j];
      sb[i >> 6][i & 63] = rb[j];
    }
    __syncthreads();
    if (k0 + 16 < ke) fetch(k0 + 16);
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
    if (((k0 - kb) & 255) == 240 || k0 + 16 >= ke) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) { tot[i][j] += acc[i][j]; acc[i][j] = 0.f; }
    }
  }
  float* out = C + (size_t)blockIdx.y * M * N;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) {
        const size_t at = (size_t)m * N + n;
        out[at] = tot[i][j] + (base ? base[at] : 0.f);
      }
    }
}

// dE = the slices' sums, in order.
__global__ void __launch_bounds__(256) router_slices_kernel(const float4* __restrict__ P, int S,
                                                            int n4, float4* __restrict__ dE) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 a = P[i];
  for (int s = 1; s < S; ++s) {
    const float4 b = P[(size_t)s * n4 + i];
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  dE[i] = a;
}

// Slices of the tokens for a float32 dE: two blocks an SM, at least 256 tokens
// each.  (The whole float32 backward at T 1262, d 512, 317 experts: 70 us, 192 in
// one slice; T 8192, d 2048, 64 experts: 219 and 1500.)
int de_slices(int T, int d, int N_r) {
  const int tiles = (d + 63) / 64 * ((N_r + 63) / 64);
  const int most = (2 * 148 + tiles - 1) / tiles, by_rows = T / 256 + (T % 256 != 0);
  return most < by_rows ? most : by_rows;
}

int dispatch_v(int N) {
  const int V = (N + 31) / 32;
  return V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : V <= 16 ? 16 : 32;
}

}  // namespace

// Partial rows (sum and count of every expert): one for every (chunk,
// sequence) pair.
size_t balance_ws_bytes(int T, int N_r, int n_seq) {
  const size_t rows = (size_t)(T + kChunk - 1) / kChunk + n_seq;
  return align_up(rows * N_r * sizeof(float2), 256);
}

moe_status launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                               int n_seq, int T, int N_r, int K, int score, float alpha,
                               float* loss, float* coef, void* ws, cudaStream_t s) {
  float2* part = static_cast<float2*>(ws);
  int* err = device_error_word();
  if (!err) return fail(MOE_ERR_CUDA, "device error word unavailable");
  const int softmax = score == MOE_SCORE_SOFTMAX;
  const int blocks = (T + kChunk - 1) / kChunk;
  // sums of W warps and the counts in at most 36 KB
#define MOE_BAL(v, w)                                                                         \
  case v:                                                                                     \
    balance_partial_kernel<v, w><<<blocks, 32 * w, (size_t)(w + 1) * N_r * 4, s>>>(           \
        logits, idx, off, n_seq, T, N_r, K, softmax, part);                                   \
    break;
  if (blocks > 0) {
    switch (dispatch_v(N_r)) {
      MOE_BAL(1, 16) MOE_BAL(2, 16) MOE_BAL(4, 16) MOE_BAL(8, 32) MOE_BAL(16, 16) MOE_BAL(32, 8)
    }
    const moe_status st = cuda_check(cudaGetLastError(), "balance_partial launch");
    if (st != MOE_OK) return st;
  }
#undef MOE_BAL
  int cols = 32;
  while (cols < N_r) cols *= 2;
  return launch_after(balance_final_kernel, dim3(n_seq), dim3(kFinalThreads), 0, s, 1,
                      "balance_final launch", part, off, T, N_r, K, cols, alpha, loss, coef, err);
}

size_t route_scored_bwd_ws_bytes(moe_dtype dt, int T, int d, int N_r) {
  // bf16: d_logit as bf16 planes and dE's slices; float32: d_logit itself and dE's slices
  if (dt == MOE_BF16) return router_grad_tc_ws_bytes(T, d, N_r);
  const int S = de_slices(T, d, N_r);
  return align_up((size_t)T * N_r * 4, 256) + (S > 1 ? (size_t)S * N_r * d * 4 : 0);
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
  const bool pair = N_r % 2 == 0 && N_r > 32 && reinterpret_cast<uintptr_t>(logits) % 8 == 0 &&
                    reinterpret_cast<uintptr_t>(d_logit) % 8 == 0;
#define MOE_GRAD_RUN(v, p)                                                                    \
  router_logit_grad_kernel<v, p><<<blocks, 32 * kGradWarps, smem, s>>>(                       \
      logits, idx, d_gate, off, n_seq, coef, d_loss, T, N_r, K, softmax, renorm, scale, dl,   \
      planes, pl.Tp, pl.Np)
#define MOE_GRAD(v)                                                                           \
  case v:                                                                                     \
    if (pair) MOE_GRAD_RUN(v, (v > 1));                                                       \
    else MOE_GRAD_RUN(v, false);                                                              \
    break;
  switch (dispatch_v(N_r)) {
    MOE_GRAD(1) MOE_GRAD(2) MOE_GRAD(4) MOE_GRAD(8) MOE_GRAD(16) MOE_GRAD(32)
  }
#undef MOE_GRAD_RUN
#undef MOE_GRAD
  moe_status st = cuda_check(cudaGetLastError(), "router_logit_grad launch");
  if (st != MOE_OK) return st;
  if (tc) return launch_router_grad_tc(u, E, T, d, N_r, du_base, du, dE, ws, s);
  const unsigned nd = (d + 63) / 64, gu = nd * ((T + 63) / 64), ge = nd * ((N_r + 63) / 64);
  router_product_kernel<false><<<gu, 256, 0, s>>>(dl, N_r, static_cast<const float*>(E), d,
                                                  static_cast<const float*>(du_base),
                                                  static_cast<float*>(du), T, d, N_r);
  const int S = de_slices(T, d, N_r);
  float* part = S > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                                 align_up((size_t)T * N_r * 4, 256))
                      : dE;
  router_product_kernel<true><<<dim3(ge, S), 256, 0, s>>>(dl, N_r, static_cast<const float*>(u), d,
                                                          nullptr, part, N_r, d, T);
  if (S > 1) {
    const int n4 = N_r * d / 4;                // d is a multiple of 64
    router_slices_kernel<<<(n4 + 255) / 256, 256, 0, s>>>(
        reinterpret_cast<const float4*>(part), S, n4, reinterpret_cast<float4*>(dE));
  }
  return cuda_check(cudaGetLastError(), "router_product launch");
}

}  // namespace moe
