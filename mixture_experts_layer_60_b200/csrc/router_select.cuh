// One token's scored routing by one warp (moe_route_scored): scores of every
// expert from its logit row, the K largest keys f32(score) + bias, optionally
// inside the best expert groups, and the gates.
//
//   sigmoid  s_i = 1 / (1 + e^-x_i)          softmax  s_i = e^(x_i - m) / sum_j e^(x_j - m)
//   key_i = f32(s_i) + b_i;  a group's score is the sum of its group_top largest keys
//   gate_k = scale * s_k  or  scale * s_k / sum of the selected s
//
// X = double: the row holds exact logits (float64 sums of products), every
// score is float64 and rounded once, so the keys are the definition's.
// X = float: the row holds float32 logits; a token with a decision closer than
// the float32 error bound below is listed for the exact pass.
//
// Lane l holds experts j*32 + l (j < V).  Order: key descending, lower index
// first on equal keys, a NaN key before every number.  Experts outside the
// kept groups are never selected; one whose key is -inf (b = -inf) is selected
// only when the kept groups hold fewer than K others.
#pragma once

#include <math.h>

#include "launch.h"

namespace moe {

// Order-preserving map of a key to an unsigned integer above 0 (-0 as +0, NaN on top).
__device__ __forceinline__ uint32_t sel_ord(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float sel_val(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// e^x for the scores: float64 in the exact pass; float32 with expf, whose
// error (2 ulp) the listing bound counts.
__device__ __forceinline__ float sel_exp(float x) { return expf(x); }
__device__ __forceinline__ double sel_exp(double x) { return exp(x); }

template <typename X>
__device__ __forceinline__ X sel_sigmoid(X x) {
  const X e = sel_exp(x < X(0) ? x : -x);      // e^-|x| never overflows; NaN stays NaN
  return (x < X(0) ? e : X(1)) / (X(1) + e);
}

template <typename X>
__device__ __forceinline__ X sel_warp_max(X v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const X w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v || w != w ? w : v;
  }
  return v;
}
template <typename X>
__device__ __forceinline__ X sel_warp_sum(X v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct SelectRule {
  int N_r, K, score, n_groups, topk_groups, group_top, renorm;
  float scale;
};

// Listing bound.  The tensor-core logits (chunks of at most 32 accumulation
// steps, joined in float32 round-to-nearest) stay within kLogitError of the
// exact ones per unit of logit magnitude: measured over N(0,1) rows at
// d = 7168 the largest error is 1.6e-6 at max|x| = 5, and the bound below
// leaves six times that.
constexpr float kLogitError = 2.5e-6f;

// What the float32 pass says about a token: whether a decision was closer than
// its error bound, and per lane the mask of the experts (bit j: j*32 + lane)
// whose exact keys can take part in it.
struct CloseCall {
  bool close;
  uint32_t mask;
};

// wk: this warp's N_r floats of shared memory (used under a group limit).
// x[j]: the lane's logits, getx(e): the logit of any expert; absmax: the
// row's largest |logit|, summed over its slices' magnitudes (X = float).
// Writes the token's idx and gate.
template <int V, typename X, typename GetX>
__device__ __forceinline__ CloseCall select_token(const X (&x)[V], GetX getx,
                                                  const float* __restrict__ bias,
                                                  const SelectRule& r, float absmax, float* wk,
                                                  int32_t* __restrict__ idx,
                                                  float* __restrict__ gate) {
  constexpr bool kExact = sizeof(X) == 8;
  const int lane = threadIdx.x & 31, N = r.N_r;
  const bool softmax = r.score == MOE_SCORE_SOFTMAX;
  X m = X(0), inv = X(1);
  if (softmax) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) m = x[j] > m || x[j] != x[j] ? x[j] : m;
    m = sel_warp_max(m);
    X z = X(0);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) z += sel_exp(x[j] - m);
    inv = sel_warp_sum(z);
  }
  float key[V];
  float wmax = 0.f, smax = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    key[j] = -INFINITY;
    if (e < N) {
      const float s = softmax ? (float)(sel_exp(x[j] - m) / inv) : (float)sel_sigmoid(x[j]);
      key[j] = bias ? s + bias[e] : s;
      if (!kExact) {
        wmax = fmaxf(wmax, s * (1.f - s));
        smax = fmaxf(smax, s);
      }
    }
  }
  // |key error| <= err + 2^-23 |key|: d s = s(1-s) dx (sigmoid), at most
  // 2 s(1-s) max|dx| (softmax), and the scores' own rounding.  A row of exact
  // zeros (a padding token) has exact scores.
  float err = 0.f, rel = 0.f;
  if (!kExact && absmax != 0.f) {
    wmax = sel_warp_max(wmax);
    smax = sel_warp_max(smax);
    err = kLogitError * fmaxf(4.f, absmax) * wmax * (softmax ? 2.f : 1.f) + 4.8e-7f * smax;
    rel = 2.4e-7f;
  }
  bool group_close = false;
  uint32_t ko[V];
#pragma unroll
  for (int j = 0; j < V; ++j) ko[j] = j * 32 + lane < N ? sel_ord(key[j]) : 0u;
  if (r.topk_groups < r.n_groups) {
    const int gs = N / r.n_groups;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) wk[j * 32 + lane] = key[j];
    __syncwarp();
    // lane g: the score of group g, its largest or its two largest keys
    uint32_t go = 0u;
    if (lane < r.n_groups) {
      uint32_t a = 0u, b = 0u;
      for (int i = 0, at = lane < gs ? lane : 0; i < gs; ++i) {   // banks spread over the lanes
        const uint32_t o = sel_ord(wk[lane * gs + at]);
        if (o > a) { b = a; a = o; } else if (o > b) b = o;
        if (++at == gs) at = 0;
      }
      float sc = sel_val(a);
      if (a == 0xffffffffu) sc = NAN;
      if (r.group_top == 2) sc = sc + (b == 0xffffffffu ? NAN : sel_val(b));
      go = sel_ord(sc);
    }
    __syncwarp();
    unsigned kept = 0;
    float last = INFINITY;
    for (int k = 0; k <= r.topk_groups; ++k) {       // one more round: the best group left out
      const uint32_t mx = __reduce_max_sync(0xffffffffu, go);
      const int bg = __reduce_min_sync(0xffffffffu, go == mx && mx ? lane : 32);
      if (mx == 0u) break;
      const float v = mx == 0xffffffffu ? NAN : sel_val(mx);
      if (k < r.topk_groups) {
        kept |= 1u << bg;
        last = v;
        if (lane == bg) go = 0u;
      } else {
        group_close = last - v < r.group_top * 2.f * err + rel * (fabsf(last) + fabsf(v));
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      if (e < N && !((kept >> (e / gs)) & 1u)) ko[j] = 0u;
    }
  }
  // K rounds of a warp arg-max; lane k % 32 keeps and writes winner k
  float lo = INFINITY, hi = -INFINITY, prev = INFINITY;
  int my_e = 0;
  for (int k = 0; k < r.K; ++k) {
    uint32_t lb = 0u;
    int lj = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (ko[j] > lb) { lb = ko[j]; lj = j; }
    const uint32_t mx = __reduce_max_sync(0xffffffffu, lb);
    const int be = __reduce_min_sync(0xffffffffu, lb == mx ? lj * 32 + lane : 0x7fffffff);
    if (!kExact) {
      const float v = mx == 0xffffffffu ? NAN : sel_val(mx);
      if (prev - v < 2.f * err + rel * (fabsf(prev) + fabsf(v))) {
        lo = fminf(lo, v);
        hi = fmaxf(hi, prev);
      }
      prev = v;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == be) ko[j] = 0u;
    if (lane == (k & 31)) {
      my_e = be;
      idx[k] = be;
    }
  }
  // gates: lane k takes slots k, k + 32, ... (it wrote their idx itself)
  const auto slot_x = [&](int k) { return getx(r.K <= 32 ? my_e : idx[k]); };
  if (!r.renorm) {
    for (int k = lane; k < r.K; k += 32) {
      const X xk = slot_x(k);
      const X s = softmax ? sel_exp(xk - m) / inv : sel_sigmoid(xk);
      gate[k] = (float)(s * (X)r.scale);
    }
  } else {
    // scores relative to the largest selected one, so that their sum cannot
    // underflow: e^(x - xm), or s(x) / s(xm) of sigmoids (e^(x - xm) to
    // e^-30 where xm < -30)
    X xm = -INFINITY;
    for (int k = lane; k < r.K; k += 32) {
      const X xk = slot_x(k);
      xm = xk > xm || xk != xk ? xk : xm;
    }
    xm = sel_warp_max(xm);
    const bool ratio = !softmax && !(xm < X(-30));
    const X sm = ratio ? sel_sigmoid(xm) : X(1);
    const auto weight = [&](int k) {
      const X xk = slot_x(k);
      return ratio ? sel_sigmoid(xk) / sm : sel_exp(xk - xm);
    };
    X sum = X(0);
    for (int k = lane; k < r.K; k += 32) sum += weight(k);
    sum = sel_warp_sum(sum);
    for (int k = lane; k < r.K; k += 32) gate[k] = (float)(weight(k) / sum * (X)r.scale);
  }
  CloseCall out;
  out.close = false;
  out.mask = 0u;
  if (!kExact) {
    // the K-th against the next
    uint32_t lb = 0u;
#pragma unroll
    for (int j = 0; j < V; ++j) lb = max(lb, ko[j]);
    const uint32_t mx = __reduce_max_sync(0xffffffffu, lb);
    if (mx) {
      const float v = mx == 0xffffffffu ? NAN : sel_val(mx);
      if (prev - v < 2.f * err + rel * (fabsf(prev) + fabsf(v))) {
        lo = fminf(lo, v);
        hi = fmaxf(hi, prev);
      }
    }
    out.close = group_close || lo <= hi;
    if (out.close) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = j * 32 + lane;
        if (e >= N) continue;
        // an expert whose key lies further than its bound from every close
        // decision cannot take part in it; a softmax score needs every logit
        const float pad = 3.f * err + 2.f * rel * fabsf(key[j]);
        if (softmax || group_close || (key[j] >= lo - pad && key[j] <= hi + pad))
          out.mask |= 1u << j;
      }
    }
  }
  return out;
}

}  // namespace moe
