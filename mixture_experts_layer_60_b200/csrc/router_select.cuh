// One token's scored routing (moe_route_scored), by a warp or by a block: scores of every
// expert from its logit row, the K largest keys f32(score) + bias, optionally
// inside the best expert groups, and the gates.
//
//   sigmoid  s_i = 1 / (1 + e^-x_i)          softmax  s_i = e^(x_i - m) / sum_j e^(x_j - m)
//   key_i = f32(s_i) + b_i;  a group's score is the sum of its group_top largest keys
//   gate_k = scale * s_k  or  scale * s_k / sum of the selected s
//
// Warp: lane l holds experts j*32 + l (j < V) and K rounds of an arg-max pick
// the experts (fewest instructions: many tokens).  Block: a thread per expert
// counts the keys before its own, which is its place in the order (no rounds
// and little code to fetch: few tokens, and the exact pass).  Order: key descending, lower index
// first on equal keys, a NaN key before every number.  Experts outside the
// kept groups are never selected; one whose key is -inf (b = -inf) is selected
// only when the kept groups hold fewer than K others.
//
// Exactness.  A token is first selected from float32 keys.  A decision (two
// neighbours in the order, the last kept against the best excluded group)
// whose gap is inside the keys' error bound is open; the experts that can take
// part in it get their exact key (float64 logit and score, rounded once) and
// the token is selected again, until no decision is open.  Equal exact keys
// are ties of the definition.
#pragma once

#include <math.h>

#include "launch.h"

namespace moe {

// Order-preserving map of a key to an unsigned integer above 0 (-0 as +0, NaN on top).
__device__ __forceinline__ uint32_t sel_ord(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float sel_val(uint32_t o) {
  if (o == 0xffffffffu) return NAN;
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

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

// Bound on a tensor-core logit's error, from the square sums of the token's and
// of the largest expert's values.  A step of 16 products cuts each of them at
// 2^-25 and its sum at 2^-23 of the step's largest product or running sum A (a
// model, fitted to large values held over chains of small ones): at most 6e-7 A.
// A chunk sums 8 steps from zero, with A <= |u| |E| over the chunk's columns, which
// summed over the chunks is at most |u| |E| of the whole rows: 4.8e-6 |u| |E|.  (A
// sum that is large across the chunks loses at most half a step at each join
// instead, 4e-6 over 16384 columns.)  Rows made for it reach 3.7e-6, N(0,1) rows
// 6e-8.  A bound that follows the logits instead lists fewer of those and is wrong
// where large products cancel.
constexpr float kLogitError = 5e-6f;
// Past this the scores' error is no longer their slope's: every logit is made exact.
constexpr float kWideError = 0.25f;
__device__ __forceinline__ float logit_error(float u2, float e2) {
  if (u2 == 0.f || (e2 == 0.f && u2 < INFINITY)) return 0.f;   // zeros: exact
  if (u2 != u2) return 1e-30f;                                 // every logit is NaN, exactly
  const float e = kLogitError * sqrtf(u2) * sqrtf(e2);
  return e <= kWideError ? fmaxf(e, 1e-30f) : INFINITY;
}

// Per token: the softmax's largest logit and sum, and the bound on a float32
// key's error against the others', from its score s:
//   slope s (1 - s)   sigmoid; softmax with a bias (twice: its sum's error too)
//   slope s           softmax without: the sum's error scales every score alike
// plus `flat` for the float32 functions and kKeyRounding |key|.  top: the largest
// (0: exact).
struct TokenScale {
  float m, z, slope, flat, top;
  bool whole;                    // slope s
  float b_lo, b_hi;              // least and largest bias
  __device__ __forceinline__ float score_error(float s) const {
    return fmaf(slope, whole ? s : s * (1.f - s), flat);
  }
  // Of any expert whose key lies between lo and hi (so its score between lo - b_hi
  // and hi - b_lo).
  __device__ __forceinline__ float range_error(float lo, float hi) const {
    const float s0 = lo - b_hi, s1 = hi - b_lo;
    const float s = s0 > 0.5f ? fminf(s0, 1.f) : s1 < 0.5f ? fmaxf(s1, 0.f) : 0.5f;
    return whole ? fminf(top, fmaf(slope, s1, flat)) : fminf(top, fmaf(slope, s * (1.f - s), flat));
  }
};
constexpr float kKeyRounding = 1.2e-7f;
__device__ __forceinline__ TokenScale exact_scale() {
  return TokenScale{0.f, 1.f, 0.f, 0.f, 0.f, true, 0.f, 0.f};
}
// The slope for logits off by at most dx <= kWideError, over which a score's own
// slope grows by at most e^(4 dx) <= 1 + 8 dx.
__device__ __forceinline__ float error_slope(float dx, bool softmax, bool bias) {
  return dx * fmaf(8.f, dx, 1.f) * (softmax && bias ? 2.f : 1.f);
}
// What float32 functions may lose of a score below the normal range.
constexpr float kFloor = 2.4e-38f;
// A key's whole error (an infinite key has none).
__device__ __forceinline__ float key_error(float score_error, float key) {
  return fabsf(key) < INFINITY ? fmaf(kKeyRounding, fabsf(key), score_error) : 0.f;
}

// Float32 keys and scores of a row of float32 logits.  logit_err: bound on
// their error (past kWideError: of no use, the caller has every logit made
// exact).  d s = s(1-s) dx (sigmoid), at most 2 s(1-s) max|dx| (softmax);
// the fast exponential and division cost a score of size s at most 8 * 2^-23 s
// (the exponential's argument error, |x| 2^-23, is weighted by s(1-s) or by
// s ln(smax / s) < 0.4 smax).
template <int V>
__device__ __forceinline__ TokenScale select_keys(const float (&x)[V], const float* bias,
                                                  const SelectRule& r, float logit_err,
                                                  float (&sc)[V], float (&key)[V]) {
  const int lane = threadIdx.x & 31, N = r.N_r;
  TokenScale ts = exact_scale();
  const bool softmax = r.score == MOE_SCORE_SOFTMAX;
  if (logit_err == 0.f) {
    // a row of exact zeros (a padding token): every score is 1/2, or 1/N_r
    const float s0 = softmax ? 1.f / (float)N : 0.5f;
    ts.z = (float)N;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      sc[j] = e < N ? s0 : 0.f;
      key[j] = e < N ? (bias ? s0 + bias[e] : s0) : -INFINITY;
    }
    return ts;
  }
  if (softmax) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < N) m = x[j] > m || x[j] != x[j] ? x[j] : m;
    ts.m = sel_warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sc[j] = j * 32 + lane < N ? __expf(x[j] - ts.m) : 0.f;
      z += sc[j];
    }
    ts.z = sel_warp_sum(z);
    const float inv = __fdividef(1.f, ts.z);
#pragma unroll
    for (int j = 0; j < V; ++j) sc[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float e = __expf(x[j] < 0.f ? x[j] : -x[j]);
      sc[j] = j * 32 + lane < N ? __fdividef(x[j] < 0.f ? e : 1.f, 1.f + e) : 0.f;
    }
  }
  ts.whole = softmax && !bias;
  float w = 0.f, s = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    key[j] = e < N ? (bias ? sc[j] + bias[e] : sc[j]) : -INFINITY;
    w = fmaxf(w, ts.whole ? sc[j] : sc[j] * (1.f - sc[j]));
    s = fmaxf(s, sc[j]);
  }
  // non-negative floats compare as integers
  w = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(w)));
  s = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(s)));
  ts.slope = error_slope(fminf(logit_err, kWideError), softmax, bias != nullptr);
  ts.flat = fmaf(9.6e-7f, s, kFloor);
  ts.top = fmaf(ts.slope, w, ts.flat);
  return ts;
}

// What a warp's selection decided: lane k's expert of slot k (k < 32; every
// slot is in idx), whether a decision is open, the range of keys that the open
// decisions of the order lie in (none: lo > hi), and this lane's experts (bit j)
// that an open choice of groups waits for.
struct Selection {
  int e;
  bool open;
  float lo, hi;
  uint32_t mask;
};

// Whether an expert with this key can take part in the open decisions.
__device__ __forceinline__ bool takes_part(float key, float err, float lo, float hi) {
  return key + err >= lo && key - err <= hi;
}

// The sizes at which a group's keys and their sum are rounded (a sum may be far
// smaller than its keys); 0 where one is infinite: no rounding moves that score.
__device__ __forceinline__ float group_rounding(float a, float b) {
  const float v = fabsf(a) + fabsf(b) + fabsf(a + b);
  return v < INFINITY ? v : 0.f;
}

// key: this lane's keys, off by what ts says.  wk: N_r floats of shared memory for
// this warp.  A decision is first held against the largest error of all (ts.top);
// where that leaves it open, against the largest of the keys that it is among
// (saturated scores have next to none).
template <int V>
__device__ __forceinline__ Selection select_core(const float (&key)[V], const TokenScale& ts,
                                                 const float* bias, const SelectRule& r, float* wk,
                                                 int32_t* __restrict__ idx) {
  const int lane = threadIdx.x & 31, N = r.N_r;
  const float err = ts.top, rel = err > 0.f ? kKeyRounding : 0.f;
  Selection out{0, false, INFINITY, -INFINITY, 0u};
  uint32_t ko[V];
#pragma unroll
  for (int j = 0; j < V; ++j) ko[j] = j * 32 + lane < N ? sel_ord(key[j]) : 0u;
  if (r.topk_groups < r.n_groups) {
    const int gs = N / r.n_groups;
    // e / gs as a product: exact while e < 1024 and e * gs < 2^22
    const uint32_t inv_gs = ((1u << 22) + gs - 1) / gs;
    const bool two = r.group_top == 2;
    uint32_t ga = 0u, gb = 0u;                      // lane g: the largest keys of group g
    if (gs % 32 == 0) {
      const int per = gs / 32;                      // a group is `per` whole rows of lanes
      uint32_t a = 0u, b = 0u;
      int left = per, g = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * 32 < N) {
          b = max(b, min(a, ko[j]));
          a = max(a, ko[j]);
          if (--left == 0) {
            const uint32_t m1 = __reduce_max_sync(0xffffffffu, a);
            uint32_t m2 = 0u;
            if (two) {
              // one holder of the largest key steps back to its second
              const int who = __ffs(__ballot_sync(0xffffffffu, a == m1)) - 1;
              m2 = __reduce_max_sync(0xffffffffu, lane == who ? b : a);
            }
            if (lane == g) { ga = m1; gb = m2; }
            a = b = 0u;
            left = per;
            ++g;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * 32 + lane < N) wk[j * 32 + lane] = key[j];
      __syncwarp();
      if (lane < r.n_groups) {
        for (int i = 0, at = lane < gs ? lane : 0; i < gs; ++i) {   // banks spread over the lanes
          const uint32_t o = sel_ord(wk[lane * gs + at]);
          gb = max(gb, min(ga, o));
          ga = max(ga, o);
          if (++at == gs) at = 0;
        }
      }
      __syncwarp();
    }
    uint32_t go = 0u;
    float gm = 0.f;
    if (lane < r.n_groups) {
      const float ka = sel_val(ga), kb = two ? sel_val(gb) : 0.f;
      go = sel_ord(two ? ka + kb : ka);
      gm = group_rounding(ka, kb);
    }
    // what rounding the keys and their sum moves a group's score by
    const float grel = rel * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(gm)));
    unsigned kept = 0;
    float last = INFINITY, next = 0.f;
    const float gsc = lane < r.n_groups ? sel_val(go) : NAN;
    for (int k = 0; k <= r.topk_groups; ++k) {       // one more round: the best group left out
      const uint32_t mx = __reduce_max_sync(0xffffffffu, go);
      if (mx == 0u) break;
      const int bg = __ffs(__ballot_sync(0xffffffffu, go == mx)) - 1;
      next = sel_val(mx);
      if (k < r.topk_groups) {
        kept |= 1u << bg;
        last = next;
        if (lane == bg) go = 0u;
      } else {
        out.open = last - next < 2.f * (r.group_top * err + grel);
      }
    }
    if (out.open) {
      // the groups near the border, and the last keys that their scores count
      const float wide = 4.f * (r.group_top * err + grel);
      float need = gsc >= next - wide && gsc <= last + wide ? sel_val(two ? gb : ga) : INFINITY;
      // the largest error of the experts that can enter those scores
      const bool near = need < INFINITY;
      const float low = -sel_warp_max(near ? -need : -INFINITY);
      const float high = sel_warp_max(near ? sel_val(ga) : -INFINITY);
      const float own = ts.range_error(low - 2.f * err - 2.f * rel * fabsf(low), high);
      out.open = last - next < 2.f * (r.group_top * own + grel);
      // the members that can enter the scores of the groups near the border
      const float room = 4.f * (r.group_top * own + grel);
      if (!out.open || !(gsc >= next - room && gsc <= last + room)) need = INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 32 + lane, g = e < (uint32_t)N ? e * inv_gs >> 22 : 0u;
        const float want = __shfl_sync(0xffffffffu, need, g);
        if (e < (uint32_t)N && key[j] >= want - 2.f * own - 2.f * rel * fabsf(want))
          out.mask |= 1u << j;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = j * 32 + lane;
      if (e < (uint32_t)N && !((kept >> (e * inv_gs >> 22)) & 1u)) ko[j] = 0u;
    }
  }
  // K rounds of a warp arg-max, and one more for the best expert left out;
  // lane k % 32 keeps and writes winner k
  float prev = INFINITY, won = 0.f;
  int n = 0;
  const bool few = r.K < 32;                         // a lane for every round
  for (int k = 0; k <= r.K; ++k) {
    uint32_t lb = ko[0];
    int lj = 0;
#pragma unroll
    for (int j = 1; j < V; ++j)
      if (ko[j] > lb) { lb = ko[j]; lj = j; }
    const uint32_t mx = __reduce_max_sync(0xffffffffu, lb);
    if (mx == 0u) break;                             // nothing eligible is left
    const int be = __reduce_min_sync(0xffffffffu, lb == mx ? lj * 32 + lane : 0x7fffffff);
    const float v = sel_val(mx);
    if (!few) {                                      // by the largest error of all
      const float ev = key_error(err, v), ep = key_error(err, prev);
      if (err > 0.f && prev - v < ev + ep) {
        out.lo = fminf(out.lo, v - ev);
        out.hi = fmaxf(out.hi, prev + ep);
      }
      prev = v;
    }
    if (lane == (k & 31)) {
      won = v;
      if (few || k < r.K) out.e = be;
      if (k < r.K) idx[k] = be;
    }
    n = k + 1;
    if (k == r.K) break;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == be) ko[j] = 0u;
  }
  if (few && err > 0.f) {
    // lane k: winner k against the one before, each by its own error
    float ke = 0.f;
    if (lane < n) {
      const float be = bias ? bias[out.e] : 0.f;
      // a score regained from its key is off by the key's rounding
      ke = key_error(fabsf(be) <= 4.f ? ts.score_error(won - be) + 5e-7f * ts.slope : err, won);
    }
    const float lo = won - ke, hi = won + ke;
    const float up_lo = __shfl_up_sync(0xffffffffu, lo, 1), up_hi = __shfl_up_sync(0xffffffffu, hi, 1);
    if (lane > 0 && lane < n && hi > up_lo) {
      out.lo = lo;
      out.hi = up_hi;
    }
    // the last one kept against every expert left out: none has a larger key than
    // the best of them, nor an error past the largest
    float rest = __shfl_sync(0xffffffffu, won + key_error(err, won), r.K & 31);
    if (n <= r.K) rest = -INFINITY;
    const float last_lo = __shfl_sync(0xffffffffu, lo, r.K - 1);
    const float last_hi = __shfl_sync(0xffffffffu, hi, r.K - 1);
    if (rest > last_lo) {
      const float next = __shfl_sync(0xffffffffu, won, r.K & 31);
      rest = next + key_error(ts.range_error(last_lo - key_error(err, last_lo), next), next);
    }
    if (rest > last_lo) {
      out.lo = fminf(out.lo, last_lo);
      out.hi = fmaxf(out.hi, last_hi);
    }
    if (__any_sync(0xffffffffu, out.lo <= out.hi)) {
      out.lo = -sel_warp_max(-out.lo);
      out.hi = sel_warp_max(out.hi);
    }
  }
  out.open = out.open || out.lo <= out.hi;
  return out;
}

// Gates of the selected experts from their logits (X: float or float64); m, z:
// the softmax's largest logit and sum.
template <int V, typename X>
__device__ __forceinline__ void select_gates(const X (&x)[V], int my_e, X m, X z,
                                             const SelectRule& r, const int32_t* idx,
                                             float* __restrict__ gate) {
  const int lane = threadIdx.x & 31;
  const bool softmax = r.score == MOE_SCORE_SOFTMAX;
  // the logit of slot k0 + lane (0 past the last slot); every lane takes part
  const auto slot_x = [&](int k0) {
    const int e = k0 + lane < r.K ? (r.K <= 32 ? my_e : idx[k0 + lane]) : 0;
    X v = X(0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const X w = __shfl_sync(0xffffffffu, x[j], e & 31);
      if (j == (e >> 5)) v = w;
    }
    return v;
  };
  if (!r.renorm) {
    for (int k0 = 0; k0 < r.K; k0 += 32) {
      const X xk = slot_x(k0);
      const X s = softmax ? sel_exp(xk - m) / z : sel_sigmoid(xk);
      if (k0 + lane < r.K) gate[k0 + lane] = (float)(s * (X)r.scale);
    }
    return;
  }
  // scores relative to the largest selected one, so that their sum cannot
  // underflow: e^(x - xm), or s(x) / s(xm) of sigmoids (e^(x - xm), right to
  // e^-30, where xm < -30)
  X xm = -INFINITY;
  for (int k0 = 0; k0 < r.K; k0 += 32) {
    const X xk = slot_x(k0);
    if (k0 + lane < r.K) xm = xk > xm || xk != xk ? xk : xm;
  }
  xm = sel_warp_max(xm);
  const bool ratio = !softmax && !(xm < X(-30));
  const X sm = ratio ? sel_sigmoid(xm) : X(1);
  X sum = X(0), w = X(0);
  for (int k0 = 0; k0 < r.K; k0 += 32) {
    const X xk = slot_x(k0);
    w = ratio ? sel_sigmoid(xk) / sm : sel_exp(xk - xm);
    if (k0 + lane < r.K) sum += w;
  }
  sum = sel_warp_sum(sum);
  for (int k0 = 0; k0 < r.K; k0 += 32) {
    if (r.K > 32) {
      const X xk = slot_x(k0);
      w = ratio ? sel_sigmoid(xk) / sm : sel_exp(xk - xm);
    }
    if (k0 + lane < r.K) gate[k0 + lane] = (float)(w / sum * (X)r.scale);
  }
}

// ---------------------------------------------------------------- by a block
// Shared memory of the block path, for N experts, K slots and up to
// max(256, N) threads.
struct BlockRoute {
  double* x;          // [N] logits: exact, or float32 ones where exact_f is 0
  uint32_t* ord;      // [N] keys in order form
  uint32_t* best;     // [warps][block_keep(K)] each warp's best eligible keys in order (0: none)
  float* top_key;     // [K + 1] keys in order, the best one left out last
  float* top_err;     // [K + 1] their errors
  uint16_t* top_id;   // [K + 1] their experts
  uint16_t* list;     // [N] experts whose exact logit is wanted
  uint8_t* exact_f;   // [N]
};
// Keys of one warp that can be among the first K + 1, in whole vectors of four.
__host__ __device__ __forceinline__ int block_keep(int K) {
  return K + 1 < 32 ? (K + 4) / 4 * 4 : 32;
}
__host__ __device__ __forceinline__ int block_best(int N, int K) {
  const int warps = N > 256 ? (N + 31) / 32 : 8;
  return warps * block_keep(K);
}
__host__ __device__ inline size_t block_route_bytes(int N, int K) {
  return (size_t)N * 8 + 8 + ((size_t)N + 4) * 4 + (size_t)block_best(N, K) * 4 +
         ((size_t)K + 2) * 12 + (size_t)N * 2 + N + 16;
}
__device__ __forceinline__ BlockRoute block_route_smem(uint8_t* p, int N, int K) {
  BlockRoute b;
  b.x = reinterpret_cast<double*>(p);
  b.ord = reinterpret_cast<uint32_t*>(p + (size_t)((N + 1) / 2 * 2) * 8);   // 16-byte aligned
  b.best = b.ord + (N + 3) / 4 * 4;                                         // 16-byte aligned
  b.top_key = reinterpret_cast<float*>(b.best + block_best(N, K));
  b.top_err = b.top_key + K + 1;
  b.top_id = reinterpret_cast<uint16_t*>(b.top_err + K + 1);
  b.list = b.top_id + K + 1;
  b.exact_f = reinterpret_cast<uint8_t*>(b.list + N);
  return b;
}

// Sum of v over the block, in warp order; largest of a whole number.  red: 32
// of its kind, not touched again before the block's next barrier but one.
__device__ __forceinline__ double block_sum(double v, double* red) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = sel_warp_sum(v);
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return sel_warp_sum(lane < nw ? red[lane] : 0.0);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = __reduce_max_sync(0xffffffffu, v);
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

// Routes one token by the whole block; false: exact scores that only the error
// of the softmax's sum keeps apart, so that every logit has to be exact first
// (nothing has been written).  blockDim.x >= N, whole warps; from b.x and
// b.exact_f; logit_err bounds the error of the inexact logits.
// fetch(n): fills b.x for the experts b.list[0, n) with their exact logits and
// synchronises the block.  Its last reads of b are warp 0's: the caller
// synchronises before it fills b again.
template <typename Fetch>
__device__ __forceinline__ bool block_route(const BlockRoute& b, const SelectRule& r,
                                            const float* __restrict__ bias, float logit_err,
                                            Fetch fetch, int32_t* __restrict__ idx,
                                            float* __restrict__ gate,
                                            int32_t* __restrict__ counts) {
  __shared__ double red_z[32];
  __shared__ uint32_t red_m[32], red_w[32], red_s[32];
  __shared__ float gkey[32][2], gneed[32];
  __shared__ uint32_t gerr[32];        // the largest error of the inexact keys near a group's score
  __shared__ int n_list;
  __shared__ uint32_t s_lo, s_hi;      // the keys, in order form, between which open pairs lie
  const int e = threadIdx.x, N = r.N_r, K = r.K, lane = e & 31;
  const bool softmax = r.score == MOE_SCORE_SOFTMAX, mine = e < N;
  const bool grouped = r.topk_groups < r.n_groups, two = r.group_top == 2;
  const int gs = N / r.n_groups, g = mine ? e / gs : 0;
  const float bi = bias && mine ? bias[e] : 0.f;
  double m = 0.0, z = 1.0;
  while (true) {
    __syncthreads();
    const bool ex = mine && b.exact_f[e];
    const bool all = __syncthreads_and(!mine || ex);
    const double x = mine ? b.x[e] : 0.0;
    // scores: float64 for exact logits, float32 (expf and division: within
    // 4 * 2^-23 of themselves) for the others
    float s = 0.f;
    if (softmax) {
      m = (double)sel_val(block_max(mine ? sel_ord((float)x) : 0u, red_m));
      const double ev = !mine ? 0.0 : ex ? exp(x - m) : (double)expf((float)(x - m));
      z = block_sum(ev, red_z);
      if (mine) s = ex ? (float)(ev / z) : (float)ev / (float)z;
    } else if (mine) {
      s = ex ? (float)sel_sigmoid(x) : sel_sigmoid((float)x);
    }
    const float key = bias ? s + bi : s;
    // errors of the keys, and of the softmax's sum, which exact ones share
    TokenScale ts = exact_scale();
    float eta = 0.f, smax = 0.f, ke = 0.f;
    if (!all) {
      ts.whole = softmax && !bias;
      // non-negative floats compare as whole numbers (fmaxf drops a NaN)
      const float w = __uint_as_float(
          block_max(__float_as_uint(fmaxf(0.f, ts.whole ? s : s * (1.f - s))), red_w));
      smax = __uint_as_float(block_max(__float_as_uint(fmaxf(0.f, s)), red_s));
      ts.slope = error_slope(logit_err, softmax, bias != nullptr);
      ts.flat = fmaf(4.8e-7f, smax, kFloor);
      ts.top = fmaf(ts.slope, w, ts.flat);
      eta = softmax ? logit_err : 0.f;
      if (mine && !ex) ke = key_error(ts.score_error(s), key);
      if (mine && ex && softmax) ke = key_error(bias ? 2.f * eta * s : 0.f, key);
    }
    const float err = ts.top, rel = err > 0.f ? kKeyRounding : 0.f;
    uint32_t o = mine ? sel_ord(key) : 0u;
    if (mine) b.ord[e] = o;
    if (e == 0) { n_list = 0; s_lo = 0xffffffffu; s_hi = 0u; }
    if (e < 32) { gkey[e][0] = gkey[e][1] = gneed[e] = 0.f; gerr[e] = 0u; }
    __syncthreads();
    bool want = false, z_open = false;
    if (grouped) {
      // place inside the group; the first one or two make its score
      int place = 0;
      if (mine && gs % 4 == 0) {
        const uint4* row = reinterpret_cast<const uint4*>(b.ord) + g * (gs / 4);
        const int at = e - g * gs;
#pragma unroll 4
        for (int i = 0; i < gs; i += 4) {
          const uint4 v = row[i / 4];
          place += (v.x > o || (v.x == o && i < at)) + (v.y > o || (v.y == o && i + 1 < at)) +
                   (v.z > o || (v.z == o && i + 2 < at)) + (v.w > o || (v.w == o && i + 3 < at));
        }
      } else if (mine) {
        for (int i = g * gs; i < g * gs + gs; ++i) {
          const uint32_t v = b.ord[i];
          place += v > o || (v == o && i < e);
        }
      }
      // gneed: what the last key that the group's score counts is at least
      if (mine && place < 2) gkey[g][place] = key;
      if (mine && place == (two ? 1 : 0)) gneed[g] = key - ke;
      __syncthreads();
      const bool near = mine && !ex && key + ke >= gneed[g];
      if (near) atomicMax(&gerr[g], __float_as_uint(ke));
      __syncthreads();
      // groups: lane q of every warp holds group q
      const bool has = lane < r.n_groups;
      const float gsc = has ? (two ? gkey[lane][0] + gkey[lane][1] : gkey[lane][0]) : 0.f;
      const uint32_t go = has ? sel_ord(gsc) : 0u;
      // a score with an inexact key near it: that error for each key it counts (an exact
      // one among them has less), and the sum's rounding
      const float gmax = has ? __uint_as_float(gerr[lane]) : 0.f;
      const float ge = gmax > 0.f ? r.group_top * gmax +
                                        rel * group_rounding(gkey[lane][0], two ? gkey[lane][1] : 0.f)
                                  : 0.f;
      int before = 0;
      for (int q = 0; q < r.n_groups; ++q) {
        const uint32_t v = __shfl_sync(0xffffffffu, go, q);
        before += v > go || (v == go && q < lane);
      }
      const bool keep = has && before < r.topk_groups;
      const unsigned kept = __ballot_sync(0xffffffffu, keep);
      // The choice is open where a kept group's score may lie below that of one
      // left out; the inexact members of the groups that can be either are wanted.
      // (NaN scores are exact and come first: they open nothing.)
      const bool number = has && gsc == gsc;
      const float least = -sel_warp_max(number && keep ? ge - gsc : -INFINITY);
      const float most = sel_warp_max(number && !keep ? gsc + ge : -INFINITY);
      if (least < most) {
        const float mine_sc = two ? gkey[g][0] + gkey[g][1] : gkey[g][0];
        const float mine_ge = __shfl_sync(0xffffffffu, ge, g);
        want = near && (((kept >> g) & 1u) ? mine_sc - mine_ge < most : mine_sc + mine_ge > least);
      } else if (eta > 0.f) {
        // Scores that no member's error joins: the error of the softmax's sum, which a
        // bias lets tell groups apart, and the keys' roundings may still.
        const float gr = sel_warp_max(has ? group_rounding(gkey[lane][0], two ? gkey[lane][1] : 0.f) : 0.f);
        const float ze = 2.f * kKeyRounding * gr + (bias ? 2.f * r.group_top * eta * smax : 0.f);
        z_open = least - most <= ze;
      }
      if (mine && !((kept >> g) & 1u)) o = 0u;
    }
    // place in the order: how many eligible keys come before.  First inside the
    // warp, whose best `keep` go into its row of b.best; only they can be among
    // the first K + 1, and they count the other warps' rows.
    const int warp = e >> 5, nw = blockDim.x >> 5;
    int place = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t v = __shfl_sync(0xffffffffu, o, i);
      place += v > o || (v == o && i < lane);
    }
    const int keep = block_keep(K), n4 = keep / 4;
    if (place < keep) b.best[warp * keep + place] = o;
    __syncthreads();
    if (o != 0u && place <= K) {
      const uint4* row = reinterpret_cast<const uint4*>(b.best);
      int i = 0;
#pragma unroll 4
      for (; i < warp * n4; ++i) {                   // an equal key of a lower expert comes first
        const uint4 v = row[i];
        place += (v.x >= o) + (v.y >= o) + (v.z >= o) + (v.w >= o);
      }
      i += n4;
#pragma unroll 4
      for (; i < nw * n4; ++i) {
        const uint4 v = row[i];
        place += (v.x > o) + (v.y > o) + (v.z > o) + (v.w > o);
      }
    }
    const bool placed = mine && o != 0u && place <= K;
    if (placed) {
      b.top_key[place] = key;
      b.top_err[place] = ke;
      b.top_id[place] = (uint16_t)e;
    }
    const int n_top = __syncthreads_count(placed);   // K + 1, or K where no other is eligible
    bool open = false;
    if (!all) {
      // key a of expert ia comes before key c of expert ic: may their errors turn
      // them around?  Of two exact keys only the softmax's sum's can.
      const auto pair = [&](float a, float ea, int ia, float c, float ec, int ic) {
        if (b.exact_f[ia] && b.exact_f[ic]) {
          const float gap = bias ? fabsf((a - bias[ia]) - (c - bias[ic])) : 0.f;
          if (eta > 0.f && a - c <= 2.f * eta * gap + 2.f * kKeyRounding * fmaxf(fabsf(a), fabsf(c)))
            z_open = true;
        } else if (a - c < ea + ec) {
          atomicMin(&s_lo, sel_ord(c - ec));
          atomicMax(&s_hi, sel_ord(a + ea));
        }
      };
      for (int k = e; k + 1 < n_top; k += blockDim.x)
        pair(b.top_key[k], b.top_err[k], b.top_id[k], b.top_key[k + 1], b.top_err[k + 1],
             b.top_id[k + 1]);
      // the last one kept against the experts further down
      if (o != 0u && !placed) pair(b.top_key[K - 1], b.top_err[K - 1], b.top_id[K - 1], key, ke, e);
      if (__syncthreads_or(z_open)) return false;
      if (s_hi != 0u && o != 0u && !ex)
        want = want || takes_part(key, ke, sel_val(s_lo), sel_val(s_hi));
      open = __syncthreads_or(want);
    }
    if (!open) break;
    if (want) b.list[atomicAdd(&n_list, 1)] = (uint16_t)e;
    __syncthreads();
    fetch(n_list);
    if (want) b.exact_f[e] = 1;
  }
  // slots: load, and the gates by warp 0 (every logit in float64)
  for (int k = e; k < K; k += blockDim.x) {
    const int id = b.top_id[k];
    idx[k] = id;
    atomicAdd(&counts[id], 1);
  }
  if (e >= 32) return true;
  const auto slot_x = [&](int k) { return b.x[b.top_id[k]]; };
  double xm = -INFINITY, sm = 1.0, sum = 1.0;
  bool ratio = false;
  if (r.renorm) {
    for (int k = lane; k < K; k += 32) {
      const double v = slot_x(k);
      xm = v > xm || v != v ? v : xm;
    }
    xm = sel_warp_max(xm);
    ratio = !softmax && !(xm < -30.0);
    if (ratio) sm = sel_sigmoid(xm);
    sum = 0.0;
    for (int k = lane; k < K; k += 32)
      sum += ratio ? sel_sigmoid(slot_x(k)) / sm : exp(slot_x(k) - xm);
    sum = sel_warp_sum(sum);
  } else if (softmax) {
    xm = m;
    sum = z;
  } else {
    ratio = true;
  }
  for (int k = lane; k < K; k += 32) {
    const double v = slot_x(k);
    gate[k] = (float)((ratio ? sel_sigmoid(v) / sm : exp(v - xm)) / sum * (double)r.scale);
  }
  return true;
}

}  // namespace moe
